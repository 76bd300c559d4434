// blk_norm.hip -- the norm after a block with its gate, the scaled residual and the
// norm before the next block, in one pass over the rows, and its gradients
// (block_norm, block_norm_backward).
#include "blk_common.hpp"

namespace blk {

constexpr int kMaxHidden = 32768;

struct NormArgs {
    int32_t tokens, hidden;
    int32_t post, pre, gate_kind, gate_act;
    int32_t wide_weights;  // weights and channel gate in fp32, else in the rows' type
    float residual_scale, branch_scale, eps;
    const void *x, *branch, *gate, *post_weight, *pre_weight;
    void *h, *y;
    uint64_t x_ld, branch_ld, gate_ld, h_ld, y_ld;
    // backward
    const void *dh, *dy;
    void *dx, *dbranch, *dgate;
    uint64_t dh_ld, dy_ld, dx_ld, dbranch_ld, dgate_ld;
    float* part;           // [workgroups][sums][hidden]
    int32_t sums;          // weight gradients wanted: 0 .. 3
    int32_t at_pre, at_post, at_gate;  // their places among the sums, or -1
};

__device__ __forceinline__ float gate_value(int act, float z) {
    return act == RR_ACT_SIGMOID ? logistic(z) : act == RR_ACT_SILU ? z * logistic(z) : z;
}
__device__ __forceinline__ float gate_slope(int act, float z) {
    return act == RR_ACT_SIGMOID ? slope_of<RR_ACT_SIGMOID>(z) : act == RR_ACT_SILU ? slope_of<RR_ACT_SILU>(z) : 1.0f;
}

// Where the columns of a row lie: thread g of G holds NV vectors, vector v at column
// (v * G + g) * N, so that every access of a wave is one stretch of the row.
template <typename T, int G, int NV> struct Row {
    static constexpr int N = Vec<T>::N;
    __device__ static int column(int v) { return (v * G + (int)threadIdx.x % G) * N; }

    __device__ static void load(Vec<T> (&r)[NV], const void* p, uint64_t ld, int64_t t, int len) {
        const T* row = (const T*)p + (uint64_t)t * ld;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (column(v) < len) r[v] = load_vec(row, column(v), len);
    }
    __device__ static void zero(Vec<T> (&r)[NV]) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < N; ++i) r[v].e[i] = (T)0.0f;
    }
    __device__ static void store(const Vec<T> (&r)[NV], void* p, uint64_t ld, int64_t t, int len) {
        T* row = (T*)p + (uint64_t)t * ld;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (column(v) < len) store_vec(row, column(v), len, r[v]);
    }
    // weights of these columns; 1 where there are none
    __device__ static void weights(float (&w)[NV][N], const void* p, bool wide, int len) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int c = column(v) + i;
                w[v][i] = !p || c >= len ? 1.0f
                          : wide         ? ((const float*)p)[c]
                                         : (float)((const T*)p)[c];
            }
    }
};

// K sums over the G threads of a row, to all of them: lanes first, then the waves
// through LDS (a slot per call, so that one barrier a call is enough).
template <int G, int K>
__device__ __forceinline__ void row_sums(float (&s)[K], float* lds) {
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = lane_sum<64>(s[k]);
    if constexpr (G > 64) {
        constexpr int W = G / 64;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) lds[k * W + (threadIdx.x >> 6)] = s[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            s[k] = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) s[k] += lds[k * W + w];
        }
    }
}

template <int G> struct Shape {
    static constexpr int block = G < 256 ? 256 : G;
    static constexpr int rows = block / G;  // rows of a workgroup at a time
};

template <typename T, int G, int NV>
__global__ void __launch_bounds__(Shape<G>::block) norm_kernel(const NormArgs a) {
    typedef Row<T, G, NV> R;
    constexpr int N = Vec<T>::N;
    __shared__ float lds[2][2][16];
    const int len = a.hidden;
    float wp[NV][N], wn[NV][N], wg[NV][N];
    R::weights(wp, a.post_weight, a.wide_weights, len);
    R::weights(wn, a.pre_weight, a.wide_weights, len);
    R::weights(wg, a.gate_kind == RR_GATE_CHANNEL ? a.gate : nullptr, a.wide_weights, len);
    const float inv = 1.0f / (float)len;
    int turn = 0;
    // G >= 256: one row a workgroup, so every wave takes the same turns of this loop
    for (int64_t t = (int64_t)blockIdx.x * Shape<G>::rows + threadIdx.x / G; t < a.tokens;
         t += (int64_t)gridDim.x * Shape<G>::rows, turn ^= 1) {
        Vec<T> x[NV], u[NV], g[NV];
        R::zero(x);
        R::zero(u);
        R::zero(g);
        R::load(x, a.x, a.x_ld, t, len);
        if (a.branch) R::load(u, a.branch, a.branch_ld, t, len);
        if (a.gate_kind == RR_GATE_ELEMENT) R::load(g, a.gate, a.gate_ld, t, len);
        float h[NV][N];
        float r = 1.0f;
        if (a.post) {
            float s[1] = {0.0f};
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < N; ++i) s[0] = fmaf((float)u[v].e[i], (float)u[v].e[i], s[0]);
            row_sums<G>(s, lds[turn][0]);
            r = rsqrtf(fmaf(s[0], inv, a.eps));
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                h[v][i] = a.residual_scale * (float)x[v].e[i];
                if (a.branch) {
                    float n = (float)u[v].e[i] * r * wp[v][i];
                    if (a.gate_kind == RR_GATE_ELEMENT) n *= gate_value(a.gate_act, (float)g[v].e[i]);
                    if (a.gate_kind == RR_GATE_CHANNEL) n *= gate_value(a.gate_act, wg[v][i]);
                    h[v][i] = fmaf(a.branch_scale, n, h[v][i]);
                }
                if (R::column(v) + i >= len) h[v][i] = 0.0f;
                s[0] = fmaf(h[v][i], h[v][i], s[0]);
                x[v].e[i] = (T)h[v][i];
            }
        if (a.h) R::store(x, a.h, a.h_ld, t, len);
        if (a.pre) {
            row_sums<G>(s, lds[turn][1]);
            const float q = rsqrtf(fmaf(s[0], inv, a.eps));
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < N; ++i) x[v].e[i] = (T)(h[v][i] * q * wn[v][i]);
            R::store(x, a.y, a.y_ld, t, len);
        }
    }
}

// The gradients.  With q = (mean(h^2) + eps)^-1/2 and p = dy * pre_weight,
//   d  = dh + q p - h q^3 mean(p h)                 gradient at the stream
//   dx = residual_scale d
// and with r the same of the branch u, n = u r post_weight, e = branch_scale d:
//   dgate = e n act'(gate);   m = e act(gate) post_weight
//   du = r m - u r^3 mean(m u)
//   dpre_weight = sum_t dy h q;  dpost_weight = sum_t e act(gate) u r.
// Two rounds of sums over a row: (h^2, p h, u^2), then (m u).  The statistics are
// computed again from the rows, which are read anyway, instead of being stored by
// the forward call.  The sums over tokens stay in registers over all rows that a
// workgroup takes, and the workgroups' parts are added by a second, short kernel
// in a fixed order.
template <typename T, int G, int NV>
__global__ void __launch_bounds__(Shape<G>::block) norm_backward_kernel(const NormArgs a) {
    typedef Row<T, G, NV> R;
    constexpr int N = Vec<T>::N;
    __shared__ float lds[2][4][16];
    const int len = a.hidden;
    float wp[NV][N], wn[NV][N], wg[NV][N];
    R::weights(wp, a.post_weight, a.wide_weights, len);
    R::weights(wn, a.pre_weight, a.wide_weights, len);
    R::weights(wg, a.gate_kind == RR_GATE_CHANNEL ? a.gate : nullptr, a.wide_weights, len);
    float sum_pre[NV][N], sum_post[NV][N], sum_gate[NV][N];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < N; ++i) sum_pre[v][i] = sum_post[v][i] = sum_gate[v][i] = 0.0f;
    const float inv = 1.0f / (float)len;
    int turn = 0;
    for (int64_t t = (int64_t)blockIdx.x * Shape<G>::rows + threadIdx.x / G; t < a.tokens;
         t += (int64_t)gridDim.x * Shape<G>::rows, turn ^= 1) {
        Vec<T> dh[NV], dy[NV], h[NV], u[NV], g[NV];
        R::zero(dh);
        R::zero(dy);
        R::zero(h);
        R::zero(u);
        R::zero(g);
        if (a.dh) R::load(dh, a.dh, a.dh_ld, t, len);
        if (a.pre) {
            R::load(dy, a.dy, a.dy_ld, t, len);
            R::load(h, a.h, a.h_ld, t, len);
        }
        if (a.branch) R::load(u, a.branch, a.branch_ld, t, len);
        if (a.gate_kind == RR_GATE_ELEMENT) R::load(g, a.gate, a.gate_ld, t, len);
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float hv = (float)h[v].e[i], uv = (float)u[v].e[i];
                s[0] = fmaf(hv, hv, s[0]);
                s[1] = fmaf((float)dy[v].e[i] * wn[v][i], hv, s[1]);
                s[2] = fmaf(uv, uv, s[2]);
            }
        if (a.pre || a.post) row_sums<G>(s, lds[turn][0]);
        const float q = rsqrtf(fmaf(s[0], inv, a.eps));
        const float back = q * q * q * s[1] * inv;
        const float r = a.post ? rsqrtf(fmaf(s[2], inv, a.eps)) : 1.0f;
        float m[NV][N];
        float s2[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float d = (float)dh[v].e[i];
                if (a.pre) {
                    const float hv = (float)h[v].e[i], dyv = (float)dy[v].e[i];
                    d += fmaf(q * wn[v][i], dyv, -back * hv);
                    sum_pre[v][i] = fmaf(dyv * q, hv, sum_pre[v][i]);
                }
                dh[v].e[i] = (T)(a.residual_scale * d);
                float e = a.branch_scale * d;
                const float unit = (float)u[v].e[i] * r;
                if (a.gate_kind != RR_GATE_NONE) {
                    const float z = a.gate_kind == RR_GATE_ELEMENT ? (float)g[v].e[i] : wg[v][i];
                    const float dg = e * unit * wp[v][i] * gate_slope(a.gate_act, z);
                    g[v].e[i] = (T)dg;
                    sum_gate[v][i] += dg;
                    e *= gate_value(a.gate_act, z);
                }
                sum_post[v][i] = fmaf(e, unit, sum_post[v][i]);
                m[v][i] = e * wp[v][i];
                s2[0] = fmaf(m[v][i], (float)u[v].e[i], s2[0]);
            }
        if (a.dx) R::store(dh, a.dx, a.dx_ld, t, len);
        if (a.dgate) R::store(g, a.dgate, a.dgate_ld, t, len);
        if (a.dbranch) {
            float bu = 0.0f;
            if (a.post) {
                row_sums<G>(s2, lds[turn][3]);
                bu = r * r * r * s2[0] * inv;
            }
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    u[v].e[i] = (T)fmaf(r, m[v][i], -bu * (float)u[v].e[i]);
            R::store(u, a.dbranch, a.dbranch_ld, t, len);
        }
    }
    if (a.sums == 0) return;
    // one part for each row a workgroup takes at a time
    const int64_t part = (int64_t)blockIdx.x * Shape<G>::rows + threadIdx.x / G;
    float* to = a.part + (uint64_t)part * a.sums * len;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = R::column(v) + i;
            if (c >= len) continue;
            if (a.at_pre >= 0) to[(uint64_t)a.at_pre * len + c] = sum_pre[v][i];
            if (a.at_post >= 0) to[(uint64_t)a.at_post * len + c] = sum_post[v][i];
            if (a.at_gate >= 0) to[(uint64_t)a.at_gate * len + c] = sum_gate[v][i];
        }
}

// Adds the parts of one gradient: 16 columns a workgroup, 16 threads each.
__global__ void __launch_bounds__(256)
norm_parts_kernel(const float* part, int parts, uint64_t stride, int hidden, float* o0, float* o1,
                  float* o2) {
    __shared__ float lds[16][17];
    const int col = blockIdx.x * 16 + (threadIdx.x & 15), s = threadIdx.x >> 4;
    float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
    float sum = 0.0f;
    if (col < hidden)
        for (int p = s; p < parts; p += 16)
            sum += part[(uint64_t)p * stride + (uint64_t)blockIdx.y * hidden + col];
    lds[s][threadIdx.x & 15] = sum;
    __syncthreads();
    if (s == 0 && col < hidden) {
        float all = 0.0f;
        for (int q = 0; q < 16; ++q) all += lds[q][threadIdx.x];
        out[col] = all;
    }
}

// ------------------------------------------------------------------ host side --

struct Config {
    int group, vecs;
};

// Threads and vectors per row.  A row of few vectors goes to one wave (no barrier);
// a longer one to as many threads as keep it in registers.
static Config pick(int hidden, int dt) {
    const int n = (int)(16 / type_bytes(dt));
    const int vecs = (int)ceil_div(hidden, n);
    if (vecs <= 64) return {64, 1};
    if (vecs <= 128) return {64, 2};
    if (vecs <= 256) return {256, 1};
    if (vecs <= 512) return {256, 2};
    if (vecs <= 1024) return {512, 2};
    if (vecs <= 2048) return {1024, 2};
    if (vecs <= 4096) return {1024, 4};
    return {1024, 8};   // fp32 rows beyond 16384
}
static int rows_of(const Config& c) { return c.group < 256 ? 256 / c.group : 1; }

// Workgroups: enough to fill every compute unit with as many as fit, so that each
// keeps the weights in registers over many rows.
static unsigned grid_of(const Config& c, size_t tokens, int per_cu) {
    const int cus = compute_units();
    const uint64_t want = ceil_div(tokens, rows_of(c));
    const uint64_t most = (uint64_t)(cus > 0 ? cus : 256) * per_cu;
    return (unsigned)(want < most ? want : most);
}
constexpr int kForwardPerCu = 8, kBackwardPerCu = 2;

#define BLK_NORM_LAUNCH(KERNEL, T, c, grid, s, a)                                     \
    if (c.group == 64 && c.vecs == 1) KERNEL<T, 64, 1><<<grid, 256, 0, s>>>(a);       \
    else if (c.group == 64) KERNEL<T, 64, 2><<<grid, 256, 0, s>>>(a);                 \
    else if (c.group == 256 && c.vecs == 1) KERNEL<T, 256, 1><<<grid, 256, 0, s>>>(a);\
    else if (c.group == 256) KERNEL<T, 256, 2><<<grid, 256, 0, s>>>(a);               \
    else if (c.group == 512) KERNEL<T, 512, 2><<<grid, 512, 0, s>>>(a);               \
    else if (c.vecs == 2) KERNEL<T, 1024, 2><<<grid, 1024, 0, s>>>(a);                \
    else if (c.vecs == 4) KERNEL<T, 1024, 4><<<grid, 1024, 0, s>>>(a);                \
    else if constexpr (sizeof(T) == 4) KERNEL<T, 1024, 8><<<grid, 1024, 0, s>>>(a);

static bool rows_ok(const rr_rows_t& r, size_t tokens, size_t hidden, int dt) {
    return tokens == 0 ||
           (r.data && aligned_to(r.data, type_bytes(dt)) && r.ld >= hidden && r.ld <= (1ull << 40));
}
static bool rows_ok_if(const rr_rows_t& r, size_t tokens, size_t hidden, int dt) {
    return !r.data || rows_ok(r, tokens, hidden, dt);
}

static rr_status_t check_norm(const rr_norm_t* a) {
    if (!a) return RR_ERR_INVALID;
    if (!is_float_type(a->dt) || (a->weight_dt != a->dt && a->weight_dt != RR_FP32))
        return RR_ERR_INVALID;
    if (a->hidden < 1 || (a->post_norm & ~1) || (a->pre_norm & ~1) || a->reserved)
        return RR_ERR_INVALID;
    if (a->hidden > kMaxHidden || a->tokens > (1ull << 40)) return RR_ERR_UNSUPPORTED;
    if (a->tokens > 0x7FFFFFFFull) return RR_ERR_UNSUPPORTED;
    if (a->gate_kind != RR_GATE_NONE && a->gate_kind != RR_GATE_CHANNEL &&
        a->gate_kind != RR_GATE_ELEMENT)
        return RR_ERR_INVALID;
    if (a->gate_act != RR_ACT_NONE && a->gate_act != RR_ACT_SIGMOID && a->gate_act != RR_ACT_SILU)
        return RR_ERR_INVALID;
    if (!(a->eps >= 0.0f)) return RR_ERR_INVALID;
    if (!a->branch.data && a->tokens && (a->post_norm || a->gate_kind != RR_GATE_NONE))
        return RR_ERR_INVALID;
    if (a->gate_kind == RR_GATE_NONE && (a->gate.data || a->gate_act != RR_ACT_NONE))
        return RR_ERR_INVALID;
    const uint64_t wb = type_bytes(a->weight_dt);
    if (!aligned_to(a->post_weight, wb) || !aligned_to(a->pre_weight, wb)) return RR_ERR_INVALID;
    if (!rows_ok_if(a->branch, a->tokens, a->hidden, a->dt)) return RR_ERR_INVALID;
    if (a->gate_kind == RR_GATE_ELEMENT && !rows_ok(a->gate, a->tokens, a->hidden, a->dt))
        return RR_ERR_INVALID;
    if (a->gate_kind == RR_GATE_CHANNEL && (!a->gate.data || !aligned_to(a->gate.data, wb)))
        return RR_ERR_INVALID;
    return RR_OK;
}

struct Span {
    const void* p;
    uint64_t n;
    uint64_t ld;
};
static Span span(const rr_norm_t* a, const rr_rows_t& r) {
    return {r.data, r.data ? extent(a->tokens, r.ld, a->hidden, type_bytes(a->dt)) : 0, r.ld};
}
static Span flat(const void* p, uint64_t n) { return {p, p ? n : 0, 0}; }
static bool meet(const Span& a, const Span& b) { return overlap(a.p, a.n, b.p, b.n); }
// the same rows, which a kernel reads before it writes them
static bool same(const Span& a, const Span& b) { return a.p == b.p && a.ld == b.ld; }

static NormArgs args_of(const rr_norm_t* a) {
    NormArgs k = {};
    k.tokens = (int32_t)a->tokens;
    k.hidden = (int32_t)a->hidden;
    k.post = a->post_norm;
    k.pre = a->pre_norm;
    k.gate_kind = a->gate_kind;
    k.gate_act = a->gate_act;
    k.wide_weights = a->weight_dt == RR_FP32;
    k.residual_scale = a->residual_scale;
    k.branch_scale = a->branch_scale;
    k.eps = a->eps;
    k.x = a->x.data;
    k.x_ld = a->x.ld;
    k.branch = a->branch.data;
    k.branch_ld = a->branch.ld;
    k.gate = a->gate.data;
    k.gate_ld = a->gate.ld;
    k.post_weight = a->post_weight;
    k.pre_weight = a->pre_weight;
    k.h = a->h.data;
    k.h_ld = a->h.ld;
    k.y = a->y.data;
    k.y_ld = a->y.ld;
    return k;
}

static int sums_of(const rr_norm_grad_t* g) {
    return (g->dpre_weight != nullptr) + (g->dpost_weight != nullptr) +
           (g->dgate_channel != nullptr);
}

// Parts of the sums over tokens: one for each row the grid takes at a time.
static uint64_t parts_of(const rr_norm_t* a) {
    const Config c = pick((int)a->hidden, a->dt);
    return (uint64_t)grid_of(c, a->tokens, kBackwardPerCu) * rows_of(c);
}

static rr_status_t check_norm_grad(const rr_norm_t* a, const rr_norm_grad_t* g) {
    const rr_status_t st = check_norm(a);
    if (st != RR_OK) return st;
    if (!g) return RR_ERR_INVALID;
    const size_t t = a->tokens, h = a->hidden;
    if (a->pre_norm && (!rows_ok(g->dy, t, h, a->dt) || !rows_ok(a->h, t, h, a->dt)))
        return RR_ERR_INVALID;
    if (!a->pre_norm && (g->dy.data || g->dpre_weight)) return RR_ERR_INVALID;
    if (!a->post_norm && g->dpost_weight) return RR_ERR_INVALID;
    if (a->gate_kind != RR_GATE_CHANNEL && g->dgate_channel) return RR_ERR_INVALID;
    if (a->gate_kind != RR_GATE_ELEMENT && g->dgate.data) return RR_ERR_INVALID;
    if (t && !a->branch.data && g->dbranch.data) return RR_ERR_INVALID;
    if (!rows_ok_if(g->dh, t, h, a->dt) || !rows_ok_if(g->dx, t, h, a->dt) ||
        !rows_ok_if(g->dbranch, t, h, a->dt) || !rows_ok_if(g->dgate, t, h, a->dt))
        return RR_ERR_INVALID;
    if (!aligned_to(g->dgate_channel, 4) || !aligned_to(g->dpost_weight, 4) ||
        !aligned_to(g->dpre_weight, 4))
        return RR_ERR_INVALID;
    return RR_OK;
}

}  // namespace blk

using namespace blk;

extern "C" {

rr_status_t block_norm(const rr_norm_t* a, rr_stream_t stream) {
    const rr_status_t st = check_norm(a);
    if (st != RR_OK) return st;
    const size_t t = a->tokens, h = a->hidden;
    if (!rows_ok(a->x, t, h, a->dt) || !rows_ok_if(a->h, t, h, a->dt)) return RR_ERR_INVALID;
    if (a->pre_norm ? !rows_ok(a->y, t, h, a->dt) : a->y.data != nullptr) return RR_ERR_INVALID;
    if (t && !a->h.data && !a->pre_norm) return RR_ERR_INVALID;
    const uint64_t wn = h * type_bytes(a->weight_dt);
    const Span x = span(a, a->x), u = span(a, a->branch), sh = span(a, a->h), sy = span(a, a->y);
    const Span gate = a->gate_kind == RR_GATE_ELEMENT ? span(a, a->gate) : flat(a->gate.data, wn);
    const Span wa = flat(a->post_weight, wn), wb = flat(a->pre_weight, wn);
    if (meet(sh, sy)) return RR_ERR_INVALID;
    for (const Span& o : {sh, sy}) {
        if (meet(o, gate) || meet(o, wa) || meet(o, wb)) return RR_ERR_INVALID;
        if (meet(o, x) && !(o.p == sh.p && same(o, x))) return RR_ERR_INVALID;
        if (meet(o, u) && !(o.p == sy.p && same(o, u))) return RR_ERR_INVALID;
    }
    if (t == 0) return RR_OK;
    const NormArgs k = args_of(a);
    const Config c = pick((int)h, a->dt);
    const unsigned grid = grid_of(c, t, kForwardPerCu);
    hipStream_t s = (hipStream_t)stream;
    switch (a->dt) {
        case RR_FP32: { BLK_NORM_LAUNCH(norm_kernel, float, c, grid, s, k) break; }
        case RR_BF16: { BLK_NORM_LAUNCH(norm_kernel, bf16, c, grid, s, k) break; }
        default: { BLK_NORM_LAUNCH(norm_kernel, f16, c, grid, s, k) break; }
    }
    return launched();
}

rr_status_t block_norm_backward_workspace(const rr_norm_t* a, const rr_norm_grad_t* g,
                                          size_t* bytes) {
    if (!bytes) return RR_ERR_INVALID;
    const rr_status_t st = check_norm_grad(a, g);
    if (st != RR_OK) return st;
    *bytes = (size_t)sums_of(g) * parts_of(a) * a->hidden * sizeof(float);
    return RR_OK;
}

rr_status_t block_norm_backward(const rr_norm_t* a, const rr_norm_grad_t* g, void* workspace,
                                size_t workspace_bytes, rr_stream_t stream) {
    rr_status_t st = check_norm_grad(a, g);
    if (st != RR_OK) return st;
    size_t need = 0;
    if ((st = block_norm_backward_workspace(a, g, &need)) != RR_OK) return st;
    if (need && (!workspace || !aligned_to(workspace, 4) || workspace_bytes < need))
        return RR_ERR_INVALID;
    const size_t t = a->tokens, h = a->hidden;
    const uint64_t wn = h * type_bytes(a->weight_dt), fn = h * sizeof(float);
    const Span dh = span(a, g->dh), dy = span(a, g->dy), dx = span(a, g->dx),
               du = span(a, g->dbranch);
    const Span in[] = {dh, dy, a->pre_norm ? span(a, a->h) : flat(nullptr, 0), span(a, a->branch),
                       a->gate_kind == RR_GATE_ELEMENT ? span(a, a->gate) : flat(a->gate.data, wn),
                       flat(a->post_weight, wn), flat(a->pre_weight, wn)};
    const Span out[] = {dx, du, span(a, g->dgate), flat(g->dgate_channel, fn),
                        flat(g->dpost_weight, fn), flat(g->dpre_weight, fn), flat(workspace, need)};
    for (const Span& o : out) {
        for (const Span& i : in)
            if (meet(o, i) && !(o.p == dx.p && i.p == dh.p && same(dx, dh)) &&
                !(o.p == du.p && i.p == dy.p && same(du, dy)))
                return RR_ERR_INVALID;
        for (const Span& q : out)
            if (&q != &o && meet(o, q)) return RR_ERR_INVALID;
    }
    NormArgs k = args_of(a);
    k.dh = g->dh.data;
    k.dh_ld = g->dh.ld;
    k.dy = g->dy.data;
    k.dy_ld = g->dy.ld;
    k.dx = g->dx.data;
    k.dx_ld = g->dx.ld;
    k.dbranch = g->dbranch.data;
    k.dbranch_ld = g->dbranch.ld;
    k.dgate = g->dgate.data;
    k.dgate_ld = g->dgate.ld;
    k.part = (float*)workspace;
    k.at_pre = k.at_post = k.at_gate = -1;
    float* sums[3] = {nullptr, nullptr, nullptr};
    if (g->dpre_weight) sums[k.at_pre = k.sums++] = g->dpre_weight;
    if (g->dpost_weight) sums[k.at_post = k.sums++] = g->dpost_weight;
    if (g->dgate_channel) sums[k.at_gate = k.sums++] = g->dgate_channel;
    const Config c = pick((int)h, a->dt);
    const unsigned grid = grid_of(c, t, kBackwardPerCu);
    hipStream_t s = (hipStream_t)stream;
    if (t) {
        switch (a->dt) {
            case RR_FP32: { BLK_NORM_LAUNCH(norm_backward_kernel, float, c, grid, s, k) break; }
            case RR_BF16: { BLK_NORM_LAUNCH(norm_backward_kernel, bf16, c, grid, s, k) break; }
            default: { BLK_NORM_LAUNCH(norm_backward_kernel, f16, c, grid, s, k) break; }
        }
        if ((st = launched()) != RR_OK) return st;
    }
    if (k.sums) {
        const dim3 parts((unsigned)ceil_div(h, 16), (unsigned)k.sums);
        norm_parts_kernel<<<parts, 256, 0, s>>>(k.part, (int)parts_of(a), (uint64_t)k.sums * h,
                                                (int)h, sums[0], sums[1], sums[2]);
        if ((st = launched()) != RR_OK) return st;
    }
    return RR_OK;
}

}  // extern "C"
