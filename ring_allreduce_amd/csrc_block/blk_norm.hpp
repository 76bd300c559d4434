// blk_norm.hpp -- the kernels of block_norm and its gradients.
#pragma once

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
    float *dpre, *dpost, *dgate_channel;
    const void* any;       // a matrix that is there
    uint64_t any_ld;
};

// act(z) and act'(z) of a gate.
__device__ __forceinline__ float gate_value(int act, float z) {
    const float q = logistic(z);
    return act == RR_ACT_SILU ? z * q : act == RR_ACT_SIGMOID ? q : z;
}
__device__ __forceinline__ float gate_slope(int act, float z) {
    const float q = logistic(z);
    return act == RR_ACT_NONE ? 1.0f : act == RR_ACT_SILU ? q * (1.0f + z * (1.0f - q)) : q * (1.0f - q);
}

// Where the columns of a row lie: thread g of G holds NV vectors, vector v at column
// (v * G + g) * N, so that every access of a wave is one stretch of the row.  Loads have
// no branches: a vector that reaches past the row is read so that it ends with the row,
// and mended once all loads are on their way (TINY: a row shorter than a vector, element
// by element).
template <typename T, int G, int NV, bool TINY> struct Row {
    static constexpr int N = Vec<T>::N;
    __device__ __forceinline__ static int column(int v) { return (v * G + (int)threadIdx.x % G) * N; }

    __device__ __forceinline__ static void load(u32x4 (&r)[NV], const void* p, uint64_t ld, int64_t t, int len) {
        const T* row = (const T*)p + (uint64_t)t * ld;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if constexpr (TINY) r[v] = __builtin_bit_cast(u32x4, load_vec(row, column(v), len));
            else r[v] = load_raw(row + min(column(v), len - N));
        }
    }
    __device__ __forceinline__ static void mend(u32x4 (&r)[NV], int len) {
        if constexpr (TINY) return;
        if (len % N == 0) {
            if (G * NV * N == len) return;
#pragma unroll
            for (int v = 0; v < NV; ++v) r[v] = zero_unless(column(v) < len, r[v]);
        } else {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                r[v] = drop_first(r[v], (int)sizeof(T) * min(max(column(v) + N - len, 0), N));
        }
    }
    __device__ __forceinline__ static void zero(u32x4 (&r)[NV]) {
#pragma unroll
        for (int v = 0; v < NV; ++v) r[v] = u32x4{0, 0, 0, 0};
    }
    __device__ __forceinline__ static void store(const Vec<T>& r, int v, void* p, uint64_t ld, int64_t t, int len) {
        if (column(v) < len) store_vec((T*)p + (uint64_t)t * ld, column(v), len, r);
    }
    __device__ __forceinline__ static void store(const Vec<T> (&r)[NV], void* p, uint64_t ld, int64_t t, int len) {
        T* row = (T*)p + (uint64_t)t * ld;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (column(v) < len) store_vec(row, column(v), len, r[v]);
    }
    // weights of vector v's columns; 1 where there are none.  Read where they are used: they
    // stay in the caches, while registers for them would take workgroups off the compute units.
    __device__ __forceinline__ static void weights(float (&w)[N], const void* p, bool wide, int v, int len) {
        const int c = column(v);
        if (!p) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = 1.0f;
        } else if (TINY) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                w[i] = c + i >= len ? 0.0f : wide ? ((const float*)p)[c + i] : (float)((const T*)p)[c + i];
        } else if (wide) {
            const int at = min(c, len - N);
            u32x4 r[N / 4];
#pragma unroll
            for (int h = 0; h < N / 4; ++h) r[h] = zero_unless(c < len, load_raw((const float*)p + at + h * 4));
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __uint_as_float(r[i / 4][i % 4]);
            if (len % N) {
                const int skip = c - at;
#pragma unroll
                for (int s = N / 2; s > 0; s >>= 1)
#pragma unroll
                    for (int i = 0; i < N; ++i) w[i] = skip & s ? (i + s < N ? w[i + s < N ? i + s : i] : 0.0f) : w[i];
            }
        } else {
            const int at = min(c, len - N);
            u32x4 raw = zero_unless(c < len, load_raw((const T*)p + at));
            if (len % N) raw = drop_first(raw, (int)sizeof(T) * min(c - at, N));
            const Vec<T> r = vec_of<T>(raw);
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = (float)r.e[i];
        }
    }
    __device__ __forceinline__ static float value(const u32x4 (&r)[NV], int v, int i) {
        return (float)vec_of<T>(r[v]).e[i];
    }
};

// K sums over the G threads of a row, to all of them: lanes first, then the waves
// through LDS (a slot per call, so that one barrier a call is enough).
template <int G, int K>
__device__ __forceinline__ void row_sums(float (&s)[K], float* lds) {
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = lane_sum<(G < 64 ? G : 64)>(s[k]);
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

// One row per G threads, and as many workgroups as rows ask for: a row is its own chain of
// load, sum, sum, store, and what hides it is the other workgroups of the compute unit.
// Bound by HBM: 16384 x 4096 bf16 with an element gate moves 671 MB in 128 us (5.2 TB/s;
// workgroups that went through rows with the weights in registers took 232).
template <typename T, int G, int NV, int GATE, bool TINY>
__global__ void __launch_bounds__(Shape<G>::block) norm_kernel(const NormArgs a) {
    typedef Row<T, G, NV, TINY> R;
    constexpr int N = Vec<T>::N;
    __shared__ float lds[2][2][16];
    const int len = a.hidden;
    const float inv = 1.0f / (float)len;
    int turn = 0;
    // G >= 256: one row a workgroup, so that every wave takes the same turns of this loop (of
    // which there is one, but for more rows than a grid holds)
    for (int64_t t = (int64_t)blockIdx.x * Shape<G>::rows + threadIdx.x / G; t < a.tokens;
         t += (int64_t)gridDim.x * Shape<G>::rows, turn ^= 1) {
        u32x4 x[NV], u[NV], g[NV];
        const bool some = a.branch != nullptr;
        R::load(u, some ? a.branch : a.x, some ? a.branch_ld : a.x_ld, t, len);
        R::load(x, a.x, a.x_ld, t, len);
        if constexpr (GATE == RR_GATE_ELEMENT) R::load(g, a.gate, a.gate_ld, t, len);
        R::mend(u, len);
        if (!some) R::zero(u);
        float r = 1.0f;
        if (a.post) {
            float s[1] = {0.0f};
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < N; ++i) s[0] = fmaf(R::value(u, v, i), R::value(u, v, i), s[0]);
            row_sums<G>(s, lds[turn][0]);
            r = rsqrtf(fmaf(s[0], inv, a.eps));
        }
        R::mend(x, len);
        if constexpr (GATE == RR_GATE_ELEMENT) R::mend(g, len);
        float h[NV][N];
        float s[1] = {0.0f};
        Vec<T> out[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float wp[N], wg[N];
            R::weights(wp, a.post_weight, a.wide_weights, v, len);
            if constexpr (GATE == RR_GATE_CHANNEL) {
                R::weights(wg, a.gate, a.wide_weights, v, len);
            } else if constexpr (GATE == RR_GATE_ELEMENT) {
#pragma unroll
                for (int i = 0; i < N; ++i) wg[i] = R::value(g, v, i);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                h[v][i] = a.residual_scale * R::value(x, v, i);
                if (some) {
                    float n = R::value(u, v, i) * r * wp[i];
                    if constexpr (GATE != RR_GATE_NONE) n *= gate_value(a.gate_act, wg[i]);
                    h[v][i] = fmaf(a.branch_scale, n, h[v][i]);
                }
                s[0] = fmaf(h[v][i], h[v][i], s[0]);
                out[v].e[i] = (T)h[v][i];
            }
        }
        if (a.h) R::store(out, a.h, a.h_ld, t, len);
        if (!a.pre) continue;
        row_sums<G>(s, lds[turn][1]);
        const float q = rsqrtf(fmaf(s[0], inv, a.eps));
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float wn[N];
            R::weights(wn, a.pre_weight, a.wide_weights, v, len);
#pragma unroll
            for (int i = 0; i < N; ++i) out[v].e[i] = (T)(h[v][i] * q * wn[i]);
        }
        R::store(out, a.y, a.y_ld, t, len);
    }
}

// The gradients.  With q = (mean(h^2) + eps)^-1/2 and p = dy * pre_weight,
//   d  = dh + q (p - h q (q mean(p h)))             gradient at the stream
//   dx = residual_scale d
// and with r the same of the branch u, n = u r post_weight, e = branch_scale d:
//   dgate = e n act'(gate);   m = e act(gate) post_weight
//   du = r (m - u r (r mean(m u)))
//   dpre_weight = sum_t dy h q;  dpost_weight = sum_t e act(gate) u r.
// d and du in this order: the cubes of q and r leave 32 bits for rows near 1e15, or near 1e-13
// with eps 0, where everything else is still far from it.
// A channel gate is the same for all tokens: with S = sum_t e u r, dpost_weight is act(gate) S
// and the gate's gradient post_weight act'(gate) S.
// Two rounds of sums over a row: (h^2, p h, u^2), then (m u).  The statistics are
// computed again from the rows, which are read anyway, instead of being stored by
// the forward call.  The sums over tokens stay in registers over all rows that a
// workgroup takes (of the longest rows in LDS, where they fit), and the workgroups' parts
// are added by a second, short kernel in a fixed order.  Registers decide the rate: the
// loads of the next row on their way beside this one took 295 us for 16384 x 4096 bf16
// with an element gate, with spills, against 226 to 236 (1074 MB: 4.6 to 4.8 TB/s) without.
template <typename T, int G, int NV, int GATE, bool TINY>
__global__ void __launch_bounds__(Shape<G>::block, G <= 64 ? (NV == 1 ? 3 : 2) : 4)
norm_backward_kernel(const NormArgs a) {
    typedef Row<T, G, NV, TINY> R;
    constexpr int N = Vec<T>::N;
    constexpr bool IN_LDS = G == 1024 && NV * N <= 16 && NV > 1;
    __shared__ float lds[2][4][16];
    __shared__ float held[IN_LDS ? 2 * NV * N : 1][IN_LDS ? G : 1];
    const int len = a.hidden;
    float sum_pre[NV][N], sum_post[NV][N];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            sum_pre[v][i] = sum_post[v][i] = 0.0f;
            if constexpr (IN_LDS) held[v * N + i][threadIdx.x] = held[(NV + v) * N + i][threadIdx.x] = 0.0f;
        }
    const float inv = 1.0f / (float)len;
    struct Input {
        u32x4 dh[NV], dy[NV], h[NV], u[NV], g[NV];
    };
    // What is absent is read from what is there, and taken as zero.
    const auto fetch = [&](Input& in, int64_t t) {
        R::load(in.h, a.pre ? a.h : a.any, a.pre ? a.h_ld : a.any_ld, t, len);
        R::load(in.dy, a.pre ? a.dy : a.any, a.pre ? a.dy_ld : a.any_ld, t, len);
        R::load(in.u, a.branch ? a.branch : a.any, a.branch ? a.branch_ld : a.any_ld, t, len);
        R::load(in.dh, a.dh ? a.dh : a.any, a.dh ? a.dh_ld : a.any_ld, t, len);
        if constexpr (GATE == RR_GATE_ELEMENT) R::load(in.g, a.gate, a.gate_ld, t, len);
    };
    int turn = 0;
    const int64_t stride = (int64_t)gridDim.x * Shape<G>::rows;
    int64_t t = (int64_t)blockIdx.x * Shape<G>::rows + threadIdx.x / G;
    for (; t < a.tokens; t += stride, turn ^= 1) {
        Input in;
        fetch(in, t);
        R::mend(in.h, len);
        R::mend(in.dy, len);
        R::mend(in.u, len);
        R::mend(in.dh, len);
        if constexpr (GATE == RR_GATE_ELEMENT) R::mend(in.g, len);
        if (!a.pre) R::zero(in.h), R::zero(in.dy);
        if (!a.branch) R::zero(in.u);
        if (!a.dh) R::zero(in.dh);
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float wn[N];
            R::weights(wn, a.pre_weight, a.wide_weights, v, len);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float hv = R::value(in.h, v, i), uv = R::value(in.u, v, i);
                s[0] = fmaf(hv, hv, s[0]);
                s[1] = fmaf(R::value(in.dy, v, i) * wn[i], hv, s[1]);
                s[2] = fmaf(uv, uv, s[2]);
            }
        }
        if (a.pre || a.post) row_sums<G>(s, lds[turn][0]);
        const float q = rsqrtf(fmaf(s[0], inv, a.eps));
        const float back = q * (q * s[1] * inv);
        const float r = a.post ? rsqrtf(fmaf(s[2], inv, a.eps)) : 1.0f;
        float m[NV][N];
        float s2[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float wn[N], wp[N], z[N];
            Vec<T> dx, dg;
            R::weights(wn, a.pre_weight, a.wide_weights, v, len);
            R::weights(wp, a.post_weight, a.wide_weights, v, len);
            if constexpr (GATE == RR_GATE_CHANNEL) {
                R::weights(z, a.gate, a.wide_weights, v, len);
            } else if constexpr (GATE == RR_GATE_ELEMENT) {
#pragma unroll
                for (int i = 0; i < N; ++i) z[i] = R::value(in.g, v, i);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float d = R::value(in.dh, v, i);
                if (a.pre) {
                    const float hv = R::value(in.h, v, i), dyv = R::value(in.dy, v, i);
                    d = fmaf(q, fmaf(-back, hv, wn[i] * dyv), d);
                    if constexpr (IN_LDS) held[v * N + i][threadIdx.x] = fmaf(dyv * q, hv, held[v * N + i][threadIdx.x]);
                    else sum_pre[v][i] = fmaf(dyv * q, hv, sum_pre[v][i]);
                }
                dx.e[i] = (T)(a.residual_scale * d);
                float e = a.branch_scale * d;
                const float unit = R::value(in.u, v, i) * r;
                if constexpr (GATE == RR_GATE_ELEMENT) {
                    dg.e[i] = (T)(e * unit * wp[i] * gate_slope(a.gate_act, z[i]));
                    e *= gate_value(a.gate_act, z[i]);
                }
                if constexpr (IN_LDS) held[(NV + v) * N + i][threadIdx.x] = fmaf(e, unit, held[(NV + v) * N + i][threadIdx.x]);
                else sum_post[v][i] = fmaf(e, unit, sum_post[v][i]);
                if constexpr (GATE == RR_GATE_CHANNEL) e *= gate_value(a.gate_act, z[i]);
                m[v][i] = e * wp[i];
                s2[0] = fmaf(m[v][i], R::value(in.u, v, i), s2[0]);
            }
            if (a.dx) R::store(dx, v, a.dx, a.dx_ld, t, len);
            if constexpr (GATE == RR_GATE_ELEMENT)
                if (a.dgate) R::store(dg, v, a.dgate, a.dgate_ld, t, len);
        }
        if (a.dbranch) {
            float bu = 0.0f;
            if (a.post) {
                row_sums<G>(s2, lds[turn][3]);
                bu = r * (r * s2[0] * inv);
            }
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                Vec<T> du;
#pragma unroll
                for (int i = 0; i < N; ++i) du.e[i] = (T)(a.post ? r * fmaf(-bu, R::value(in.u, v, i), m[v][i]) : m[v][i]);
                R::store(du, v, a.dbranch, a.dbranch_ld, t, len);
            }
        }
    }
    if (a.sums == 0) return;
    // one workgroup writes the gradients themselves
    const auto write = [&](const float (&sum)[NV][N], int at, float* whole) {
        if (at < 0) return;
        float* const to = gridDim.x == 1 ? whole : a.part + ((uint64_t)blockIdx.x * a.sums + at) * len;
        if constexpr (G > 64) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (R::column(v) + i < len) to[R::column(v) + i] = sum[v][i];
        } else {                       // the workgroup's rows, added in their order
            __shared__ float joined[Shape<G>::rows][NV * N * G];
            const int g = threadIdx.x % G, row = threadIdx.x / G;
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int i = 0; i < N; ++i) joined[row][(v * N + i) * G + g] = sum[v][i];
            __syncthreads();
            for (int k = threadIdx.x; k < NV * N * G; k += Shape<G>::block) {
                float all = 0.0f;
                for (int w = 0; w < Shape<G>::rows; ++w) all += joined[w][k];
                const int c = (k / (N * G) * G + k % G) * N + k / G % N;
                if (c < len) to[c] = all;
            }
            __syncthreads();
        }
    };
    if constexpr (IN_LDS)
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                sum_pre[v][i] = held[v * N + i][threadIdx.x];
                sum_post[v][i] = held[(NV + v) * N + i][threadIdx.x];
            }
    write(sum_pre, a.at_pre, a.dpre);
    if constexpr (GATE == RR_GATE_CHANNEL) {
        float sum_gate[NV][N];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float wp[N], z[N];
            R::weights(wp, a.post_weight, a.wide_weights, v, len);
            R::weights(z, a.gate, a.wide_weights, v, len);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                sum_gate[v][i] = sum_post[v][i] * wp[i] * gate_slope(a.gate_act, z[i]);
                sum_post[v][i] *= gate_value(a.gate_act, z[i]);
            }
        }
        write(sum_gate, a.at_gate, a.dgate_channel);
    }
    write(sum_post, a.at_post, a.dpost);
}

struct Config {
    int group, vecs;
    bool tiny;
};

void launch_norm_f32(const NormArgs& a, const Config& c, unsigned grid, bool back, hipStream_t s);
void launch_norm_bf16(const NormArgs& a, const Config& c, unsigned grid, bool back, hipStream_t s);
void launch_norm_f16(const NormArgs& a, const Config& c, unsigned grid, bool back, hipStream_t s);

template <typename T, int G, int NV, bool TINY, bool BACK>
static void launch_rows(const NormArgs& a, unsigned grid, hipStream_t s) {
    constexpr int B = Shape<G>::block;
    const auto go = [&](auto kernel) { kernel<<<grid, B, 0, s>>>(a); };
    if constexpr (BACK) {
        if (a.gate_kind == RR_GATE_NONE) go(norm_backward_kernel<T, G, NV, RR_GATE_NONE, TINY>);
        else if (a.gate_kind == RR_GATE_CHANNEL) go(norm_backward_kernel<T, G, NV, RR_GATE_CHANNEL, TINY>);
        else go(norm_backward_kernel<T, G, NV, RR_GATE_ELEMENT, TINY>);
    } else {
        if (a.gate_kind == RR_GATE_NONE) go(norm_kernel<T, G, NV, RR_GATE_NONE, TINY>);
        else if (a.gate_kind == RR_GATE_CHANNEL) go(norm_kernel<T, G, NV, RR_GATE_CHANNEL, TINY>);
        else go(norm_kernel<T, G, NV, RR_GATE_ELEMENT, TINY>);
    }
}
template <typename T>
static void launch_rows(const NormArgs& a, const Config& c, unsigned grid, bool back, hipStream_t s) {
#define BLK_ROWS(G, NV, TINY, BACK)                                        \
    if (c.group == G && c.vecs == NV && c.tiny == TINY && back == BACK)    \
        return launch_rows<T, G, NV, TINY, BACK>(a, grid, s)
    BLK_ROWS(8, 1, true, false);
    BLK_ROWS(8, 1, false, false);
    BLK_ROWS(16, 1, false, false);
    BLK_ROWS(32, 1, false, false);
    BLK_ROWS(64, 1, false, false);
    BLK_ROWS(64, 2, false, false);
    BLK_ROWS(256, 1, false, false);
    BLK_ROWS(256, 2, false, false);
    BLK_ROWS(512, 2, false, false);
    BLK_ROWS(1024, 2, false, false);
    BLK_ROWS(1024, 4, false, false);
    BLK_ROWS(8, 1, true, true);
    BLK_ROWS(8, 1, false, true);
    BLK_ROWS(16, 1, false, true);
    BLK_ROWS(32, 1, false, true);
    BLK_ROWS(64, 1, false, true);
    BLK_ROWS(64, 2, false, true);
    BLK_ROWS(256, 1, false, true);
    BLK_ROWS(512, 1, false, true);
    BLK_ROWS(1024, 1, false, true);
    BLK_ROWS(1024, 2, false, true);
    BLK_ROWS(1024, 4, false, true);
    if constexpr (sizeof(T) == 4) {
        BLK_ROWS(1024, 8, false, false);
        BLK_ROWS(1024, 8, false, true);
    }
#undef BLK_ROWS
}

}  // namespace blk
