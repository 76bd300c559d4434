// blk_norm.hip -- the norm after a block with its gate, the scaled residual and the
// norm before the next block, in one pass over the rows, and its gradients
// (block_norm, block_norm_backward): the entry points.  The kernels: blk_norm.hpp.
#include "blk_norm.hpp"

namespace blk {

// Adds the parts of one gradient: 16 columns a workgroup, 16 threads each.
__global__ void __launch_bounds__(256)
norm_parts_kernel(const float* part, int parts, uint64_t stride, int hidden, float* o0, float* o1,
                  float* o2) {
    __shared__ float lds[16][17];
    const int col = blockIdx.x * 16 + (threadIdx.x & 15), s = threadIdx.x >> 4;
    float* out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : o2;
    float sum = 0.0f;
    if (col < hidden)
#pragma unroll 4
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

// Threads and vectors per row.  A row of few vectors goes to a part of a wave or one wave (no barrier); a longer
// one to as many threads as keep it in registers.  The backward kernel holds five rows and the
// sums over tokens, so it takes twice the threads (16384 x 4096 bf16 with an element gate: 358
// us with 256 threads of two vectors, 226 to 233 with 512 of one).  1024 threads leave each 128
// registers, which the longest rows do not fit: the build spills
//   bf16, fp16   backward beyond 8192 elements 26 to 36 registers, beyond 16384 238 to 400;
//                forward beyond 16384 30 to 60
//   fp32         backward beyond 8192 elements 38 to 122, beyond 16384 516 to 821; forward
//                beyond 8192 with a gate 6 to 10, beyond 16384 154 to 378
// at 128 MiB a matrix, without a gate and with one for each element (TB/s, forward; backward):
//   bf16 16384  4.8, 4.6; 3.0, 3.2     32768  3.3, 3.4; 1.0, 0.8
//   fp32 16384  4.8, 4.3; 2.9, 2.3     32768  1.8, 0.9; 1.0, 0.9
static Config pick(int hidden, int dt, bool back) {
    const int n = (int)(16 / type_bytes(dt));
    const int vecs = (int)ceil_div(hidden, n);
    if (hidden < n) return {8, 1, true};
    if (vecs <= 8) return {8, 1, false};
    if (vecs <= 16) return {16, 1, false};
    if (vecs <= 32) return {32, 1, false};
    if (vecs <= 64) return {64, 1, false};
    if (vecs <= 128) return {64, 2, false};
    if (vecs <= 256) return {256, 1, false};
    if (vecs <= 512) return back ? Config{512, 1, false} : Config{256, 2, false};
    if (vecs <= 1024) return back ? Config{1024, 1, false} : Config{512, 2, false};
    if (vecs <= 2048) return {1024, 2, false};
    if (vecs <= 4096) return {1024, 4, false};
    return {1024, 8, false};   // fp32 rows beyond 16384
}
static int rows_of(const Config& c) { return c.group < 256 ? 256 / c.group : 1; }

// Workgroups of the backward call: what fits every compute unit at once, so that each
// keeps its sums over tokens in registers over many rows.
static unsigned grid_of(const Config& c, size_t tokens) {
    const int cus = compute_units();
    const uint64_t want = ceil_div(tokens, rows_of(c));
    if (want <= 2) return 1;       // a second row costs less than the launch that adds two parts
    const uint64_t most = (uint64_t)(cus > 0 ? cus : 256) * (c.group <= 64 ? (c.vecs == 1 ? 3 : 2) : c.group == 256 ? 4 : c.group == 512 ? 2 : 1);
    return (unsigned)(want < most ? want : most);
}

static rr_status_t launch_norm(const NormArgs& a, int dt, const Config& c, unsigned grid, bool back,
                               hipStream_t s) {
    if (dt == RR_FP32) launch_norm_f32(a, c, grid, back, s);
    else if (dt == RR_BF16) launch_norm_bf16(a, c, grid, back, s);
    else launch_norm_f16(a, c, grid, back, s);
    return launched();
}

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

// Parts of the sums over tokens: one for each workgroup.
static uint64_t parts_of(const rr_norm_t* a) {
    return grid_of(pick((int)a->hidden, a->dt, true), a->tokens);
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
    const Config c = pick((int)h, a->dt, false);
    const uint64_t blocks = ceil_div(t, rows_of(c));
    return launch_norm(k, a->dt, c, (unsigned)(blocks < 1u << 20 ? blocks : 1u << 20), false, (hipStream_t)stream);
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
    k.dpre = g->dpre_weight;
    k.dpost = g->dpost_weight;
    k.dgate_channel = g->dgate_channel;
    k.at_pre = k.at_post = k.at_gate = -1;
    float* sums[3] = {nullptr, nullptr, nullptr};
    if (g->dpre_weight) sums[k.at_pre = k.sums++] = g->dpre_weight;
    if (g->dpost_weight) sums[k.at_post = k.sums++] = g->dpost_weight;
    if (g->dgate_channel) sums[k.at_gate = k.sums++] = g->dgate_channel;
    for (const rr_rows_t& r : {g->dx, a->branch, g->dh, g->dy})
        if (r.data) {
            k.any = r.data;
            k.any_ld = r.ld;
        }
    if (t && !k.any) return RR_OK;      // no gradient comes in, and none is asked for
    const Config c = pick((int)h, a->dt, true);
    const unsigned grid = grid_of(c, t);
    hipStream_t s = (hipStream_t)stream;
    if (t && (st = launch_norm(k, a->dt, c, grid, true, s)) != RR_OK) return st;
    if (k.sums && (grid > 1 || t == 0)) {
        const dim3 parts((unsigned)ceil_div(h, 16), (unsigned)k.sums);
        norm_parts_kernel<<<parts, 256, 0, s>>>(k.part, t ? (int)parts_of(a) : 0, (uint64_t)k.sums * h,
                                                (int)h, sums[0], sums[1], sums[2]);
        if ((st = launched()) != RR_OK) return st;
    }
    return RR_OK;
}

}  // extern "C"
