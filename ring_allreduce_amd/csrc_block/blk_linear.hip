// blk_linear.hip -- the entry points of a block's matrix products (block_linear,
// block_linear_backward): the choice of kernel for each product, the gradient of the
// activation, and the checks.  The products themselves: blk_gemm.hpp.
#include "blk_gemm.hpp"

namespace blk {

// ------------------------------------------------------- activation's gradient --
//
// dz = dout act'(z), rounded to the rows' type as the next products' operand, and the
// column sums of each group in 32 bits.  A workgroup takes 8 columns a thread and one
// of `splits` parts of a group's rows; the parts are added in a fixed order.
struct SlopeArgs {
    GemmArgs g;            // rows, groups, offsets
    const void *dout, *z;
    void* dz;              // or null: nothing but the sums
    uint64_t dout_ld, z_ld, dz_ld;
    float* part;           // [groups][splits][n], or null
    int32_t n, act, splits;
};

template <typename T>
__global__ void __launch_bounds__(256) slope_kernel(const SlopeArgs a) {
    const int col = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 8;
    const Range g = range_of(a.g, (int)blockIdx.z + 1);
    if (col >= a.n) return;
    const int per = (g.hi - g.lo + a.splits - 1) / a.splits;
    const int lo = g.lo + min((int)blockIdx.y * per, g.hi - g.lo), hi = min(lo + per, g.hi);
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
    for (int r = lo; r < hi; ++r) {
        const Vec<T> d = load_vec((const T*)a.dout + (uint64_t)r * a.dout_ld, col, a.n);
        Vec<T> o;
        float v[8];
        if (a.act != RR_ACT_NONE) {
            const Vec<T> z = load_vec((const T*)a.z + (uint64_t)r * a.z_ld, col, a.n);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)z.e[e];
            act_slopes(a.act, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] *= (float)d.e[e];
                sum[e] += v[e];
                o.e[e] = (T)v[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += (float)d.e[e];
        }
        if (a.dz) store_vec((T*)a.dz + (uint64_t)r * a.dz_ld, col, a.n, o);
    }
    if (!a.part) return;
    float* to = a.part + ((uint64_t)blockIdx.z * a.splits + blockIdx.y) * a.n;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (col + e < a.n) to[col + e] = sum[e];
}

__global__ void __launch_bounds__(256)
slope_parts_kernel(const float* part, int splits, int n, float* db) {
    const int col = (int)blockIdx.x * 256 + (int)threadIdx.x;
    if (col >= n) return;
    const float* from = part + (uint64_t)blockIdx.y * splits * n + col;
    float sum = 0.0f;
    for (int s = 0; s < splits; ++s) sum += from[(uint64_t)s * n];
    db[(uint64_t)blockIdx.y * n + col] = sum;
}

// ------------------------------------------------------------------ host side --

constexpr uint64_t kMaxSize = 0x7FFFFFFFull - 1024;
constexpr uint64_t kMaxLd = 1ull << 22;

static bool rows_ok(const rr_rows_t& r, uint64_t rows, uint64_t width, uint64_t bytes) {
    return rows == 0 || (r.data && aligned_to(r.data, bytes) && r.ld >= width);
}
static bool rows_ok_if(const rr_rows_t& r, uint64_t rows, uint64_t width, uint64_t bytes) {
    return !r.data || rows_ok(r, rows, width, bytes);
}

static rr_status_t check_linear(const rr_linear_t* a) {
    if (!a || a->reserved) return RR_ERR_INVALID;
    if (a->dt != RR_BF16 && a->dt != RR_FP16)
        return a->dt == RR_FP32 ? RR_ERR_UNSUPPORTED : RR_ERR_INVALID;
    if (a->n < 1 || a->k < 1 || a->groups < 1) return RR_ERR_INVALID;
    if (a->act < RR_ACT_NONE || a->act > RR_ACT_SILU) return RR_ERR_INVALID;
    if (a->rows > kMaxSize || a->n > kMaxSize || a->k > kMaxSize || a->groups > RR_MAX_EXPERTS)
        return RR_ERR_UNSUPPORTED;
    if (!a->offsets && a->rows % (uint64_t)a->groups) return RR_ERR_INVALID;
    if (!aligned_to(a->offsets, 4)) return RR_ERR_INVALID;
    if (!a->w || !aligned_to(a->w, 2) || a->w_ld < a->k) return RR_ERR_INVALID;
    if (a->groups > 1 && a->w_stride < extent(a->n, a->w_ld, a->k, 1)) return RR_ERR_INVALID;
    if (!rows_ok(a->x, a->rows, a->k, 2) || !rows_ok_if(a->z, a->rows, a->n, 2))
        return RR_ERR_INVALID;
    if (a->x.ld > kMaxLd || a->w_ld > kMaxLd) return RR_ERR_UNSUPPORTED;
    if (a->groups > 1 && a->w_stride > (1ull << 44)) return RR_ERR_UNSUPPORTED;
    return RR_OK;
}

static rr_status_t check_grad(const rr_linear_t* a, const rr_linear_grad_t* g) {
    const rr_status_t st = check_linear(a);
    if (st != RR_OK) return st;
    if (!g || g->reserved) return RR_ERR_INVALID;
    if (g->dw_dt != a->dt && g->dw_dt != RR_FP32) return RR_ERR_INVALID;
    if (!rows_ok(g->dout, a->rows, a->n, 2) || !rows_ok_if(g->dx, a->rows, a->k, 2))
        return RR_ERR_INVALID;
    if (a->act != RR_ACT_NONE && !rows_ok(a->z, a->rows, a->n, 2)) return RR_ERR_INVALID;
    if (!aligned_to(g->dw, type_bytes(g->dw_dt)) || !aligned_to(g->db, 4)) return RR_ERR_INVALID;
    if (g->dout.ld > kMaxLd || (g->dx.data && g->dx.ld > kMaxLd) || (a->act != RR_ACT_NONE && a->n > kMaxLd)) return RR_ERR_UNSUPPORTED;
    return RR_OK;
}

static GemmArgs groups_of(const rr_linear_t* a) {
    GemmArgs k = {};
    k.rows = (int32_t)a->rows;
    k.groups = a->groups;
    k.offsets = a->offsets;
    return k;
}

// Row tiles of all groups: each can add one partly filled, and so can the rows before
// the first and after the last one.
static uint64_t row_tiles(const rr_linear_t* a, uint64_t height) {
    if (a->groups == 1 && !a->offsets) return ceil_div(a->rows, height);
    return a->rows / height + a->groups + 2;
}

static bool good_operand(const void* p, uint64_t ld) { return aligned_to(p, 16) && ld % 8 == 0; }

// The kernel for one product: i x j outputs (i rows in all, or per group for dw), c deep.
static GemmPlan choose(const rr_linear_t* a, int form, bool direct, int* splits) {
    const uint64_t groups = (uint64_t)a->groups, mean = ceil_div(a->rows, groups);
    const uint64_t i = form == kByW ? a->n : a->rows, j = form == kForward ? a->n : a->k;
    const uint64_t c = form == kForward ? a->k : form == kByX ? a->n : mean;
    GemmPlan p = {form, kTile64, direct};
    *splits = 1;
    if (form == kForward && mean <= 64) {
        p.tile = mean <= 16 ? kStream16 : mean <= 32 ? kStream32 : kStream64;
        return p;
    }
    const auto tiles = [&](uint64_t t) {
        const uint64_t rows = form == kByW ? groups * ceil_div(i, t) : i / t + ceil_div(groups, 2) + (i % t != 0 && groups == 1);
        return rows * ceil_div(j, t);
    };
    const uint64_t n64 = tiles(64), n128 = tiles(128), n256 = tiles(256);
    double best = (double)ceil_div(n64, 1024) * 0.25 * 2.2;
    const double by128 = (double)ceil_div(n128, 512) * 0.5 * 1.35, by256 = (double)ceil_div(n256, 256);
    if (by128 <= best) {
        best = by128;
        p.tile = kTile128;
    }
    if (direct && by256 <= best) p.tile = kTile256;
    const uint64_t n = p.tile == kTile64 ? n64 : p.tile == kTile128 ? n128 : n256;
    if (n < 256 && p.tile != kTile256) {
        const uint64_t want = 512 / (n ? n : 1), most = c / (4 * kDepth);
        const uint64_t s = want < most ? want : most;
        *splits = s < 2 ? 1 : s > 64 ? 64 : (int)s;
    }
    return p;
}

// Bytes of a product's parts, whatever the operands' alignment turns out to be.
static uint64_t part_bytes(const rr_linear_t* a, int form) {
    uint64_t most = 0;
    for (int direct = 0; direct < 2; ++direct) {
        int splits;
        choose(a, form, direct != 0, &splits);
        const uint64_t rows = form == kByW ? (uint64_t)a->groups * a->n : a->rows;
        const uint64_t j = form == kForward ? a->n : a->k;
        const uint64_t bytes = splits > 1 ? (uint64_t)splits * rows * j * sizeof(float) : 0;
        if (bytes > most) most = bytes;
    }
    return ceil_div(most, 256) * 256;
}

// `a`: operands, sizes and epilogue are set; the rest follows from the plan.
static rr_status_t run_gemm(GemmArgs k, const rr_linear_t* a, int form, void* workspace, hipStream_t s) {
    bool direct = good_operand(k.p, k.p_ld) && good_operand(k.q, k.q_ld) && k.q_group % 8 == 0;
    // the sizes along which 16 bytes are read
    if (form == kForward) direct = direct && k.c % 8 == 0;
    else if (form == kByX) direct = direct && k.c % 8 == 0 && k.j % 8 == 0;
    else direct = direct && k.i % 8 == 0 && k.j % 8 == 0;
    int splits;
    const GemmPlan p = choose(a, form, direct, &splits);
    const uint64_t ti = form == kByW ? ceil_div(k.i, tile_rows(p.tile)) : row_tiles(a, tile_rows(p.tile));
    const uint64_t tj = ceil_div(k.j, tile_cols(p.tile));
    if (ti * tj == 0) return RR_OK;
    if (ti * tj * splits * (form == kByW ? (uint64_t)a->groups : 1) > (1u << 23) - 1)
        return RR_ERR_UNSUPPORTED;
    k.tiles_i = (int32_t)ti;
    k.tiles_j = (int32_t)tj;
    k.splits = splits;
    k.part = (float*)workspace;
    k.part_stride = (form == kByW ? (uint64_t)k.groups * k.i : (uint64_t)k.rows) * k.j;
    if (splits > 1 && ceil_div((k.part_stride / k.j) * ceil_div(k.j, 4), 256) > (1u << 24) - 1)
        return RR_ERR_UNSUPPORTED;
    return a->dt == RR_BF16 ? launch_gemm_bf16(k, p, s) : launch_gemm_f16(k, p, s);
}

// Parts of a group's rows in the sums over rows: enough workgroups to fill the device.
static uint64_t splits_of(const rr_linear_t* a) {
    const uint64_t cols = ceil_div(a->n, 256 * 8) * a->groups;
    const uint64_t each = ceil_div(a->rows, a->groups);
    const uint64_t want = ceil_div(2048, cols), most = ceil_div(each, 16);
    const uint64_t n = want < most ? want : most;
    return n < 1 ? 1 : n > 1024 ? 1024 : n;
}

struct BackwardPlan {
    uint64_t dz, part, split;  // bytes of scratch
};
static BackwardPlan plan_of(const rr_linear_t* a, const rr_linear_grad_t* g) {
    BackwardPlan p = {0, 0, 0};
    if (a->act != RR_ACT_NONE && (g->dx.data || g->dw))
        p.dz = ceil_div(a->rows * ceil_div(a->n, 8) * 8 * 2, 256) * 256;
    if (g->db) p.part = ceil_div((uint64_t)a->groups * splits_of(a) * a->n * sizeof(float), 256) * 256;
    if (g->dx.data) p.split = part_bytes(a, kByX);
    if (g->dw && part_bytes(a, kByW) > p.split) p.split = part_bytes(a, kByW);
    return p;
}

}  // namespace blk

using namespace blk;

extern "C" {

rr_status_t block_linear_workspace(const rr_linear_t* a, size_t* bytes) {
    if (!bytes) return RR_ERR_INVALID;
    const rr_status_t st = check_linear(a);
    if (st != RR_OK) return st;
    *bytes = part_bytes(a, kForward);
    return RR_OK;
}

rr_status_t block_linear(const rr_linear_t* a, void* workspace, size_t workspace_bytes,
                         rr_stream_t stream) {
    const rr_status_t st = check_linear(a);
    if (st != RR_OK) return st;
    const uint64_t need = part_bytes(a, kForward);
    if (need && (!workspace || !aligned_to(workspace, 16) || workspace_bytes < need))
        return RR_ERR_INVALID;
    if (!rows_ok(a->out, a->rows, a->n, 2) || !rows_ok_if(a->residual, a->rows, a->n, 2) ||
        !aligned_to(a->bias, 2))
        return RR_ERR_INVALID;
    if (a->out.ld > kMaxLd || (a->residual.data && a->residual.ld > kMaxLd) || (a->z.data && a->z.ld > kMaxLd))
        return RR_ERR_UNSUPPORTED;
    const uint64_t wide = extent(a->groups, a->w_stride, extent(a->n, a->w_ld, a->k, 1), 2);
    const uint64_t n_out = extent(a->rows, a->out.ld, a->n, 2), n_z = extent(a->rows, a->z.ld, a->n, 2);
    const uint64_t n_res = extent(a->rows, a->residual.ld, a->n, 2);
    const struct { const void* p; uint64_t n; } in[] = {
        {a->x.data, extent(a->rows, a->x.ld, a->k, 2)}, {a->w, wide},
        {a->bias, (uint64_t)a->groups * a->n * 2},
        {a->offsets, (uint64_t)(a->groups + 1) * 4}};
    for (const auto& i : in)
        if (overlap(i.p, i.n, a->out.data, n_out) || overlap(i.p, i.n, a->z.data, n_z) ||
            overlap(i.p, i.n, workspace, need))
            return RR_ERR_INVALID;
    if (overlap(a->out.data, n_out, workspace, need) || overlap(a->z.data, n_z, workspace, need) ||
        overlap(a->residual.data, n_res, workspace, need))
        return RR_ERR_INVALID;
    if (overlap(a->out.data, n_out, a->z.data, n_z) ||
        overlap(a->residual.data, n_res, a->z.data, n_z))
        return RR_ERR_INVALID;
    if (overlap(a->residual.data, n_res, a->out.data, n_out) &&
        !(a->residual.data == a->out.data && a->residual.ld == a->out.ld))
        return RR_ERR_INVALID;
    if (a->rows == 0) return RR_OK;
    GemmArgs k = groups_of(a);
    k.p = a->x.data;
    k.p_ld = a->x.ld;
    k.q = a->w;
    k.q_ld = a->w_ld;
    k.q_group = a->w_stride;
    k.i = (int32_t)a->rows;
    k.j = (int32_t)a->n;
    k.c = (int32_t)a->k;
    k.bias = a->bias;
    k.residual = a->residual.data;
    k.residual_ld = a->residual.ld;
    k.z = a->z.data;
    k.z_ld = a->z.ld;
    k.out = a->out.data;
    k.out_ld = a->out.ld;
    k.act = a->act;
    return run_gemm(k, a, kForward, workspace, (hipStream_t)stream);
}

rr_status_t block_linear_backward_workspace(const rr_linear_t* a, const rr_linear_grad_t* g,
                                            size_t* bytes) {
    if (!bytes) return RR_ERR_INVALID;
    const rr_status_t st = check_grad(a, g);
    if (st != RR_OK) return st;
    const BackwardPlan p = plan_of(a, g);
    *bytes = p.dz + p.part + p.split;
    return RR_OK;
}

rr_status_t block_linear_backward(const rr_linear_t* a, const rr_linear_grad_t* g,
                                  void* workspace, size_t workspace_bytes, rr_stream_t stream) {
    rr_status_t st = check_grad(a, g);
    if (st != RR_OK) return st;
    const BackwardPlan plan = plan_of(a, g);
    const uint64_t need = plan.dz + plan.part + plan.split;
    if (need && (!workspace || !aligned_to(workspace, 16) || workspace_bytes < need))
        return RR_ERR_INVALID;
    const uint64_t w_bytes = extent(a->groups, a->w_stride, extent(a->n, a->w_ld, a->k, 1), 2);
    const struct { const void* p; uint64_t n; } in[] = {
        {g->dout.data, extent(a->rows, g->dout.ld, a->n, 2)},
        {a->x.data, extent(a->rows, a->x.ld, a->k, 2)}, {a->w, w_bytes},
        {a->act != RR_ACT_NONE ? a->z.data : nullptr, extent(a->rows, a->z.ld, a->n, 2)},
        {a->offsets, (uint64_t)(a->groups + 1) * 4}},
    out[] = {
        {g->dx.data, extent(a->rows, g->dx.ld, a->k, 2)},
        {g->dw, (uint64_t)a->groups * a->n * a->k * type_bytes(g->dw_dt)},
        {g->db, (uint64_t)a->groups * a->n * 4}, {workspace, need}};
    for (int o = 0; o < 4; ++o) {
        for (const auto& i : in)
            if (overlap(out[o].p, out[o].n, i.p, i.n)) return RR_ERR_INVALID;
        for (int q = o + 1; q < 4; ++q)
            if (overlap(out[o].p, out[o].n, out[q].p, out[q].n)) return RR_ERR_INVALID;
    }
    hipStream_t s = (hipStream_t)stream;
    rr_rows_t dz = g->dout;
    void* const split = (char*)workspace + plan.dz + plan.part;
    if (plan.dz || plan.part) {
        SlopeArgs k = {};
        k.g = groups_of(a);
        k.dout = g->dout.data;
        k.dout_ld = g->dout.ld;
        k.z = a->z.data;
        k.z_ld = a->z.ld;
        k.n = (int32_t)a->n;
        k.act = a->act;
        k.splits = (int32_t)splits_of(a);
        if (plan.dz) {
            dz = {workspace, ceil_div(a->n, 8) * 8};
            k.dz = dz.data;
            k.dz_ld = dz.ld;
        }
        if (plan.part) k.part = (float*)((char*)workspace + plan.dz);
        const uint64_t cols = ceil_div(a->n, 256 * 8);
        if (cols > (1u << 24) - 1) return RR_ERR_UNSUPPORTED;
        const dim3 grid((unsigned)cols, (unsigned)k.splits, (unsigned)a->groups);
        if (a->dt == RR_BF16)
            slope_kernel<bf16><<<grid, 256, 0, s>>>(k);
        else
            slope_kernel<f16><<<grid, 256, 0, s>>>(k);
        if ((st = launched()) != RR_OK) return st;
        if (g->db) {
            const dim3 sums((unsigned)ceil_div(a->n, 256), (unsigned)a->groups);
            slope_parts_kernel<<<sums, 256, 0, s>>>(k.part, k.splits, k.n, g->db);
            if ((st = launched()) != RR_OK) return st;
        }
    }
    if (g->dx.data && a->rows) {
        GemmArgs k = groups_of(a);
        k.p = dz.data;
        k.p_ld = dz.ld;
        k.q = a->w;
        k.q_ld = a->w_ld;
        k.q_group = a->w_stride;
        k.i = (int32_t)a->rows;
        k.j = (int32_t)a->k;
        k.c = (int32_t)a->n;
        k.out = g->dx.data;
        k.out_ld = g->dx.ld;
        if ((st = run_gemm(k, a, kByX, split, s)) != RR_OK) return st;
    }
    if (g->dw) {
        GemmArgs k = groups_of(a);
        k.p = dz.data;
        k.p_ld = dz.ld;
        k.q = a->x.data;
        k.q_ld = a->x.ld;
        k.i = (int32_t)a->n;
        k.j = (int32_t)a->k;
        k.out = g->dw;
        k.out_ld = a->k;
        k.out_group = (uint64_t)a->n * a->k;
        k.wide_out = g->dw_dt == RR_FP32;
        if ((st = run_gemm(k, a, kByW, split, s)) != RR_OK) return st;
    }
    return RR_OK;
}

}  // extern "C"
