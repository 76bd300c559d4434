// blk_linear.hip -- a block's matrix products with bias, activation and residual in
// the epilogue, dense or over the sorted rows of experts, and their gradients
// (block_linear, block_linear_backward).
//
// Three products, all out[i][j] = sum over c of P(i, c) Q(j, c):
//   forward  i = row, j = n, c = k:    P = x,  Q = w_e         both contiguous along c
//   dx       i = row, j = k, c = n:    P = dz, Q = w_e         Q contiguous along j
//   dw       i = n,   j = k, c = row:  P = dz, Q = x           both contiguous along i, j
#include "blk_common.hpp"

namespace blk {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
#define BLK_LDS __attribute__((address_space(3)))

struct GemmArgs {
    const void *p, *q;
    uint64_t p_ld, q_ld, q_group;    // q_group: elements from one group's Q to the next
    int32_t rows;                    // rows of all groups (P and out, or the contraction)
    int32_t i, j, c;                 // sizes; the grouped one of i and c is not read
    int32_t groups;
    const int32_t* offsets;          // or null: rows / groups rows each
    // epilogue
    const void *bias, *residual;
    void *z, *out;
    uint64_t residual_ld, z_ld, out_ld, out_group;
    int32_t act;
    int32_t wide_out;                // out in fp32
    int32_t tiles_i, tiles_j;        // tiles_i: an upper bound over all groups
};

// ------------------------------------------------------------------- groups --

struct Range {
    int32_t group;   // -1: rows of no group
    int32_t lo, hi;
};

// Range r of rows: 0 is what lies before the first group, groups + 1 what lies after
// the last one.  Whatever the offsets hold, 0 <= lo <= hi <= rows.
__device__ __forceinline__ Range range_of(const GemmArgs& a, int r) {
    Range g = {-1, 0, 0};
    if (r > a.groups + 1) return g;
    if (!a.offsets) {
        if (r < 1 || r > a.groups) return g;
        const int32_t each = a.rows / a.groups;
        return {r - 1, (r - 1) * each, r * each};
    }
    const auto edge = [&](int k) { return min(max(a.offsets[k], 0), a.rows); };
    g.lo = r == 0 ? 0 : edge(r - 1);
    g.hi = r > a.groups ? a.rows : edge(r);
    if (g.hi < g.lo) g.hi = g.lo;
    if (r >= 1 && r <= a.groups) g.group = r - 1;
    return g;
}

// The range and the first row of row tile `tile` (tiles of `height` rows, counted
// through the ranges one after another).  Called by whole waves; false past the end.
__device__ __forceinline__ bool find_tile(const GemmArgs& a, int tile, int height, Range& g) {
    if (a.groups == 1 && !a.offsets) {
        g = {0, tile * height, a.rows};
        return g.lo < a.rows;
    }
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int r0 = 0; r0 < a.groups + 2; r0 += 64) {
        const Range r = range_of(a, r0 + lane);
        const int n = (r.hi - r.lo + height - 1) / height;
        int sum = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(sum, d);
            if (lane >= d) sum += up;
        }
        const uint64_t past = __ballot(tile < before + sum);
        if (past) {
            const int at = __ffsll((unsigned long long)past) - 1;
            g.group = __shfl(r.group, at);
            g.lo = __shfl(r.lo, at) + (tile - before - (__shfl(sum, at) - __shfl(n, at))) * height;
            g.hi = __shfl(r.hi, at);
            return true;
        }
        before += __shfl(sum, 63);
    }
    return false;
}

// ----------------------------------------------------------------- the tiles --
//
// A tile of an operand in LDS is 64 deep along c, in one of two layouts:
//   contiguous along c:  [row][64], the eight 16-byte pieces of a row permuted by the
//     row number, so that the 16 rows a fragment read touches lie in different banks;
//   contiguous along the rows:  [64][rows], the 32-byte pieces (16 rows) of a line
//     permuted by the line number, for the transposing read, in which 16 lanes
//     read four lines of 16 rows and each gets four values of one row.
constexpr int kDepth = 64;

__device__ __forceinline__ int line_mix(int c) { return (c & 3) | ((c >> 1) & 4); }

template <bool ACROSS, int ROWS> struct Tile {
    // byte address of the 16-byte piece that holds elements (row, c .. c + 7), or
    // ACROSS: (row .. row + 7, c)
    __device__ static int piece(int row, int c) {
        if constexpr (!ACROSS) return row * (kDepth * 2) + (((c >> 3) ^ (row & 7)) << 4);
        else return c * (ROWS * 2) + (((row >> 4) ^ line_mix(c)) << 5) + ((row & 8) << 1);
    }
    // this lane's part of the fragment of 16 rows from `row`, 32 deep from c: row
    // row + lane % 16, c + (lane / 16) * 8 .. + 7
    template <typename V>
    __device__ static V fragment(const BLK_LDS char* tile, int row, int c) {
        const int lane = threadIdx.x & 63;
        if constexpr (!ACROSS) {
            return __builtin_bit_cast(
                V, *(const BLK_LDS u32x4*)(tile + piece(row + (lane & 15), c + (lane >> 4) * 8)));
        } else {
            s16x4 half[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int line = c + (lane >> 4) * 8 + h * 4 + ((lane & 15) >> 2);
                half[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (BLK_LDS s16x4*)(tile + line * (ROWS * 2) + (((row >> 4) ^ line_mix(line)) << 5) +
                                     (lane & 3) * 8));
            }
            return __builtin_bit_cast(V, half);
        }
    }
};

template <typename T> struct Mma;
template <> struct Mma<bf16> {
    typedef bf16x8 V;
    __device__ static f32x4 run(V a, V b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct Mma<f16> {
    typedef f16x8 V;
    __device__ static f32x4 run(V a, V b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// Loads of one operand's tile through registers: any alignment, any size; what lies
// outside [row, row_end) x [c, c_end) is zero.
template <typename T, bool ACROSS, int ROWS, int THREADS> struct Loader {
    static constexpr int kPieces = ROWS * kDepth / 8 / THREADS;
    u32x4 r[kPieces];
    __device__ void load(const T* base, uint64_t ld, int row, int row_end, int c, int c_end) {
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int id = k * THREADS + (int)threadIdx.x;
            Vec<T> v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v.e[e] = (T)0.0f;
            if constexpr (!ACROSS) {
                const int y = row + id / 8, x = c + id % 8 * 8;
                if (y < row_end && x < c_end) v = load_vec(base + (uint64_t)y * ld, x, c_end);
            } else {
                const int y = c + id / (ROWS / 8), x = row + id % (ROWS / 8) * 8;
                if (y < c_end && x < row_end) v = load_vec(base + (uint64_t)y * ld, x, row_end);
            }
            r[k] = __builtin_bit_cast(u32x4, v);
        }
    }
    __device__ void store(BLK_LDS char* tile) const {
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int id = k * THREADS + (int)threadIdx.x;
            const int at = ACROSS ? Tile<ACROSS, ROWS>::piece(id % (ROWS / 8) * 8, id / (ROWS / 8))
                                  : Tile<ACROSS, ROWS>::piece(id / 8, id % 8 * 8);
            *(BLK_LDS u32x4*)(tile + at) = r[k];
        }
    }
};

// Four neighbouring columns of one output row.
template <typename T>
__device__ __forceinline__ void finish(const GemmArgs& a, const Range& g, bool by_rows, int i, int j,
                                       f32x4 v) {
    if (j >= a.j) return;
    const int n = min(4, a.j - j);
    const bool none = by_rows && g.group < 0;   // a row of no group: zeros
    T* out = (T*)a.out + (by_rows ? 0 : (uint64_t)g.group * a.out_group);
    for (int e = 0; e < n; ++e) {
        float z = v[e];
        if (a.bias && !none) z += (float)((const T*)a.bias)[(uint64_t)g.group * a.j + j + e];
        if (none) z = 0.0f;
        if (a.z) ((T*)a.z)[(uint64_t)i * a.z_ld + j + e] = (T)z;
        if (!none) {
            z = act_value(a.act, z);
            if (a.residual) z += (float)((const T*)a.residual)[(uint64_t)i * a.residual_ld + j + e];
        }
        if (a.wide_out)
            ((float*)a.out)[(uint64_t)g.group * a.out_group + (uint64_t)i * a.out_ld + j + e] = z;
        else
            out[(uint64_t)i * a.out_ld + j + e] = (T)z;
    }
}

// 128 x 128 outputs a workgroup, 64 x 64 a wave.  The matrix instruction takes Q as its
// first operand, so that a lane's four results are neighbours in a row of the output.
constexpr int kTile = 128;

template <typename T, bool PA, bool QA, bool BY_ROWS>
__global__ void __launch_bounds__(256) gemm_kernel(const GemmArgs a) {
    typedef typename Mma<T>::V V;
    __shared__ __align__(16) char lds[2 * kTile * kDepth * 2];
    BLK_LDS char* tp = (BLK_LDS char*)lds;
    BLK_LDS char* tq = tp + kTile * kDepth * 2;
    const int tj = (int)(blockIdx.x % (unsigned)a.tiles_j);
    const int ti = (int)(blockIdx.x / (unsigned)a.tiles_j);
    Range g;
    int i0, i_end, c0, c_end;
    if constexpr (BY_ROWS) {
        if (!find_tile(a, ti, kTile, g)) return;
        i0 = g.lo;
        i_end = g.hi;
        c0 = 0;
        c_end = g.group < 0 ? 0 : a.c;
    } else {
        g = range_of(a, (int)blockIdx.y + 1);
        i0 = ti * kTile;
        i_end = a.i;
        c0 = g.lo;
        c_end = g.hi;
    }
    const int j0 = tj * kTile;
    const T* p = (const T*)a.p;
    const T* q = (const T*)a.q + (BY_ROWS && g.group > 0 ? (uint64_t)g.group * a.q_group : 0);
    const int wave = threadIdx.x >> 6, wi = (wave >> 1) * 64, wj = (wave & 1) * 64;
    f32x4 acc[4][4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) acc[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    Loader<T, PA, kTile, 256> lp;
    Loader<T, QA, kTile, 256> lq;
    if (c0 < c_end) {
        lp.load(p, a.p_ld, i0, i_end, c0, c_end);
        lq.load(q, a.q_ld, j0, a.j, c0, c_end);
    }
    for (int c = c0; c < c_end; c += kDepth) {
        lp.store(tp);
        lq.store(tq);
        __syncthreads();
        if (c + kDepth < c_end) {
            lp.load(p, a.p_ld, i0, i_end, c + kDepth, c_end);
            lq.load(q, a.q_ld, j0, a.j, c + kDepth, c_end);
        }
#pragma unroll
        for (int k = 0; k < kDepth; k += 32) {
            V fp[4], fq[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                fp[x] = Tile<PA, kTile>::template fragment<V>(tp, wi + x * 16, k);
                fq[x] = Tile<QA, kTile>::template fragment<V>(tq, wj + x * 16, k);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) acc[x][y] = Mma<T>::run(fq[y], fp[x], acc[x][y]);
        }
        __syncthreads();
    }
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int i = i0 + wi + x * 16 + (lane & 15);
        if (i >= i_end) continue;
#pragma unroll
        for (int y = 0; y < 4; ++y)
            finish<T>(a, g, BY_ROWS, i, j0 + wj + y * 16 + (lane >> 4) * 4, acc[x][y]);
    }
}

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
        if (a.act != RR_ACT_NONE) {
            const Vec<T> z = load_vec((const T*)a.z + (uint64_t)r * a.z_ld, col, a.n);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = (float)d.e[e] * act_slope(a.act, (float)z.e[e]);
                sum[e] += v;
                o.e[e] = (T)v;
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
    if (g->dout.ld > kMaxLd || (a->act != RR_ACT_NONE && a->n > kMaxLd)) return RR_ERR_UNSUPPORTED;
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

template <bool PA, bool QA, bool BY_ROWS>
static rr_status_t run_gemm(const GemmArgs& k, int dt, int groups, hipStream_t s) {
    const uint64_t blocks = (uint64_t)k.tiles_i * k.tiles_j;
    if (blocks == 0) return RR_OK;
    if (blocks > (1u << 24) - 1) return RR_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks, BY_ROWS ? 1u : (unsigned)groups);
    if (dt == RR_BF16)
        gemm_kernel<bf16, PA, QA, BY_ROWS><<<grid, 256, 0, s>>>(k);
    else
        gemm_kernel<f16, PA, QA, BY_ROWS><<<grid, 256, 0, s>>>(k);
    return launched();
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
    uint64_t dz, part;  // bytes of scratch
};
static BackwardPlan plan_of(const rr_linear_t* a, const rr_linear_grad_t* g) {
    BackwardPlan p = {0, 0};
    if (a->act != RR_ACT_NONE && (g->dx.data || g->dw))
        p.dz = ceil_div(a->rows * ceil_div(a->n, 8) * 8 * 2, 256) * 256;
    if (g->db) p.part = (uint64_t)a->groups * splits_of(a) * a->n * sizeof(float);
    return p;
}

}  // namespace blk

using namespace blk;

extern "C" {

rr_status_t block_linear_workspace(const rr_linear_t* a, size_t* bytes) {
    if (!bytes) return RR_ERR_INVALID;
    const rr_status_t st = check_linear(a);
    if (st != RR_OK) return st;
    *bytes = 0;
    return RR_OK;
}

rr_status_t block_linear(const rr_linear_t* a, void* workspace, size_t workspace_bytes,
                         rr_stream_t stream) {
    (void)workspace;
    (void)workspace_bytes;
    const rr_status_t st = check_linear(a);
    if (st != RR_OK) return st;
    if (!rows_ok(a->out, a->rows, a->n, 2) || !rows_ok_if(a->residual, a->rows, a->n, 2) ||
        !aligned_to(a->bias, 2))
        return RR_ERR_INVALID;
    const uint64_t wide = extent(a->groups, a->w_stride, extent(a->n, a->w_ld, a->k, 1), 2);
    const uint64_t n_out = extent(a->rows, a->out.ld, a->n, 2), n_z = extent(a->rows, a->z.ld, a->n, 2);
    const uint64_t n_res = extent(a->rows, a->residual.ld, a->n, 2);
    const struct { const void* p; uint64_t n; } in[] = {
        {a->x.data, extent(a->rows, a->x.ld, a->k, 2)}, {a->w, wide},
        {a->bias, (uint64_t)a->groups * a->n * 2},
        {a->offsets, (uint64_t)(a->groups + 1) * 4}};
    for (const auto& i : in)
        if (overlap(i.p, i.n, a->out.data, n_out) || overlap(i.p, i.n, a->z.data, n_z))
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
    const uint64_t ti = row_tiles(a, kTile), tj = ceil_div(a->n, kTile);
    if (ti > kMaxSize || tj > kMaxSize) return RR_ERR_UNSUPPORTED;
    k.tiles_i = (int32_t)ti;
    k.tiles_j = (int32_t)tj;
    return run_gemm<false, false, true>(k, a->dt, a->groups, (hipStream_t)stream);
}

rr_status_t block_linear_backward_workspace(const rr_linear_t* a, const rr_linear_grad_t* g,
                                            size_t* bytes) {
    if (!bytes) return RR_ERR_INVALID;
    const rr_status_t st = check_grad(a, g);
    if (st != RR_OK) return st;
    const BackwardPlan p = plan_of(a, g);
    *bytes = p.dz + p.part;
    return RR_OK;
}

rr_status_t block_linear_backward(const rr_linear_t* a, const rr_linear_grad_t* g,
                                  void* workspace, size_t workspace_bytes, rr_stream_t stream) {
    rr_status_t st = check_grad(a, g);
    if (st != RR_OK) return st;
    const BackwardPlan plan = plan_of(a, g);
    const uint64_t need = plan.dz + plan.part;
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
    const uint64_t tj = ceil_div(a->k, kTile);
    const uint64_t ti_x = row_tiles(a, kTile), ti_w = ceil_div(a->n, kTile);
    if (ti_x * tj > (1u << 24) - 1 || ti_w * tj > (1u << 24) - 1) return RR_ERR_UNSUPPORTED;
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
        k.tiles_i = (int32_t)ti_x;
        k.tiles_j = (int32_t)tj;
        if ((st = run_gemm<false, true, true>(k, a->dt, a->groups, s)) != RR_OK) return st;
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
        k.tiles_i = (int32_t)ti_w;
        k.tiles_j = (int32_t)tj;
        if ((st = run_gemm<true, true, false>(k, a->dt, a->groups, s)) != RR_OK) return st;
    }
    return RR_OK;
}

}  // extern "C"
