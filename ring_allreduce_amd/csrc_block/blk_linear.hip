// blk_linear.hip -- the entry points of a block's matrix products (block_linear,
// block_linear_backward): the choice of kernel for each product, the gradient of the
// activation, and the checks.  The products themselves: blk_gemm.hpp.
#include "blk_product.hpp"

namespace blk {

// ------------------------------------------------------- activation's gradient --
//
// dz = dout act'(z), rounded to the rows' type as the next products' operand (or dout as
// it is, where its rows cannot be loaded in 16-byte pieces), and the column sums of each
// group in 32 bits.  A thread takes 8 columns; a workgroup takes
// as many threads across as the columns need, the rest along the rows, and one of `splits`
// parts of a group's rows; the sums are added in a fixed order.
struct SlopeArgs {
    GemmArgs g;            // rows, groups, offsets
    const void *dout, *z;
    void* dz;              // or null: nothing but the sums
    uint64_t dout_ld, z_ld, dz_ld;
    float* part;           // [groups][splits][n], or null
    int32_t n, act, splits, threads;
};

template <typename T>
__global__ void __launch_bounds__(256) slope_kernel(const SlopeArgs a) {
    __shared__ float lds[8][256];
    const int wide = a.threads, high = 256 / wide;      // threads across and along the rows
    const int x = (int)threadIdx.x % wide, y = (int)threadIdx.x / wide;
    const int col = ((int)blockIdx.x * wide + x) * 8;
    const Range g = range_of(a.g, (int)blockIdx.z + 1);
    const int per = (g.hi - g.lo + a.splits - 1) / a.splits;
    const int lo = g.lo + min((int)blockIdx.y * per, g.hi - g.lo), hi = min(lo + per, g.hi);
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
    const T* dout = (const T*)a.dout + col;
    const T* z = a.act != RR_ACT_NONE ? (const T*)a.z + col : dout;
    const uint64_t z_ld = a.act != RR_ACT_NONE ? a.z_ld : a.dout_ld;
    const auto row = [&](int r, u32x4 draw, u32x4 zraw) {
        const Vec<T> d = vec_of<T>(draw), zv = vec_of<T>(zraw);
        Vec<T> o = d;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (float)zv.e[e];
        if (a.act != RR_ACT_NONE) {
            act_slopes(a.act, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] *= (float)d.e[e];
                o.e[e] = (T)v[e];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += v[e];
        // whole vectors: zeros follow the row
        if (a.dz) *(u32x4*)((T*)a.dz + (uint64_t)r * a.dz_ld + col) = __builtin_bit_cast(u32x4, o);
    };
    if (col + 8 <= a.n) {
        int r = lo + y;
        for (; r + 3 * high < hi; r += 4 * high) {
            u32x4 dv[4], zv[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                dv[u] = load_raw(dout + (uint64_t)(r + u * high) * a.dout_ld);
                zv[u] = load_raw(z + (uint64_t)(r + u * high) * z_ld);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) row(r + u * high, dv[u], zv[u]);
        }
        for (; r < hi; r += high)
            row(r, load_raw(dout + (uint64_t)r * a.dout_ld), load_raw(z + (uint64_t)r * z_ld));
    } else if (col < a.n) {
        for (int r = lo + y; r < hi; r += high)
            row(r, __builtin_bit_cast(u32x4, load_vec(dout + (uint64_t)r * a.dout_ld, 0, a.n - col)),
                __builtin_bit_cast(u32x4, load_vec(z + (uint64_t)r * z_ld, 0, a.n - col)));
    }
    if (!a.part) return;
    if (high > 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) lds[e][threadIdx.x] = sum[e];
        __syncthreads();
        if (y > 0) return;
        for (int q = 1; q < high; ++q)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += lds[e][q * wide + x];
    }
    float* to = a.part + ((uint64_t)blockIdx.z * a.splits + blockIdx.y) * a.n;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (col + e < a.n) to[col + e] = sum[e];
}

// Adds the parts of column sums: 16 columns a workgroup, 16 threads each.
__global__ void __launch_bounds__(256)
sum_parts_kernel(const float* part, int splits, int n, float* db) {
    __shared__ float lds[16][17];
    const int c = threadIdx.x & 15, s = threadIdx.x >> 4, col = (int)blockIdx.x * 16 + c;
    const float* from = part + (uint64_t)blockIdx.y * splits * n;
    float sum = 0.0f;
    if (col < n)
#pragma unroll 4
        for (int p = s; p < splits; p += 16) sum += from[(uint64_t)p * n + col];
    lds[s][c] = sum;
    __syncthreads();
    if (s == 0 && col < n) {
        float all = 0.0f;
        for (int q = 0; q < 16; ++q) all += lds[q][c];
        db[(uint64_t)blockIdx.y * n + col] = all;
    }
}

rr_status_t launch_sums(const float* part, int splits, uint64_t n, int groups, float* db, hipStream_t s) {
    sum_parts_kernel<<<dim3((unsigned)ceil_div(n, 16), (unsigned)groups), 256, 0, s>>>(part, splits, (int)n, db);
    return launched();
}

// ------------------------------------------------------------------- alignment --
//
// The products load whole 16-byte pieces, so a matrix whose rows are not made of them is
// copied to one whose rows are, filled up with zeros.  Loading such rows as they are, through
// registers, took 122 us for 6016 x 1111 x 1777 where the copies and the aligned product
// take 66.
struct PackPart {
    const void* from;
    void* to;
    uint64_t ld, group;    // group: elements from one group's first row to the next
    uint64_t vectors;
    int32_t rows, width, wide;   // rows of a group; wide: the copy's row length
};
struct PackArgs {
    PackPart part[2];      // both operands in one launch
};

__global__ void __launch_bounds__(256) pack_kernel(const PackArgs a) {
    const PackPart& m = a.part[blockIdx.y];
    const unsigned each = (unsigned)m.wide / 8;
    for (uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x; id < m.vectors; id += (uint64_t)gridDim.x * 256) {
        const uint64_t row = m.vectors >> 32 ? id / each : (uint32_t)id / each;
        const int at = (int)(id - row * each) * 8;
        const uint32_t group = (uint32_t)row / (uint32_t)m.rows;
        const uint16_t* from = (const uint16_t*)m.from + group * m.group + (row - group * (uint64_t)m.rows) * m.ld;
        const Some<uint16_t, 8> v = load_some<uint16_t, 8>(from + at, m.width - at);
        *(u32x4*)((uint16_t*)m.to + id * 8) = __builtin_bit_cast(u32x4, v);
    }
}

// ------------------------------------------------------------------ host side --

// All of it but the activation; the bytes of an element of x and of w.
rr_status_t check_linear_sizes(const rr_linear_t* a, uint64_t x_bytes, uint64_t w_bytes) {
    if (!a || a->reserved) return RR_ERR_INVALID;
    if (a->dt != RR_BF16 && a->dt != RR_FP16)
        return a->dt == RR_FP32 ? RR_ERR_UNSUPPORTED : RR_ERR_INVALID;
    if (a->n < 1 || a->k < 1 || a->groups < 1) return RR_ERR_INVALID;
    if (a->rows > kMaxSize || a->n > kMaxSize || a->k > kMaxSize || a->groups > RR_MAX_EXPERTS)
        return RR_ERR_UNSUPPORTED;
    if (!a->offsets && a->rows % (uint64_t)a->groups) return RR_ERR_INVALID;
    if (!aligned_to(a->offsets, 4)) return RR_ERR_INVALID;
    if (!a->w || !aligned_to(a->w, w_bytes) || a->w_ld < a->k) return RR_ERR_INVALID;
    if (a->groups > 1 && a->w_stride < extent(a->n, a->w_ld, a->k, 1)) return RR_ERR_INVALID;
    if (!rows_ok(a->x, a->rows, a->k, x_bytes)) return RR_ERR_INVALID;
    if (a->x.ld > kMaxLd || a->w_ld > kMaxLd) return RR_ERR_UNSUPPORTED;
    if (a->groups > 1 && a->w_stride > (1ull << 44)) return RR_ERR_UNSUPPORTED;
    return RR_OK;
}

static rr_status_t check_linear(const rr_linear_t* a, uint64_t x_bytes = 2, uint64_t w_bytes = 2) {
    const rr_status_t st = check_linear_sizes(a, x_bytes, w_bytes);
    if (st == RR_ERR_INVALID) return st;
    if (a->act < RR_ACT_NONE || a->act > RR_ACT_SILU) return RR_ERR_INVALID;
    if (!rows_ok_if(a->z, a->rows, a->n, 2)) return RR_ERR_INVALID;
    return st;
}

// The scales of 8-bit operands; none: 16 bits.
struct Eight {
    const float *x, *w;
};

static rr_status_t check_grad(const rr_linear_t* a, const rr_linear_grad_t* g, const Eight& e) {
    const rr_status_t st = check_linear(a, e.x ? 1 : 2, e.w ? 1 : 2);
    if (st != RR_OK) return st;
    if (!g || g->reserved) return RR_ERR_INVALID;
    if (g->dw_dt != a->dt && g->dw_dt != RR_FP32) return RR_ERR_INVALID;
    if (!rows_ok(g->dout, a->rows, a->n, 2) || !rows_ok_if(g->dx, a->rows, a->k, 2))
        return RR_ERR_INVALID;
    if (a->act != RR_ACT_NONE && !rows_ok(a->z, a->rows, a->n, 2)) return RR_ERR_INVALID;
    if (!aligned_to(g->dw, type_bytes(g->dw_dt)) || !aligned_to(g->db, 4)) return RR_ERR_INVALID;
    if (!aligned_to(e.x, 4) || !aligned_to(e.w, 4)) return RR_ERR_INVALID;
    // copies of 8-bit operands count rows in 32 bits
    if (e.w && (uint64_t)a->groups * a->n > kMaxSize) return RR_ERR_UNSUPPORTED;
    if (g->dout.ld > kMaxLd || (g->dx.data && g->dx.ld > kMaxLd) || (a->act != RR_ACT_NONE && a->n > kMaxLd)) return RR_ERR_UNSUPPORTED;
    return RR_OK;
}

GemmArgs groups_of(const rr_linear_t* a) {
    GemmArgs k = {};
    k.rows = (int32_t)a->rows;
    k.groups = a->groups;
    k.offsets = a->offsets;
    return k;
}

// Row tiles of all groups, at most: each that has rows can add one partly filled, and so can
// the rows before the first and after the last one.
uint64_t row_tiles(const rr_linear_t* a, uint64_t height) {
    if (a->groups == 1 && !a->offsets) return ceil_div(a->rows, height);
    const uint64_t ranges = (uint64_t)a->groups + 2;
    return a->rows / height + (a->rows < ranges ? a->rows : ranges);
}

// The kernel and the parts of the contraction for one product: the least of the times that
// these figures give, fitted on an MI355X to 320 products of 32 to 6400 rows and 128 to 8192
// columns and depths, each with every tile and 1 to 16 parts (microseconds; a step is 64
// deep).  Over 354 such products of 16 to 6400 rows the choice takes 1.009 of the best on
// average; 36 take more than 1.05 of it, 12 more than 1.1, the worst 1.36 (6400 x 768 x 768 by
// w).  The figures are for the whole device: with fewer compute units (a partition of it) the
// results are the same, and the choice is off.
//   tile       start   a step, with 1 .. 4 workgroups on each compute unit
//   256 x 256   11.3    1.63 (1.1 on an empty device)
//   128 x 128    6.6    0.73 (0.47), 1.16
//    64 x  64    3.8    0.28, 0.51, 0.73, 0.83
// A further round costs 0.6 of a start; parts cost 4.6 for the second launch and their bytes,
// written and read.  Up to 64 rows of a long contraction may be cut inside the workgroup
// instead (kInner64: 64 x 32, four parts; start 7.2, 3.6 for a further round, a step of all
// parts 0.3 to 0.56): 32 x 8192 x 8192 25.5 us against 29.7, 32 x 4096 x 4096 13.3 against
// 14.9, but 32 x 16384 x 4096 29.4 against 24.7 and 32 x 1024 x 4096 11.9 against 10.4.  A few
// rows go through the one-pass form, to 64 rows where the contraction is too short for parts
// to pay (48 x 8192 x 1024: 9.4 us against 10.2; 48 x 1024 x 8192: 40 against 16), and up to 16
// where that is the better time (16 x 4096 x 4096 11.8 us against 12.9, 16 x 8192 x 8192 34
// against 25; the tiles only for whole 16-byte pieces, copies of the weights would cost more).
GemmPlan choose(const rr_linear_t* a, int form, int* splits, int* slots) {
    const uint64_t groups = (uint64_t)a->groups, mean = ceil_div(a->rows, groups);
    const uint64_t i = form == kByW ? a->n : a->rows, j = form == kForward ? a->n : a->k;
    const uint64_t c = form == kForward ? a->k : form == kByX ? a->n : mean;
    const double outputs = (double)(form == kByW ? groups * i : i) * j;
    GemmPlan p = {form, kTile64, 0, 0, 0};
    *splits = 1;
    *slots = 0;
    if (form == kForward && groups == 1 && !a->offsets && a->rows <= 2) {
        p.tile = kDot;
        return p;
    }
    double best = 1e30;
    const bool few = form == kForward && mean <= 64;
    // of uneven groups, those of more than 16 rows would read their weights twice (32 groups of
    // 4096 x 2048: 400 rows 128 us with tiles of 16, 142 with 32; 512 rows 159 and 146)
    const uint64_t some = groups > 1 && a->offsets ? mean * 5 / 4 : mean;
    if (few && (mean <= 16 || c <= 1024)) {
        p.tile = some <= 16 ? kStream16 : mean <= 32 ? kStream32 : kStream64;
        // 16 columns a workgroup instead of 32 where that gives a compute unit no more than two,
        // of more rows than 16 one: 4 x 8192 x 8192 27 us against 31, 4 x 4096 x 4096 9.9 (12.2),
        // 4 x 1024 x 4096 8.7 (9.6), 64 x 4096 x 1024 9.0 (10.0); but 4 x 16384 x 1024 9.8
        // (9.2), 64 x 8200 x 1000 14.4 (12.1), and with longer rows 4 x 8192 x 16384 54 (44),
        // 4 x 2048 x 16384 20.8 (18.7)
        const uint64_t high = a->rows ? ceil_div(a->rows, tile_rows(p.tile)) : 1;
        p.narrow = c <= 8192 && ceil_div(j, 16) * high <= (p.tile == kStream16 ? 2 : 1) * kSlots;
        const uint64_t blocks = ceil_div(j, p.cols()) * high;
        const uint64_t want = 256 / blocks, most = c / 1024;
        const uint64_t n = want < most ? want : most;
        *splits = n < 2 ? 1 : n > 16 ? 16 : (int)n;
        if (mean > 16 || groups > 1 || a->offsets || c <= 1024 || c > 8192 || !good_rows(a->x, 0, a->k) ||
            !good_rows({const_cast<void*>(a->w), a->w_ld}, 0, a->k))
            return p;
        const double uneven = blocks > kSlots ? (double)ceil_div(blocks, kSlots) * kSlots / blocks : 1;
        best = 0.93 * (4 + (*splits > 1 ? 3.5 : 0) + 2.0 * j * c / 5.9e6 * (1 + mean / 64.0) * uneven);
    }
    if (few) {
        const uint64_t high = groups == 1 ? ceil_div(i, 64) : i / 64 + ceil_div(groups, 2);
        const uint64_t blocks = (high ? high : 1) * ceil_div(j, 32), more = (blocks - 1) / kSlots;
        const double fill = (double)(blocks - more * kSlots) / kSlots;
        const double steps = (double)ceil_div(ceil_div(c, kDepth), 4);
        const double time = (7.2 + 3.6 * more + steps * (0.56 * more + 0.3 + 0.26 * fill * fill)) * (0.92 + 0.09 * mean / 64);
        if (time < best) {
            best = time;
            p.tile = kInner64;
            *splits = 1;
        }
    }
    for (int tile = kTile256; tile <= kTile64; ++tile) {
        const uint64_t t = tile_rows(tile), each = tile == kTile256 ? 1 : tile == kTile128 ? 2 : 4;
        const uint64_t high = form == kByW ? groups * ceil_div(i, t)
                              : groups == 1 ? ceil_div(i, t) : i / t + ceil_div(groups, 2);
        const uint64_t tiles = (high ? high : 1) * ceil_div(j, t), steps = ceil_div(c, kDepth);
        // of few rows, no more than two tiles on a compute unit: their loads are what takes time
        // then (16 x 16384 x 8192 50 us with four, 43 with two)
        for (uint64_t s = 1; s <= 32 && (s == 1 || (s <= steps / 2 && tiles * s <= (few ? 512 : 1024))); s *= 2) {
            const uint64_t blocks = tiles * s, rounds = ceil_div(blocks, 256 * each);
            const uint64_t load = rounds > 1 ? each : ceil_div(blocks, 256);
            const double fill = blocks < 256 ? blocks / 256.0 : 1.0;
            const double start = tile == kTile256 ? 11.3 : tile == kTile128 ? 6.6 : 3.8;
            const double step = tile == kTile256   ? 1.11 + 0.52 * fill
                                : tile == kTile128 ? (load == 1 ? 0.47 + 0.26 * fill : 1.16)
                                : load == 1 ? 0.28 : load == 2 ? 0.51 : load == 3 ? 0.73 : 0.83;
            double time = start * (0.4 + 0.6 * rounds) + rounds * step * ceil_div(steps, s);
            if (s > 1) time += 4.6 + 8.0 * s * outputs / 5.95e6;
            int last = 0;
            if (tile == kTile256 && s == 1 && (form != kByW || (groups == 1 && !a->offsets))) {
                const unsigned rest = (unsigned)(tiles % kSlots);
                const int parts = last_round_parts(rest, kSlots, (int)steps);
                // how many tiles uneven groups make is known on the device only
                if (parts > 1 || (form != kByW && a->offsets && rounds < 16 && steps >= 16)) last = kSlots;
                if (parts > 1) time += 4 + 0.12 * rest * parts - step * (steps - ceil_div(steps, parts));
            }
            if (time < best) {
                best = time;
                p.tile = tile;
                p.deep = rounds == 1 && load <= (tile == kTile64 ? 2 : 1);
                *splits = (int)s;
                *slots = last;
            }
        }
    }
    return p;
}

uint64_t product_bytes(const rr_linear_t* a, int form, const Operand& p, const Operand& q) {
    int splits, slots;
    const GemmPlan plan = choose(a, form, &splits, &slots);
    uint64_t bytes = (uint64_t)slots * 256 * 256 * sizeof(float);
    if (splits > 1) {
        const uint64_t rows = form == kByW ? (uint64_t)a->groups * a->n : a->rows;
        bytes = ceil_div((uint64_t)splits * rows * (form == kForward ? a->n : a->k) * sizeof(float), 256) * 256;
    }
    if (plan.tile < kStream16) bytes += (p.good() ? 0 : p.copy_bytes()) + (q.good() ? 0 : q.copy_bytes());
    return bytes;
}

// Copies the operands that are not good into the scratch memory at `room`.
static rr_status_t pack(int dt, Operand& p, Operand& q, char* room, hipStream_t s) {
    PackArgs k = {};
    int n = 0;
    uint64_t blocks = 0;
    for (Operand* o : {&p, &q}) {
        if (o->good()) continue;
        if (o->scales) {
            BlockArgs b = {};
            b.wide = room;
            b.wide_ld = ceil_div(o->width, 8) * 8;
            b.wide_group = o->count * b.wide_ld;
            b.narrow = (uint8_t*)o->rows.data;
            b.narrow_ld = o->rows.ld;
            b.narrow_group = o->group;
            b.scales = const_cast<float*>(o->scales);
            b.rows = o->count;
            b.groups = o->groups;
            b.part = o->part;
            b.width = (int32_t)o->width;
            b.blocks = (int32_t)ceil_div(o->width, kBlock);
            b.filled = (int32_t)b.wide_ld;
            b.high = (int32_t)o->high;
            const rr_status_t st = launch_back(b, dt, s);
            if (st != RR_OK) return st;
            room += o->copy_bytes();
            *o = {{b.wide, b.wide_ld}, o->count, b.wide_ld, o->groups, b.wide_group};
            continue;
        }
        PackPart& m = k.part[n];
        m = {o->rows.data, room, o->rows.ld, o->group, 0, (int32_t)o->count, (int32_t)o->width,
             (int32_t)(ceil_div(o->width, 8) * 8)};
        m.vectors = o->groups * o->count * (uint64_t)m.wide / 8;
        if (o->groups * o->count > 0xFFFFFFFFull) return RR_ERR_UNSUPPORTED;
        room += o->copy_bytes();
        o->rows = {m.to, (uint64_t)m.wide};
        o->width = (uint64_t)m.wide;
        o->group = o->count * (uint64_t)m.wide;
        if (m.vectors == 0) continue;
        const uint64_t b = ceil_div(m.vectors, 256);
        blocks = b > blocks ? b : blocks;
        ++n;
    }
    if (n == 0) return RR_OK;
    pack_kernel<<<dim3((unsigned)(blocks < 8192 ? blocks : 8192), (unsigned)n), 256, 0, s>>>(k);
    return launched();
}

rr_status_t run_product(const rr_linear_t* a, Product r, void* workspace, hipStream_t s) {
    GemmArgs& k = r.k;
    int splits, slots;
    GemmPlan plan = choose(a, r.form, &splits, &slots);
    const uint64_t ti = r.form == kByW ? ceil_div(k.i, tile_rows(plan.tile)) : row_tiles(a, tile_rows(plan.tile));
    const uint64_t tj = ceil_div(k.j, plan.cols());
    if (ti * tj == 0) return RR_OK;
    if (ti * tj * splits * (r.form == kByW ? (uint64_t)a->groups : 1) > (1u << 23) - 1) return RR_ERR_UNSUPPORTED;
    k.tiles_i = (int32_t)ti;
    k.tiles_j = (int32_t)tj;
    k.splits = splits;
    k.part_stride = (r.form == kByW ? (uint64_t)k.groups * k.i : (uint64_t)k.rows) * k.j;
    if (splits > 1) {
        if (ceil_div((k.part_stride / k.j) * ceil_div(k.j, 4), 256) > (1u << 24) - 1) return RR_ERR_UNSUPPORTED;
        k.part = (float*)workspace;
    }
    char* room = (char*)workspace;
    if (splits > 1) room += ceil_div((uint64_t)splits * k.part_stride * sizeof(float), 256) * 256;
    if (slots) {
        k.slots = slots;
        k.steps = (int32_t)ceil_div(r.form == kByW ? a->rows : (uint64_t)k.c, kDepth);
        k.part = (float*)workspace;
        room += (uint64_t)slots * 256 * 256 * sizeof(float);
    }
    plan.direct = r.p.good() && r.q.good();
    if (plan.tile == kStream16 && !plan.direct && a->groups == 1 && !a->offsets && a->rows <= 4) {
        plan.tile = kDot;
        k.splits = 1;
    }
    if (plan.tile < kStream16) {
        const rr_status_t st = pack(a->dt, r.p, r.q, room, s);
        if (st != RR_OK) return st;
    }
    k.p = r.p.rows.data;
    k.p_ld = r.p.rows.ld;
    k.q = r.q.rows.data;
    k.q_ld = r.q.rows.ld;
    k.q_group = r.q.group;
    return a->dt == RR_BF16 ? launch_gemm_bf16(k, plan, s) : launch_gemm_f16(k, plan, s);
}

Operand rows_of(const rr_linear_t* a, const rr_rows_t& r, uint64_t width) {
    return {r, a->rows, width, 1, 0};
}
Operand weights_of(const rr_linear_t* a) {
    return {{const_cast<void*>(a->w), a->w_ld}, a->n, a->k, (uint64_t)a->groups, a->w_stride};
}

uint64_t sum_threads(const rr_linear_t* a) {
    uint64_t t = 1;
    while (t < 256 && t * 8 < a->n) t *= 2;
    return t;
}
uint64_t sum_splits(const rr_linear_t* a) {
    const uint64_t t = sum_threads(a), cols = ceil_div(a->n, t * 8) * a->groups;
    const uint64_t each = ceil_div(a->rows, a->groups);
    const uint64_t want = ceil_div(2048, cols), most = ceil_div(each, 256 / t * 4);
    const uint64_t n = want < most ? want : most;
    return n < 1 ? 1 : n > 1024 ? 1024 : n;
}

struct BackwardPlan {
    uint64_t dz, part, product;  // bytes of scratch
};
static Operand x_of(const rr_linear_t* a, const Eight& e) {
    Operand o = rows_of(a, a->x, a->k);
    o.scales = e.x;
    o.part = a->rows;
    return o;
}
static Operand w_of(const rr_linear_t* a, const Eight& e) {
    Operand o = weights_of(a);
    o.scales = e.w;
    o.high = kBlock;
    o.part = a->n;
    return o;
}
static BackwardPlan plan_of(const rr_linear_t* a, const rr_linear_grad_t* g, const Eight& e) {
    BackwardPlan p = {0, 0, 0};
    const Operand dout = rows_of(a, g->dout, a->n);
    if ((g->dx.data || g->dw) && (a->act != RR_ACT_NONE || !dout.good())) p.dz = dout.copy_bytes();
    if (g->db && sum_splits(a) > 1) p.part = ceil_div((uint64_t)a->groups * sum_splits(a) * a->n * sizeof(float), 256) * 256;
    Operand dz = dout;
    if (p.dz) dz.rows = {nullptr, ceil_div(a->n, 8) * 8};
    dz.width = ceil_div(a->n, 8) * 8;       // good rows, or a copy with zeros behind each
    if (g->dx.data) p.product = product_bytes(a, kByX, dz, w_of(a, e));
    if (g->dw) {
        const uint64_t bytes = product_bytes(a, kByW, dz, x_of(a, e));
        if (bytes > p.product) p.product = bytes;
    }
    return p;
}

static rr_status_t backward_bytes(const rr_linear_t* a, const rr_linear_grad_t* g, const Eight& e, size_t* bytes) {
    if (!bytes) return RR_ERR_INVALID;
    const rr_status_t st = check_grad(a, g, e);
    if (st != RR_OK) return st;
    const BackwardPlan p = plan_of(a, g, e);
    *bytes = p.dz + p.part + p.product;
    return RR_OK;
}

static rr_status_t backward(const rr_linear_t* a, const rr_linear_grad_t* g, const Eight& e,
                            void* workspace, size_t workspace_bytes, hipStream_t s) {
    rr_status_t st = check_grad(a, g, e);
    if (st != RR_OK) return st;
    const BackwardPlan plan = plan_of(a, g, e);
    const uint64_t need = plan.dz + plan.part + plan.product;
    if (need && (!workspace || !aligned_to(workspace, 16) || workspace_bytes < need))
        return RR_ERR_INVALID;
    const uint64_t blocks = ceil_div(a->k, kBlock);
    const struct { const void* p; uint64_t n; } in[] = {
        {g->dout.data, extent(a->rows, g->dout.ld, a->n, 2)},
        {a->x.data, extent(a->rows, a->x.ld, a->k, e.x ? 1 : 2)}, {a->w, weights_extent(a, e.w ? 1 : 2)},
        {e.x, a->rows * blocks * 4}, {e.w, (uint64_t)a->groups * ceil_div(a->n, kBlock) * blocks * 4},
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
    rr_rows_t dz = g->dout;
    void* const room = (char*)workspace + plan.dz + plan.part;
    if (plan.dz || g->db) {
        SlopeArgs k = {};
        k.g = groups_of(a);
        k.dout = g->dout.data;
        k.dout_ld = g->dout.ld;
        k.z = a->z.data;
        k.z_ld = a->z.ld;
        k.n = (int32_t)a->n;
        k.act = a->act;
        k.splits = (int32_t)sum_splits(a);
        k.threads = (int32_t)sum_threads(a);
        if (plan.dz) {
            dz = {workspace, ceil_div(a->n, 8) * 8};
            k.dz = dz.data;
            k.dz_ld = dz.ld;
        }
        k.part = plan.part ? (float*)((char*)workspace + plan.dz) : g->db;
        const uint64_t cols = ceil_div(a->n, (uint64_t)k.threads * 8);
        if (cols > (1u << 24) - 1) return RR_ERR_UNSUPPORTED;
        const dim3 grid((unsigned)cols, (unsigned)k.splits, (unsigned)a->groups);
        if (a->dt == RR_BF16)
            slope_kernel<bf16><<<grid, 256, 0, s>>>(k);
        else
            slope_kernel<f16><<<grid, 256, 0, s>>>(k);
        if ((st = launched()) != RR_OK) return st;
        if (plan.part && (st = launch_sums(k.part, k.splits, a->n, a->groups, g->db, s)) != RR_OK) return st;
    }
    Operand by = rows_of(a, dz, ceil_div(a->n, 8) * 8);     // zeros behind the columns, if any
    if (g->dx.data && a->rows) {
        Product r = {kByX, by, w_of(a, e), groups_of(a)};
        r.k.i = (int32_t)a->rows;
        r.k.j = (int32_t)a->k;
        r.k.c = (int32_t)a->n;
        r.k.out = g->dx.data;
        r.k.out_ld = g->dx.ld;
        if ((st = run_product(a, r, room, s)) != RR_OK) return st;
    }
    if (g->dw) {
        Product r = {kByW, by, x_of(a, e), groups_of(a)};
        r.k.i = (int32_t)a->n;
        r.k.j = (int32_t)a->k;
        r.k.out = g->dw;
        r.k.out_ld = a->k;
        r.k.out_group = (uint64_t)a->n * a->k;
        r.k.wide_out = g->dw_dt == RR_FP32;
        if ((st = run_product(a, r, room, s)) != RR_OK) return st;
    }
    return RR_OK;
}

}  // namespace blk

using namespace blk;

extern "C" {

rr_status_t block_linear_workspace(const rr_linear_t* a, size_t* bytes) {
    if (!bytes) return RR_ERR_INVALID;
    const rr_status_t st = check_linear(a);
    if (st != RR_OK) return st;
    *bytes = product_bytes(a, kForward, rows_of(a, a->x, a->k), weights_of(a));
    return RR_OK;
}

rr_status_t block_linear(const rr_linear_t* a, void* workspace, size_t workspace_bytes,
                         rr_stream_t stream) {
    const rr_status_t st = check_linear(a);
    if (st != RR_OK) return st;
    const uint64_t need = product_bytes(a, kForward, rows_of(a, a->x, a->k), weights_of(a));
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
    Product r = {kForward, rows_of(a, a->x, a->k), weights_of(a), groups_of(a)};
    GemmArgs& k = r.k;
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
    return run_product(a, r, workspace, (hipStream_t)stream);
}

rr_status_t block_linear_backward_workspace(const rr_linear_t* a, const rr_linear_grad_t* g,
                                            size_t* bytes) {
    return backward_bytes(a, g, {nullptr, nullptr}, bytes);
}

rr_status_t block_linear_backward(const rr_linear_t* a, const rr_linear_grad_t* g,
                                  void* workspace, size_t workspace_bytes, rr_stream_t stream) {
    return backward(a, g, {nullptr, nullptr}, workspace, workspace_bytes, (hipStream_t)stream);
}

rr_status_t block_linear8_backward_workspace(const rr_linear8_t* a, const rr_linear_grad_t* g,
                                             size_t* bytes) {
    if (!a || a->z_scales) return RR_ERR_INVALID;
    return backward_bytes(&a->l, g, {a->x_scales, a->w_scales}, bytes);
}

rr_status_t block_linear8_backward(const rr_linear8_t* a, const rr_linear_grad_t* g,
                                   void* workspace, size_t workspace_bytes, rr_stream_t stream) {
    if (!a || a->z_scales) return RR_ERR_INVALID;
    return backward(&a->l, g, {a->x_scales, a->w_scales}, workspace, workspace_bytes, (hipStream_t)stream);
}

}  // extern "C"
