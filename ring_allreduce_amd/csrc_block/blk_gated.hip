// blk_gated.hip -- the entry points of a block's gated projections and of the products of 8-bit
// operands (block_gated, block_linear8 and their gradients): the checks, the operands, and the
// gradient of the gate.  The products themselves: blk_tile.hpp, for few rows blk_gemm.hpp and
// blk_gemm8.hpp, and blk_gemm.hpp for the gradients.
#include "blk_product.hpp"

namespace blk {

// --------------------------------------------------------------- gate's gradient --
//
// z = [g | u]:  dg = dout u act'(g), du = dout act(g), rounded to the rows' type as the next
// products' operand; the column sums of each group in 32 bits, and act(g) u once more, if
// wanted.  One read of dout and z for all of them.  A thread takes 8 columns of both halves,
// a workgroup as many threads across as the columns need, the rest along the rows, and one
// of `splits` parts of a group's rows; the sums are added in a fixed order.
struct GateArgs {
    GemmArgs g;                // rows, groups, offsets
    const void *dout, *z;
    const float* z_scale;      // or null: z in the rows' type
    void *dz, *out;            // or null
    float* part;               // [groups][splits][2 n], or null
    uint64_t dout_ld, z_ld, dz_ld, out_ld;
    int32_t n, act, splits, threads, blocks;
};

// act(z) and its slope at once: the exponential is most of either.
template <int ACT> __device__ __forceinline__ void gate_of(float z, float& value, float& slope) {
    if constexpr (ACT == RR_ACT_GELU) {
        const float a = magnitude(z);
        float tail;
        const float e = normal_tail(a, &tail);
        value = fmaxf(z, 0.0f) - a * tail;
        slope = (z > 0.0f ? 1.0f - tail : tail) + copysignf(a, z) * e * 0.39894228040143268f;
    } else if constexpr (ACT == RR_ACT_SILU) {
        const float q = logistic(z);
        value = z * q;
        slope = q * (1.0f + z * (1.0f - q));
    } else if constexpr (ACT == RR_ACT_SIGMOID) {
        value = logistic(z);
        slope = value * (1.0f - value);
    } else {
        value = act_of<ACT>(z);
        slope = slope_of<ACT>(z);
    }
}

// 8 columns of both halves of z and of dout.
template <typename T, bool EIGHT> struct GateRow {
    u32x4 dout, z[2];
    float scale[2];
    // WHOLE: all of the 8 are there
    template <bool WHOLE> __device__ __forceinline__ void load(const GateArgs& a, int r, int col) {
        const T* d = (const T*)a.dout + (uint64_t)r * a.dout_ld + col;
        if constexpr (WHOLE) dout = load_raw(d);
        else dout = a.dout ? __builtin_bit_cast(u32x4, load_some<T, 8>(d, a.n - col)) : u32x4{};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (EIGHT) {
                const uint8_t* from = (const uint8_t*)a.z + (uint64_t)r * a.z_ld + (uint64_t)h * a.n + col;
                Words<8>::V v;
                if constexpr (WHOLE) v = ((const LooseWords<uint8_t, 8>*)from)->v;
                else v = __builtin_bit_cast(Words<8>::V, load_some<uint8_t, 8>(from, a.n - col));
                z[h] = u32x4{v[0], v[1], 0, 0};
                scale[h] = a.z_scale[((uint64_t)r * 2 + h) * a.blocks + col / 128];
            } else {
                const T* from = (const T*)a.z + (uint64_t)r * a.z_ld + (uint64_t)h * a.n + col;
                if constexpr (WHOLE) z[h] = load_raw(from);
                else z[h] = __builtin_bit_cast(u32x4, load_some<T, 8>(from, a.n - col));
            }
        }
    }
    __device__ __forceinline__ void values(int h, float (&v)[8]) const {
        if constexpr (EIGHT) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)z[h][k], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)z[h][k], true);
                v[k * 4] = lo[0] * scale[h], v[k * 4 + 1] = lo[1] * scale[h], v[k * 4 + 2] = hi[0] * scale[h], v[k * 4 + 3] = hi[1] * scale[h];
            }
        } else {
            const Vec<T> e = vec_of<T>(z[h]);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = (float)e.e[k];
        }
    }
};

// Bound by memory: 16384 x 4096 in bf16, 671 MB in 141 us (4.8 TB/s; one row's loads at a time,
// behind a branch, 219).
template <typename T, bool EIGHT, int ACT> __global__ void __launch_bounds__(256) gate_kernel(const GateArgs a) {
    __shared__ float lds[8][256];
    const int wide = a.threads, high = 256 / wide;      // threads across and along the rows
    const int x = (int)threadIdx.x % wide, y = (int)threadIdx.x / wide;
    const int own = ((int)blockIdx.x * wide + x) * 8;
    // The last columns' thread takes the last 8, some of them its neighbour's too, which get the
    // same values twice; but not across the border of two scales.
    const bool back = own < a.n && own + 8 > a.n && a.n >= 8 && !(EIGHT && (a.n & 127) < 8);
    const int col = back ? a.n - 8 : own, left = a.n - col;
    const bool none = (int)blockIdx.z >= a.g.groups;    // the rows of no group
    const Range g = range_of(a.g, none ? ((int)blockIdx.z == a.g.groups ? 0 : a.g.groups + 1) : (int)blockIdx.z + 1);
    const int per = (g.hi - g.lo + a.splits - 1) / a.splits;
    const int lo = g.lo + min((int)blockIdx.y * per, g.hi - g.lo), hi = min(lo + per, g.hi);
    if (none) {
        const float zeros[8] = {};
        if (a.out && left > 0)
            for (int r = lo + y; r < hi; r += high) store_some<T, 8>((T*)a.out + (uint64_t)r * a.out_ld + col, left, zeros);
        return;
    }
    float sum[2][8] = {};
    typedef GateRow<T, EIGHT> Row;
    const auto row = [&](int r, const Row& in, auto whole_) {
        const int n = decltype(whole_)::value ? 8 : left;
        float g[8], u[8], s[8];
        in.values(0, g);
        in.values(1, u);
        const Vec<T> d = vec_of<T>(in.dout);
#pragma unroll
        for (int e = 0; e < 8; ++e) gate_of<ACT>(g[e], g[e], s[e]);
        if (a.out) {
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = g[e] * u[e];
            store_some<T, 8>((T*)a.out + (uint64_t)r * a.out_ld + col, n, o);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s[e] *= (float)d.e[e] * u[e];
            g[e] *= (float)d.e[e];
            sum[0][e] += s[e];
            sum[1][e] += g[e];
        }
        if (a.dz) {
            T* const to = (T*)a.dz + (uint64_t)r * a.dz_ld;
            store_some<T, 8>(to + col, n, s);
            store_some<T, 8>(to + a.n + col, n, g);
            // zeros behind the row's 2 n columns
            if (left <= 8)
                for (uint64_t c = 2 * (uint64_t)a.n; c < a.dz_ld; ++c) to[c] = (T)0.0f;
        }
    };
    if (left >= 8 && a.dout) {
        constexpr int U = 4;                            // rows on their way
        int r = lo + y;
        for (; r + (U - 1) * high < hi; r += U * high) {
            Row in[U];
#pragma unroll
            for (int u = 0; u < U; ++u) in[u].template load<true>(a, r + u * high, col);
#pragma unroll
            for (int u = 0; u < U; ++u) row(r + u * high, in[u], std::true_type());
        }
        for (; r < hi; r += high) {
            Row in;
            in.template load<true>(a, r, col);
            row(r, in, std::true_type());
        }
    } else if (left > 0) {
        for (int r = lo + y; r < hi; r += high) {
            Row in;
            in.template load<false>(a, r, col);
            row(r, in, std::false_type());
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (high > 1) {
            if (h) __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) lds[e][threadIdx.x] = sum[h][e];
            __syncthreads();
            if (y == 0)
                for (int q = 1; q < high; ++q)
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum[h][e] += lds[e][q * wide + x];
        }
        float* to = a.part + ((uint64_t)blockIdx.z * a.splits + blockIdx.y) * 2 * a.n + (uint64_t)h * a.n;
        if (y == 0)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left && col + e >= own) to[col + e] = sum[h][e];
    }
}

template <typename T, bool EIGHT> static void launch_gate(const GateArgs& k, const dim3& grid, hipStream_t s) {
    switch (k.act) {
        case RR_ACT_RELU: gate_kernel<T, EIGHT, RR_ACT_RELU><<<grid, 256, 0, s>>>(k); break;
        case RR_ACT_GELU: gate_kernel<T, EIGHT, RR_ACT_GELU><<<grid, 256, 0, s>>>(k); break;
        case RR_ACT_SILU: gate_kernel<T, EIGHT, RR_ACT_SILU><<<grid, 256, 0, s>>>(k); break;
        case RR_ACT_SIGMOID: gate_kernel<T, EIGHT, RR_ACT_SIGMOID><<<grid, 256, 0, s>>>(k); break;
        default: gate_kernel<T, EIGHT, RR_ACT_NONE><<<grid, 256, 0, s>>>(k);
    }
}

// ------------------------------------------------------------------ host side --

// The same block with the columns of both halves for `n`, as its products see it.
static rr_linear_t both_halves(const rr_linear8_t* a) {
    rr_linear_t l = a->l;
    l.n = a->l.n * 2;
    return l;
}

static uint64_t scale_blocks(uint64_t width) { return ceil_div(width, kBlock); }

// Sizes and operands of a call; `halves` 2: of block_gated.
static rr_status_t check_operands(const rr_linear8_t* a, uint64_t halves) {
    if (!a) return RR_ERR_INVALID;
    rr_linear_t l = a->l;
    if (l.n > kMaxSize) return RR_ERR_UNSUPPORTED;
    l.n *= halves;
    const rr_status_t st = check_linear_sizes(&l, a->x_scales ? 1 : 2, a->w_scales ? 1 : 2);
    if (st == RR_ERR_INVALID) return st;
    if (l.act < RR_ACT_NONE || l.act > (halves == 2 ? RR_ACT_SIGMOID : RR_ACT_SILU)) return RR_ERR_INVALID;
    if (!aligned_to(a->x_scales, 4) || !aligned_to(a->w_scales, 4) || !aligned_to(a->z_scales, 4)) return RR_ERR_INVALID;
    if (halves == 1 ? a->z_scales != nullptr : l.residual.data != nullptr) return RR_ERR_INVALID;
    if (!rows_ok_if(l.z, l.rows, l.n, a->z_scales ? 1 : 2)) return RR_ERR_INVALID;
    if (a->z_scales && !l.z.data && l.rows) return RR_ERR_INVALID;
    if (st != RR_OK) return st;
    if (l.n > kMaxLd || (l.z.data && l.z.ld > kMaxLd)) return RR_ERR_UNSUPPORTED;
    // copies of operands count rows in 32 bits, and so do the halves of z in 8 bits
    if ((uint64_t)l.groups * l.n > kMaxSize || (a->z_scales && l.rows * 2 > kMaxSize)) return RR_ERR_UNSUPPORTED;
    return RR_OK;
}

struct Span {
    const void* p;
    uint64_t n;
};
static bool any_overlap(const Span* in, int ins, const Span* out, int outs) {
    for (int o = 0; o < outs; ++o) {
        for (int i = 0; i < ins; ++i)
            if (overlap(out[o].p, out[o].n, in[i].p, in[i].n)) return true;
        for (int q = o + 1; q < outs; ++q)
            if (overlap(out[o].p, out[o].n, out[q].p, out[q].n)) return true;
    }
    return false;
}
constexpr int kInputs = 6;
// x, w, both scales, offsets and bias.
static void inputs_of(const rr_linear8_t* a, uint64_t halves, Span (&in)[kInputs]) {
    rr_linear_t l = a->l;
    l.n *= halves;
    const uint64_t blocks = scale_blocks(l.k);
    in[0] = {l.x.data, extent(l.rows, l.x.ld, l.k, a->x_scales ? 1 : 2)};
    in[1] = {l.w, weights_extent(&l, a->w_scales ? 1 : 2)};
    in[2] = {a->x_scales, l.rows * blocks * 4};
    in[3] = {a->w_scales, (uint64_t)l.groups * halves * scale_blocks(a->l.n) * blocks * 4};
    in[4] = {l.offsets, (uint64_t)(l.groups + 1) * 4};
    in[5] = {l.bias, (uint64_t)l.groups * l.n * 2};
}

// -------------------------------------------------------------- forward products --

// What a forward product is to do: of 16- or 8-bit operands, gated or not.
struct Forward {
    GemmPlan plan;
    int splits, slots;
    bool pack_x, pack_w;
    uint64_t parts, tiles, x_bytes, w_bytes;    // of scratch memory
    uint64_t bytes() const { return parts + tiles + x_bytes + w_bytes; }
};

// Parts of the contraction, `most` of them, that fill the device.
static int parts_of(uint64_t blocks, uint64_t most) {
    int s = 1;
    while (s < 16 && blocks * s * 2 <= kSlots && (uint64_t)s * 2 <= most) s *= 2;
    return s;
}

// Few rows of 8-bit operands (of up to 64, `n` columns of both halves): microseconds on weights in
// no cache.  One row goes as dots.  Up to 16 the one-pass form, 16 columns a workgroup where it
// has them (4 x 8192 x 8192 17.6, with 32 columns 21.0; 16 x 4096 x 4096 8.8 and 10.4; 2 x 4096 x
// 8191 24 and 42; but 16 x 4112 x 8192 21.4 and 18.0), but of more than 8 by large weights 64 x
// 64 tiles, deep, and parts of the contraction to fill the device (16 x 8192 x 8192 18.9 against
// 21).  Up to 32 the one-pass form for weights under 48 MB (32 x 4096 x 4096 11.1, tiles 12.3; 32 x
// 8192 x 8192 30 and 20.3), 16 columns a workgroup where that gives no compute unit a second one
// (32 x 4096 x 4096 11.0, with 32 columns 12.7, 17 x 2064 x 2048 5.7 and 9.2; but 32 x 4112 x 2048
// 9.8 and 8.1, 32 x 6144 x 4096 18.2 and 13.3) and rows are short (17 and 32 x 4096 x 8192 14.5 and
// 15.7, 18.5 and 17.8; at any byte 32 x 4096 x 1023 8.7 and 10.7, x 4095 26.5 and 22.5); and tiles
// beyond (48 x 4096 x 4096 12.7, one pass 17; 64 x 8192 x 8192 21 and 40).  Rows of many groups,
// where the weights' read is all: to 16 a group, 8 of uneven ones, of which some have more and read
// their weights twice, the one pass (32 groups of 2 x 2048 x 4096, 256 uneven rows 124, tiles 126;
// 512 uneven ones 174 and 126, equal ones 117 and 122), then deep tiles (with two stages 137).  Of
// groups whose rows are whole words (`words`), which the one pass takes without knowing where pieces
// begin, always the tiles (32 groups of 2 x 2048 x 4088, 64, 128 and 256 uneven rows 86, 101 and 112,
// one pass 108, 127 and 155).
// `direct`: operands whose rows are whole words; the tiles copy others first.
static void choose_few(const rr_linear8_t* a, uint64_t halves, bool direct, bool words, Forward& f) {
    const rr_linear_t& l = a->l;
    const uint64_t n = l.n * halves, steps = ceil_div(l.k, kBlock), mean = ceil_div(l.rows, l.groups);
    const bool one = l.groups == 1 && !l.offsets, large = direct && n * l.k >= 48u << 20;
    GemmPlan& p = f.plan;
    const auto parts = [&](uint64_t blocks, uint64_t most) { f.splits = one ? parts_of(blocks, most) : 1; };
    p.narrow = p.deep = 0;
    f.slots = 0;
    if (one && l.rows == 1) {
        p.tile = kDot;
        f.splits = 1;
    } else if (!(words && !one) && mean <= (one || !l.offsets ? 16 : 8) && !(one && halves == 1 && mean > 8 && large)) {
        p.tile = kStream16;
        p.narrow = halves == 1 && one;
        parts(ceil_div(n, p.narrow ? 16 : 32), ceil_div(n, 32) <= 32 && !p.narrow ? l.k / 512 : 1);
    } else if (one && mean <= 32 && !large) {
        p.tile = kStream32;
        p.narrow = halves == 1 && ceil_div(n, 16) <= kSlots && l.k <= (direct && !words ? 4096 : 1024);
        parts(ceil_div(n, p.narrow ? 16 : 32), l.k / 512);
    } else {
        p.tile = kTile64;
        p.deep = 1;
        parts(ceil_div(n, 64), steps >= 16 ? steps / 4 : 1);
    }
}

static Forward forward_of(const rr_linear8_t* a, uint64_t halves) {
    const bool eight = a->x_scales != nullptr;
    rr_linear_t l = a->l;
    l.n *= halves;
    // a byte's tiles are as deep as 16-bit ones of half as many values, and take as long
    const uint64_t piece = eight ? 16 : 8;
    const rr_rows_t w = {const_cast<void*>(l.w), l.w_ld};
    const uint64_t apart = l.groups > 1 ? l.w_stride : 0;
    const bool good_x = good_rows(l.x, 0, l.k, piece), good_w = good_rows(w, apart, l.k, piece);
    const bool word_x = word_rows(l.x, 0, l.k, eight ? 1 : 2), word_w = word_rows(w, apart, l.k, eight ? 1 : 2);
    if (eight) {
        l.k = ceil_div(l.k, 2);
        l.x.ld = l.w_ld = ceil_div(l.k, 8) * 8;
        l.w_stride = 0;
        if (good_x && good_w) l.x.data = nullptr, l.w = nullptr;
    }
    Forward f = {};
    f.plan = choose(&l, kForward, &f.splits, &f.slots);
    f.plan.form = kForward;
    const uint64_t mean = ceil_div(l.rows, l.groups);
    const bool words = word_x && word_w && !(good_x && good_w);
    if (eight && mean <= 64) {
        choose_few(a, halves, word_x && word_w, words, f);
    } else if (halves == 2) {
        f.plan.narrow = 0;
        // as choose_few says of many groups (512 uneven rows over 32 of 2 x 2048 x 4096 in 16 bits 213 us,
        // 32 rows a pass 255; 256 rows 229, the one pass 193), and of rows of whole words that the
        // other forms take in single elements or from copies (5 .. 64 x 2 x 4000 x 7996 24 .. 28 us, so
        // 60 .. 75; 2 x 500 x 996 8.2 .. 8.6 and 9.7 .. 20; 2 x 1000 x 3996 9.2 .. 11.6 and 9.8 .. 24; 64
        // uneven rows over 32 groups of 2 x 2048 x 4094 168 and 378)
        if (mean <= 64 && ((l.groups > 1 && mean > (l.offsets ? 12 : 16)) || (words && (mean > 4 || l.groups > 1)))) {
            const uint64_t steps = ceil_div(l.k, (uint64_t)kDepth);
            f.plan.tile = kTile64;
            f.plan.deep = 1;
            f.splits = l.groups == 1 && !l.offsets ? parts_of(ceil_div(l.n, 64), steps >= 16 ? steps / 4 : 1) : 1;
            f.slots = 0;
        }
    }
    f.plan.direct = good_x && good_w;
    // the one-pass form takes 8-bit rows at any byte, but of no less than a piece
    if (eight && !f.plan.direct && a->l.k < 16 && f.plan.tile >= kStream16) f.plan.tile = kTile64, f.splits = 1;
    if (f.plan.tile == kStream16 && !eight && !f.plan.direct && l.groups == 1 && !l.offsets && l.rows <= 4)
        f.plan.tile = kDot;
    if (f.plan.tile == kDot) f.splits = 1;
    if (f.splits > 1) f.parts = ceil_div((uint64_t)f.splits * l.rows * l.n * sizeof(float), 256) * 256;
    f.tiles = (uint64_t)f.slots * 256 * 256 * sizeof(float);
    if (f.plan.tile < kStream16) {
        const uint64_t e = eight ? 1 : 2, row = ceil_div(a->l.k, piece) * piece * e;
        f.pack_x = f.plan.tile == kInner64 ? !good_x : !word_x;
        f.pack_w = f.plan.tile == kInner64 ? !good_w : !word_w;
        if (f.pack_x) f.x_bytes = ceil_div(l.rows * row, 256) * 256;
        if (f.pack_w) f.w_bytes = ceil_div((uint64_t)l.groups * l.n * row, 256) * 256;
    }
    return f;
}

static rr_status_t run_forward(const rr_linear8_t* a, uint64_t halves, void* workspace, hipStream_t s) {
    const bool eight = a->x_scales != nullptr;
    const Forward f = forward_of(a, halves);
    const rr_linear_t& l = a->l;
    const uint64_t ti = row_tiles(&l, tile_rows(f.plan.tile));
    const uint64_t cols = f.plan.cols() / halves, tj = ceil_div(l.n, cols);
    if (ti * tj == 0) return RR_OK;
    if (ti * tj * f.splits > (1u << 23) - 1) return RR_ERR_UNSUPPORTED;
    if (f.splits > 1 && ceil_div(l.rows * ceil_div(l.n, 4), 256) > (1u << 24) - 1) return RR_ERR_UNSUPPORTED;
    GemmArgs k = groups_of(&l);
    k.i = (int32_t)l.rows;
    k.j = (int32_t)l.n;
    k.c = (int32_t)l.k;
    k.tiles_i = (int32_t)ti;
    k.tiles_j = (int32_t)tj;
    k.splits = f.splits;
    k.part_stride = l.rows * l.n * halves;
    if (f.splits > 1 || f.slots) k.part = (float*)workspace;
    k.slots = f.slots;
    k.bias = l.bias;
    k.residual = l.residual.data;
    k.residual_ld = l.residual.ld;
    if (a->z_scales) {
        k.z8 = (uint8_t*)l.z.data;
        k.z8_ld = l.z.ld;
        k.z8_scale = a->z_scales;
    } else {
        k.z = l.z.data;
        k.z_ld = l.z.ld;
    }
    k.out = l.out.data;
    k.out_ld = l.out.ld;
    k.act = l.act;
    // copies of operands whose rows the tiles do not take
    const uint64_t e = eight ? 1 : 2, piece = 16 / e, row = ceil_div(l.k, piece) * piece;
    char* room = (char*)workspace + f.parts + f.tiles;
    k.p = l.x.data;
    k.p_ld = l.x.ld;
    k.q = l.w;
    k.q_ld = l.w_ld;
    k.q_group = l.groups > 1 ? l.w_stride : 0;
    Pack8Args copies = {};
    int n = 0;
    for (int o = 0; o < 2; ++o) {
        if (!(o ? f.pack_w : f.pack_x)) continue;
        // a 16-bit row is copied as the bytes it is
        BlockArgs& b = copies.part[n++];
        b.narrow = (uint8_t*)const_cast<void*>(o ? l.w : l.x.data);
        b.narrow_ld = (o ? l.w_ld : l.x.ld) * e;
        b.narrow_group = o && l.groups > 1 ? l.w_stride * e : 0;
        b.rows = o ? l.n * halves : l.rows;
        b.groups = o ? (uint64_t)l.groups : 1;
        b.width = (int32_t)(l.k * e);
        b.filled = (int32_t)(row * e);
        b.wide = room;
        if (o) {
            k.q = room;
            k.q_ld = row;
            k.q_group = b.rows * row;
        } else {
            k.p = room;
            k.p_ld = row;
        }
        room += o ? f.w_bytes : f.x_bytes;
    }
    if (n) {
        const rr_status_t st = launch_pack8(copies, n, s);
        if (st != RR_OK) return st;
    }
    k.q_half = k.q_ld * l.n;
    k.p_scale = a->x_scales;
    k.q_scale = a->w_scales;
    k.blocks = (int32_t)scale_blocks(l.k);
    k.q_rows = (int32_t)scale_blocks(l.n);
    if (eight && f.plan.tile < kStream16) {     // two bytes for one 16-bit value
        k.c = (int32_t)ceil_div(l.k, 2);
        k.p_ld /= 2;
        k.q_ld /= 2;
        k.q_half /= 2;
        k.q_group /= 2;
    }
    k.steps = (int32_t)ceil_div(k.c, kDepth);
    const bool b16 = l.dt == RR_BF16;
    if (eight && halves == 2) return b16 ? launch_gated8_bf16(k, f.plan, s) : launch_gated8_f16(k, f.plan, s);
    if (eight) return b16 ? launch_gemm8_bf16(k, f.plan, s) : launch_gemm8_f16(k, f.plan, s);
    return b16 ? launch_gated_bf16(k, f.plan, s) : launch_gated_f16(k, f.plan, s);
}

static rr_status_t check_forward(const rr_linear8_t* a, uint64_t halves) {
    const rr_status_t st = check_operands(a, halves);
    if (st != RR_OK) return st;
    const bool x8 = a->x_scales, w8 = a->w_scales;
    return x8 != w8 || (halves == 1 && !x8) ? RR_ERR_INVALID : RR_OK;
}

// z in 16 bits, where its 8-bit form is made from: 256 x 256 tiles have whole blocks of it.
static uint64_t z_room(const rr_linear8_t* a, const Forward& f) {
    const bool apart = a->z_scales && (f.plan.tile != kTile256 || f.splits > 1);
    return apart ? ceil_div(a->l.rows * a->l.n * 2 * 2, 256) * 256 : 0;
}

static rr_status_t forward(const rr_linear8_t* a, uint64_t halves, void* workspace, size_t workspace_bytes, hipStream_t s) {
    const rr_status_t st = check_forward(a, halves);
    if (st != RR_OK) return st;
    const rr_linear_t& l = a->l;
    const Forward f = forward_of(a, halves);
    const uint64_t own = z_room(a, f), need = f.bytes() + own;
    if (need && (!workspace || !aligned_to(workspace, 16) || workspace_bytes < need)) return RR_ERR_INVALID;
    if (!rows_ok(l.out, l.rows, l.n, 2) || !rows_ok_if(l.residual, l.rows, l.n, 2) || !aligned_to(l.bias, 2))
        return RR_ERR_INVALID;
    if (l.out.ld > kMaxLd || (l.residual.data && l.residual.ld > kMaxLd)) return RR_ERR_UNSUPPORTED;
    Span in[kInputs];
    inputs_of(a, halves, in);
    const uint64_t n_out = extent(l.rows, l.out.ld, l.n, 2), n_res = extent(l.rows, l.residual.ld, l.n, 2);
    const Span out[] = {{l.out.data, n_out},
                        {l.z.data, extent(l.rows, l.z.ld, l.n * halves, a->z_scales ? 1 : 2)},
                        {a->z_scales, l.rows * 2 * scale_blocks(l.n) * 4},
                        {workspace, need}};
    if (any_overlap(in, kInputs, out, 4)) return RR_ERR_INVALID;
    const bool same = l.residual.data == l.out.data && l.residual.ld == l.out.ld;
    for (int o = same ? 1 : 0; o < 4; ++o)
        if (overlap(l.residual.data, n_res, out[o].p, out[o].n)) return RR_ERR_INVALID;
    if (l.rows == 0) return RR_OK;
    if (!own) return run_forward(a, halves, workspace, s);
    rr_linear8_t b = *a;
    b.l.z = {workspace, l.n * 2};
    b.z_scales = nullptr;
    const rr_status_t done = run_forward(&b, halves, (char*)workspace + own, s);
    if (done != RR_OK) return done;
    // each half of a row as a row of its own; z's rows may be further apart
    rr_quantize_t q = {};
    q.dt = l.dt;
    q.width = l.n;
    q.groups = 1;
    if (l.z.ld == l.n * 2) {
        q.rows = l.rows * 2;
        q.x = {workspace, l.n};
        q.q = {l.z.data, l.n};
    } else {
        q.groups = l.rows;
        q.rows = 2;
        q.x = {workspace, l.n};
        q.q = {l.z.data, l.n};
        q.x_stride = l.n * 2;
        q.q_stride = l.z.ld;
    }
    q.scales = a->z_scales;
    return block_quantize(&q, s);
}

// ------------------------------------------------------------------ gradients --

static Operand x_of(const rr_linear8_t* a) {
    Operand o = rows_of(&a->l, a->l.x, a->l.k);
    o.scales = a->x_scales;
    o.part = a->l.rows;
    return o;
}
static Operand w_of(const rr_linear8_t* a, uint64_t halves) {
    rr_linear_t l = a->l;
    l.n *= halves;
    Operand o = weights_of(&l);
    o.scales = a->w_scales;
    o.high = kBlock;
    o.part = a->l.n;
    return o;
}

struct Wanted {
    rr_rows_t dout, dx, out;
    void* dw;
    float* db;
    int32_t dw_dt;
};

struct GradPlan {
    uint64_t dz, part, product;
    uint64_t bytes() const { return dz + part + product; }
};
static Operand dz_of(const rr_linear_t& both, void* at) {
    const uint64_t ld = ceil_div(both.n, 8) * 8;
    return rows_of(&both, {at, ld}, ld);
}
static GradPlan grad_plan(const rr_linear8_t* a, const Wanted& g) {
    GradPlan p = {};
    const rr_linear_t both = both_halves(a);
    const Operand dz = dz_of(both, nullptr);
    if (g.dx.data || g.dw) p.dz = dz.copy_bytes();
    const uint64_t splits = sum_splits(&a->l);
    if (g.db && splits > 1) p.part = ceil_div((uint64_t)a->l.groups * splits * both.n * sizeof(float), 256) * 256;
    if (g.dx.data) p.product = product_bytes(&both, kByX, dz, w_of(a, 2));
    if (g.dw) {
        const uint64_t bytes = product_bytes(&both, kByW, dz, x_of(a));
        if (bytes > p.product) p.product = bytes;
    }
    return p;
}

static rr_status_t check_gate(const rr_linear8_t* a, const rr_gated_grad_t* g) {
    const rr_status_t st = check_operands(a, 2);
    if (st != RR_OK) return st;
    if (!g || g->reserved) return RR_ERR_INVALID;
    const rr_linear_t& l = a->l;
    if (g->dw_dt != l.dt && g->dw_dt != RR_FP32) return RR_ERR_INVALID;
    const bool grads = g->dx.data || g->dw || g->db;
    if (!rows_ok(l.z, l.rows, l.n * 2, a->z_scales ? 1 : 2)) return RR_ERR_INVALID;
    if (grads ? !rows_ok(g->dout, l.rows, l.n, 2) : !rows_ok_if(g->dout, l.rows, l.n, 2)) return RR_ERR_INVALID;
    if (!rows_ok_if(g->dx, l.rows, l.k, 2) || !rows_ok_if(g->out, l.rows, l.n, 2)) return RR_ERR_INVALID;
    if (!aligned_to(g->dw, type_bytes(g->dw_dt)) || !aligned_to(g->db, 4)) return RR_ERR_INVALID;
    if ((g->dout.data && g->dout.ld > kMaxLd) || (g->dx.data && g->dx.ld > kMaxLd) || (g->out.data && g->out.ld > kMaxLd))
        return RR_ERR_UNSUPPORTED;
    return RR_OK;
}

static rr_status_t gated_backward(const rr_linear8_t* a, const rr_gated_grad_t* g, void* workspace, size_t workspace_bytes,
                                  hipStream_t s) {
    rr_status_t st = check_gate(a, g);
    if (st != RR_OK) return st;
    const rr_linear_t& l = a->l;
    const rr_linear_t both = both_halves(a);
    const Wanted want = {g->dout, g->dx, g->out, g->dw, g->db, g->dw_dt};
    const GradPlan plan = grad_plan(a, want);
    const uint64_t need = plan.bytes();
    if (need && (!workspace || !aligned_to(workspace, 16) || workspace_bytes < need)) return RR_ERR_INVALID;
    Span in[kInputs + 3];
    Span (&first)[kInputs] = *reinterpret_cast<Span(*)[kInputs]>(in);
    inputs_of(a, 2, first);
    in[5] = {nullptr, 0};                       // the bias is not read
    in[6] = {g->dout.data, extent(l.rows, g->dout.ld, l.n, 2)};
    in[7] = {l.z.data, extent(l.rows, l.z.ld, l.n * 2, a->z_scales ? 1 : 2)};
    in[8] = {a->z_scales, l.rows * 2 * scale_blocks(l.n) * 4};
    const Span out[] = {{g->dx.data, extent(l.rows, g->dx.ld, l.k, 2)},
                        {g->dw, (uint64_t)l.groups * both.n * l.k * type_bytes(g->dw_dt)},
                        {g->db, (uint64_t)l.groups * both.n * 4},
                        {g->out.data, extent(l.rows, g->out.ld, l.n, 2)},
                        {workspace, need}};
    if (any_overlap(in, kInputs + 3, out, 5)) return RR_ERR_INVALID;
    const Operand dz = dz_of(both, workspace);
    void* const room = (char*)workspace + plan.dz + plan.part;
    if (plan.dz || g->db || g->out.data) {
        GateArgs k = {};
        k.g = groups_of(&l);
        k.dout = g->dout.data;
        k.dout_ld = g->dout.ld;
        k.z = l.z.data;
        k.z_ld = l.z.ld;
        k.z_scale = a->z_scales;
        k.blocks = (int32_t)scale_blocks(l.n);
        if (plan.dz) {
            k.dz = workspace;
            k.dz_ld = dz.rows.ld;
        }
        k.out = g->out.data;
        k.out_ld = g->out.ld;
        k.n = (int32_t)l.n;
        k.act = l.act;
        k.splits = (int32_t)sum_splits(&l);
        k.threads = (int32_t)sum_threads(&l);
        if (g->db) k.part = plan.part ? (float*)((char*)workspace + plan.dz) : g->db;
        // of the rows of no group, out is cleared
        const unsigned ranges = (unsigned)l.groups + (l.offsets && g->out.data ? 2 : 0);
        const dim3 grid((unsigned)ceil_div(l.n, (uint64_t)k.threads * 8), (unsigned)k.splits, ranges);
        const bool b16 = l.dt == RR_BF16;
        if (a->z_scales) b16 ? launch_gate<bf16, true>(k, grid, s) : launch_gate<f16, true>(k, grid, s);
        else b16 ? launch_gate<bf16, false>(k, grid, s) : launch_gate<f16, false>(k, grid, s);
        if ((st = launched()) != RR_OK) return st;
        if (plan.part && (st = launch_sums(k.part, k.splits, both.n, l.groups, g->db, s)) != RR_OK) return st;
    }
    if (g->dx.data && l.rows) {
        Product r = {kByX, dz, w_of(a, 2), groups_of(&both)};
        r.k.i = (int32_t)l.rows;
        r.k.j = (int32_t)l.k;
        r.k.c = (int32_t)both.n;
        r.k.out = g->dx.data;
        r.k.out_ld = g->dx.ld;
        if ((st = run_product(&both, r, room, s)) != RR_OK) return st;
    }
    if (g->dw) {
        Product r = {kByW, dz, x_of(a), groups_of(&both)};
        r.k.i = (int32_t)both.n;
        r.k.j = (int32_t)l.k;
        r.k.out = g->dw;
        r.k.out_ld = l.k;
        r.k.out_group = both.n * l.k;
        r.k.wide_out = g->dw_dt == RR_FP32;
        if ((st = run_product(&both, r, room, s)) != RR_OK) return st;
    }
    return RR_OK;
}

}  // namespace blk

using namespace blk;

extern "C" {

rr_status_t block_linear8_workspace(const rr_linear8_t* a, size_t* bytes) {
    if (!bytes) return RR_ERR_INVALID;
    const rr_status_t st = check_forward(a, 1);
    if (st != RR_OK) return st;
    *bytes = forward_of(a, 1).bytes();
    return RR_OK;
}

rr_status_t block_linear8(const rr_linear8_t* a, void* workspace, size_t workspace_bytes, rr_stream_t stream) {
    return forward(a, 1, workspace, workspace_bytes, (hipStream_t)stream);
}

rr_status_t block_gated_workspace(const rr_linear8_t* a, size_t* bytes) {
    if (!bytes) return RR_ERR_INVALID;
    const rr_status_t st = check_forward(a, 2);
    if (st != RR_OK) return st;
    const Forward f = forward_of(a, 2);
    *bytes = f.bytes() + z_room(a, f);
    return RR_OK;
}

rr_status_t block_gated(const rr_linear8_t* a, void* workspace, size_t workspace_bytes, rr_stream_t stream) {
    return forward(a, 2, workspace, workspace_bytes, (hipStream_t)stream);
}

rr_status_t block_gated_backward_workspace(const rr_linear8_t* a, const rr_gated_grad_t* g, size_t* bytes) {
    if (!bytes) return RR_ERR_INVALID;
    const rr_status_t st = check_gate(a, g);
    if (st != RR_OK) return st;
    *bytes = grad_plan(a, {g->dout, g->dx, g->out, g->dw, g->db, g->dw_dt}).bytes();
    return RR_OK;
}

rr_status_t block_gated_backward(const rr_linear8_t* a, const rr_gated_grad_t* g, void* workspace, size_t workspace_bytes,
                                 rr_stream_t stream) {
    return gated_backward(a, g, workspace, workspace_bytes, (hipStream_t)stream);
}

}  // extern "C"
