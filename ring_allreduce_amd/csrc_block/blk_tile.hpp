// blk_tile.hpp -- the tiles of block_linear8's and block_gated's forward products, and the 8-bit
// matrix instructions.
//
// The 16 x 16 x 128 instruction takes one block of the contraction.  It is exact to 32 bits but
// for one thing: before it adds eight neighbouring products it aligns them, and cuts each at
// 2^-13 of the power of two of the largest.  (As measured: beside 2^16, 2^3 and above is kept,
// 2^2 lost; 8 bits further on all is kept.  The older 16 x 16 x 32 instruction does the same.)  Of
// 128 products of normal values that is an error of 2^-16.2 of the result at the root of the mean
// square, where e4m3 operands are 2^-5 off what they stand for and a bf16 result 2^-9.  Products
// without it are those of the values as bf16, at half the rate.
#pragma once

#include "blk_gemm.hpp"

namespace blk {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// A lane's 32 bytes of a row's 128: the same ones of both operands; which ones matters to the sum
// only by the eights that are neighbours.
typedef i32x8 Frag;
__device__ __forceinline__ Frag frag_of(u32x4 lo, u32x4 hi) {
    return __builtin_bit_cast(Frag, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}
// 16 rows of Q by 16 of P, 128 deep, from nothing.
__device__ __forceinline__ f32x4 mma8(const Frag& q, const Frag& p) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q, p, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}
// The same, times 2^(sq + sp - 254) of the lane's row of either operand, on top of c.
__device__ __forceinline__ f32x4 mma8_scaled(const Frag& q, const Frag& p, f32x4 c, uint32_t sq, uint32_t sp) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q, p, c, 0, 0, 0, (int)sq, 0, (int)sp);
}
// 0 if four scales are powers of two that the instruction takes: its exponent in 8 bits, 2^-127 and
// NaN (0 and 255) not among them.
__device__ __forceinline__ uint32_t not_power(u32x4 scales) {
    uint32_t bad = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) bad |= (scales[k] & 0x807FFFFF) | (scales[k] - 0x00800000 < 0x7F000000 ? 0 : 1);
    return bad;
}
__device__ __forceinline__ uint32_t exponent_of(float scale) { return __builtin_bit_cast(uint32_t, scale) >> 23; }

// ------------------------------------------------------------------- the tiles --
//
// The tiles of the 16-bit products, with two 8-bit values in the place of one of 16: a tile is
// 128 bytes deep, one block.  The scales of four blocks at a time go to LDS beside the
// operands: 16 bytes of a row for each of P's rows, and of up to two blocks of Q's.

__device__ __forceinline__ u32x4 descriptor(const void* base, uint64_t bytes) {
    const uint64_t p = (uint64_t)uniform((const char*)base);
    return u32x4{(uint32_t)p, (uint32_t)(p >> 32) & 0xFFFF,
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)(bytes < kReach ? (uint32_t)bytes : kReach)), 0x00027000};
}
__device__ __forceinline__ void load_to_lds(u32x4 rsrc, uint32_t offset, uint32_t to) {
    Direct<uint16_t, false, 64, 256, false>::issue(rsrc, offset, to);
}

// Rows of an operand into the places of tiles, as Direct does it, in fewer registers: what a
// lane loads next is THREADS / 8 rows on, so one offset serves them all, and the descriptor ends
// with the last row.  (Whether an offset is in its range goes by the lane's part alone, which is
// why the steps are in it.)
template <int ROWS, int THREADS> struct Load8 {
    static constexpr int kPieces = ROWS * 8 / THREADS;
    u32x4 rsrc;
    uint32_t stride;
    // r0, r_end: rows; end: bytes of a row, up to which all pieces are whole (part of one in range
    // would come as zeros); ld: bytes
    __device__ __forceinline__ void start(const char* b, uint64_t ld, int r0, int r_end, int end) {
        const int rows = max(min(r_end - r0, ROWS), 0);
        rsrc = descriptor(b + (uint64_t)r0 * ld, rows ? (uint64_t)(rows - 1) * ld + end : 0);
        stride = (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)ld * (THREADS / 8)));
    }
    __device__ __forceinline__ void piece(int k, uint32_t at, uint32_t tile) const {
        load_to_lds(rsrc, at + k * stride, tile + k * THREADS * 16);
    }
};
// A thread's first byte: of row thread / 8, the 16-byte pieces permuted by the row.
__device__ __forceinline__ int piece_of() {
    const int thread = here();
    return (thread & 7) ^ (thread >> 3 & 7);
}

// Which of Q's rows in the tile fragment y of a wave takes, so that a lane's results of two
// fragments (16 rows of Q each, of which it gets four) are 8 neighbouring columns of out, and
// those of the four lanes of a row 32: the results leave from the registers, in whole pieces of
// 64 bytes a row.  Of a gated product the first half of the fragments are rows of the gate and the
// second the same ones of the other projection.  Where a half is one fragment, a lane has four
// columns.
template <int TJ, int WJ, int FJ, bool GATED> struct Columns {
    static constexpr int HALVES = GATED ? 2 : 1, N = FJ / HALVES > 1 ? 8 : 4, GROUPS = FJ * 4 / HALVES / N;
    static constexpr int WIDE = TJ / WJ / HALVES;      // a wave's columns of out
    // the first row of fragment y, and the one in it of lane r (0 .. 15)
    static constexpr int row(int y) {
        const int in = y % (FJ / HALVES);
        return y / (FJ / HALVES) * (TJ / 2) + (N == 8 ? (in >> 1) * 32 + (in & 1) * 4 : 0);
    }
    __device__ __forceinline__ static int row_in(int r) { return N == 8 ? (r >> 2) * 8 + (r & 3) : r; }
    // by which the 16-byte pieces of a row are permuted: another for each of 8 lanes
    __device__ __forceinline__ static int mix(int row) { return N == 8 ? (row & 3) | (row >> 1 & 4) : row & 7; }
};

// Of a gated 256 x 256 tile, whose 128 columns of either half are a block of z: the largest
// magnitudes of z, rounded to T, in the blocks' rows, by the waves and then all of them through
// LDS; scales, z in 8 bits, and out.
template <typename T, int TI, int WI, int WJ, int FI, int FJ>
__device__ __forceinline__ void write_eight(const GemmArgs& a, const Spot& s, BLK_LDS char* room, const f32x4 (&acc)[FI][FJ]) {
    static_assert(WJ * 32 == 128 && FJ == 4, "the columns of a block");
    const int thread = here(), lane = thread & 63, wave = thread >> 6;
    const int row = wave / WJ * (TI / WI) + (lane & 15), part = wave % WJ;
    const int j = s.j0 + part * 32 + (lane >> 4) * 8, n = a.j - j, i0 = s.i0 + row;
    const Some<T, 8> bias[2] = {gated_bias_of<T, 8>(a, s.g.group, 0, j), gated_bias_of<T, 8>(a, s.g.group, 1, j)};
    BLK_LDS float* const sizes = (BLK_LDS float*)room;         // [half][part][row]
    const auto z_of = [&](int x, int h, float (&v)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = s.g.group < 0 ? 0.0f : acc[x][h * 2 + e / 4][e % 4] + (float)bias[h].e[e];
    };
#pragma unroll
    for (int x = 0; x < FI; ++x)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
            z_of(x, h, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)(T)v[e];
            float size = largest_of(v);
            size = fmaxf(size, __shfl_xor(size, 16));
            size = fmaxf(size, __shfl_xor(size, 32));
            if (lane < 16) sizes[(h * WJ + part) * TI + row + x * 16] = size;
        }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < FI; ++x) {
        const int i = i0 + x * 16;
        if (i >= s.i_end) continue;
        float v[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float size = 0.0f;
#pragma unroll
            for (int w = 0; w < WJ; ++w) size = fmaxf(size, sizes[(h * WJ + w) * TI + row + x * 16]);
            const float scale = scale_of(size);
            if (part == 0 && lane < 16) a.z8_scale[((uint64_t)i * 2 + h) * a.q_rows + s.j0 / 128] = scale;
            float r[8];
            z_of(x, h, v[h]);
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = (float)(T)v[h][e];
            if (n > 0) store_eight(a.z8 + (uint64_t)i * a.z8_ld + (uint64_t)h * a.j + j, n, narrow(r, inverse_of(scale)));
        }
        act_values(a.act, v[0]);
        times(v[0], v[1]);
        if (n > 0) store_some<T, 8>((T*)a.out + (uint64_t)i * a.out_ld + j, n, v[0]);
    }
}

// The results, from the registers: no LDS and no barrier, so that a wave that is done with its
// products writes while others multiply (8192 x 8192 x 2048 through LDS 169 us, so 159, before
// other steps).  Of parts of the contraction, sums in 32 bits.
template <typename T, int TI, int TJ, int WI, int WJ, int FI, int FJ, bool GATED>
__device__ __forceinline__ void write_direct(const GemmArgs& a, const Spot& s, BLK_LDS char* room, const f32x4 (&acc)[FI][FJ]) {
    typedef Columns<TJ, WJ, FJ, GATED> C;
    constexpr int N = C::N, GROUPS = C::GROUPS, HALVES = C::HALVES;
    if constexpr (GATED && TI == 256)
        if (a.z8 && s.parts == 1) {
            write_eight<T, TI, WI, WJ, FI, FJ>(a, s, room, acc);
            return;
        }
    const bool whole = a.splits == 1 && s.parts == 1, add = !GATED && whole && a.residual && s.g.group >= 0;
    if (!whole && s.g.group < 0) return;        // the kernels that join the parts know
    const int thread = here(), lane = thread & 63, wave = thread >> 6;
    const int j0 = s.j0 + wave % WJ * C::WIDE + (lane >> 4) * N, i0 = s.i0 + wave / WJ * (TI / WI) + (lane & 15);
    Some<T, N> bias[HALVES][GROUPS];
#pragma unroll
    for (int c = 0; c < GROUPS; ++c)
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            if constexpr (GATED) bias[h][c] = whole ? gated_bias_of<T, N>(a, s.g.group, h, j0 + c * 32) : Some<T, N>{};
            else bias[h][c] = whole ? bias_of<T, N>(a, s.g.group, j0 + c * 32) : Some<T, N>{};
        }
    // The rows of block row 0 by 32-bit offsets from the tile's corner, and 16 rows on for each
    // block row (rows are at most 2^22 elements apart).
    const uint64_t part_ld = s.parts > 1 ? (uint64_t)TJ : (uint64_t)a.j * HALVES;
    const uint64_t out_ld = whole ? a.out_ld : part_ld;
    const uint32_t wide = whole ? sizeof(T) : 4;
    const char* out = whole ? (const char*)((const T*)a.out + (uint64_t)s.i0 * a.out_ld + s.j0)
                      : s.parts > 1 ? (const char*)(a.part + ((uint64_t)s.tile * s.parts + s.split) * (TI * TJ))
                                    : (const char*)(a.part + (uint64_t)s.split * a.part_stride + (uint64_t)s.i0 * part_ld + s.j0);
    const char* z = (const char*)((const T*)a.z + (uint64_t)s.i0 * a.z_ld + s.j0);
    const char* res = (const char*)((const T*)a.residual + (uint64_t)s.i0 * a.residual_ld + s.j0);
    out = uniform(out);
    z = uniform(z);
    res = uniform(res);
    const uint32_t row = (uint32_t)(i0 - s.i0), col = (uint32_t)(j0 - s.j0);
    const uint32_t at_out = (row * (uint32_t)out_ld + col) * wide;
    const uint32_t at_z = (row * (uint32_t)a.z_ld + col) * (uint32_t)sizeof(T);
    const uint32_t at_res = (row * (uint32_t)a.residual_ld + col) * (uint32_t)sizeof(T);
    const int left = s.i_end - i0;           // rows from the lane's first one
    const auto rows = [&](auto inside_) {
        constexpr bool INSIDE = decltype(inside_)::value;
        Some<T, N> residual[GROUPS] = {}, later[GROUPS] = {};
        const auto fetch = [&](Some<T, N> (&to)[GROUPS], int x) {
#pragma unroll
            for (int c = 0; c < GROUPS; ++c)
                if (x * 16 < left && (INSIDE || j0 + c * 32 < a.j))
                    to[c] = load_some<T, N>((const T*)(res + at_res) + (uint64_t)(x * 16) * a.residual_ld + c * 32,
                                            INSIDE ? N : a.j - j0 - c * 32);
        };
        if (add) fetch(residual, 0);
#pragma unroll
        for (int x = 0; x < FI; ++x) {
            if (add && x + 1 < FI) fetch(later, x + 1);
            const uint64_t down = (uint64_t)(x * 16);
            if (x * 16 < left)
#pragma unroll
                for (int c = 0; c < GROUPS; ++c) {
                    const int n = INSIDE ? N : a.j - j0 - c * 32;
                    if (!INSIDE && n <= 0) continue;
                    float v[HALVES][N];
#pragma unroll
                    for (int h = 0; h < HALVES; ++h)
#pragma unroll
                        for (int e = 0; e < N; ++e) v[h][e] = acc[x][h * (FJ / 2) + c * (N / 4) + e / 4][e % 4];
                    char* const to = (char*)out + down * out_ld * wide + at_out;
                    T* const to_z = (T*)(z + down * a.z_ld * sizeof(T) + at_z) + c * 32;
                    if (!whole) {
#pragma unroll
                        for (int h = 0; h < HALVES; ++h)
                            store_wide<N>((float*)to + c * 32 + h * (s.parts > 1 ? TJ / 2 : a.j), n, v[h]);
                    } else if constexpr (GATED) {
                        finish_gated<T, N>(a, s.g.group, n, v[0], v[1], bias[0][c], bias[1][c], to_z, (T*)to + c * 32);
                    } else {
                        finish<T, N>(a, s.g.group, n, v[0], bias[0][c], residual[c], to_z, (T*)to + c * 32);
                    }
                }
#pragma unroll
            for (int c = 0; c < GROUPS; ++c) residual[c] = later[c];
        }
    };
    if (s.j0 + TJ / HALVES <= a.j) rows(std::true_type());
    else rows(std::false_type());
}

// Reads what the epilogue will want of the residual into the L2, by way of 1 KiB of LDS that nobody
// looks at: one piece of each 128 bytes of the tile's rows, three steps before the end (8192 x
// 8192 x 4096 with bias, SiLU and a residual that is in no cache 263 us, without this 269, at scales
// that are no powers of two 286 and 297; 6 to 30 steps before the end are no better).  (A piece that begins before the
// first element or ends behind the last one is one of theirs: 16 bytes at a boundary of 16.)
template <typename T, int TI, int TJ, int THREADS>
__device__ __forceinline__ void touch_residual(const GemmArgs& a, const Spot& s, uint32_t room) {
    constexpr int LINES = TJ * (int)sizeof(T) / 128;
    const uint64_t ld = a.residual_ld * sizeof(T);
    const char* const from = (const char*)((const T*)a.residual + (uint64_t)s.i0 * a.residual_ld + s.j0);
    const uint32_t skew = (uint32_t)(uintptr_t)from & 15;
    const uint64_t end = (uint64_t)(min(s.i_end - s.i0, TI) - 1) * ld + (uint64_t)min(a.j - s.j0, TJ) * sizeof(T);
    const u32x4 rsrc = descriptor(from - skew, (skew + end + 15) / 16 * 16);
#pragma unroll
    for (int l = 0; l < TI * LINES; l += THREADS) {
        const uint32_t at = l + here();
        load_to_lds(rsrc, (at / LINES * (uint32_t)ld + at % LINES * 128 + skew) / 16 * 16, room);
    }
}

// The scales on their way to LDS: four neighbouring blocks of a row, 16 bytes, a lane.
template <int TI> struct Scales {
    static constexpr int kBytes = (TI + 64) * 16;    // a wave's load for Q's
    u32x4 rsrc;
    uint32_t at;                                     // this lane's row; kReach: none
    bool mine;                                       // whether this wave loads any
    uint32_t to;
    template <bool GATED> __device__ __forceinline__ void start(const GemmArgs& a, const Spot& s, uint32_t room) {
        const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), lane = threadIdx.x & 63;
        mine = wave <= TI / 64;
        to = room + wave * 1024;
        const uint32_t line = (uint32_t)a.blocks * 4;
        const float* base;
        uint64_t bytes;
        if (wave < TI / 64) {
            const int r = wave * 64 + lane;
            at = s.i0 + r < s.i_end ? (uint32_t)r * line : kReach;
            base = a.p_scale + (uint64_t)s.i0 * a.blocks;
            bytes = (uint64_t)(a.rows - s.i0) * line;
        } else {
            // of a gated product: of either half; of others the tile's columns have two at most
            const int b = s.j0 / 128;
            at = lane < 2 && (GATED || b + lane < a.q_rows) ? (uint32_t)(GATED ? lane * a.q_rows : lane) * line : kReach;
            const uint64_t each = (uint64_t)a.q_rows * (GATED ? 2 : 1), group = s.g.group > 0 ? s.g.group : 0;
            base = a.q_scale + (group * each + b) * a.blocks;
            bytes = (each - b) * line;
        }
        rsrc = descriptor(base, bytes);
    }
    // blocks b .. b + 3 into place `which`
    __device__ __forceinline__ void load(int b, int which) const {
        if (mine) load_to_lds(rsrc, at == kReach ? kReach : at + (uint32_t)b * 4, to + which * kBytes);
    }
};

// Every wave's reads of LDS are done.
__device__ __forceinline__ void all_read() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory"); }

// Nothing moves across: reads of LDS that are moved up take registers that there are none of.
__device__ __forceinline__ void keep_order() {
    asm volatile("" : : : "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// EIGHT: operands in 8 bits, with scales; else in T.
//
// Scales: where all of four blocks of a wave's rows and columns are powers of two, as
// block_quantize makes them, the instruction itself takes their exponents (8192 x 8192 x 8192 403
// us, 2730 TFLOP/s); others are multiplied in 32 bits and come on top of each block's sum by a
// multiply-add a result on the vector units, beside the matrix cores (459 us).  Both once the
// clocks have settled, after some 100 calls; the first ones after a pause take up to 100 more.
//
// Bound, at 256 x 256: 8-bit products by the way from the L2s into LDS and by the epilogue, which no
// product overlaps (one workgroup a compute unit, nearly all of its LDS): 8192 x 8192 x 4096 takes
// 224 us, with bias, SiLU and a residual from memory 263.  16-bit ones by power, as gemm_kernel;
// beside it these tiles keep Q's fragments in registers, so that a step reads 128 KiB of LDS
// instead of 192, and have no copy of Q's next tile (16384 rows over 8 uneven groups of 2 x
// 4096 x 2048 with z 548 us, gemm_kernel's tiles 591).
template <typename T, bool EIGHT, int TI, int TJ, int WI, int WJ, int STAGES, bool GATED>
__global__ void __launch_bounds__(64 * WI * WJ, 2) tile_kernel(const GemmArgs a) {
    constexpr int THREADS = 64 * WI * WJ, FI = TI / WI / 16, FJ = TJ / WJ / 16, HALVES = GATED ? 2 : 1;
    constexpr int PB = TI * 128, QB = TJ * 128;
    constexpr bool TOUCH = !GATED && TI == 256;
    constexpr uint32_t PLACES = STAGES * (PB + QB), SCALES = EIGHT ? 2 * Scales<TI>::kBytes : 0;
    constexpr uint32_t ALL = PLACES + SCALES + (TOUCH ? 1024 : 0);
    typedef Columns<TJ, WJ, FJ, GATED> C;
    __shared__ __align__(PB) char lds[ALL];
    BLK_LDS char* const room = (BLK_LDS char*)lds;
    const RowTiles rows = count_tiles(a, TI);
    Spot s;
    if (!find_spot<true, TI, TJ / HALVES>(a, rows, blockIdx.x, s)) return;
    const int wave = threadIdx.x >> 6;
    const int tiles = __builtin_amdgcn_readfirstlane((s.c_end - s.c0 + kDepth - 1) / kDepth);
    const int wi = wave / WJ * (TI / WI), wj = wave % WJ * C::WIDE;
    Reader<false, TI> rp;
    const uint32_t p_at = (uint32_t)(uintptr_t)room, q_at = p_at + STAGES * PB, s_at = p_at + PLACES;
    rp.start(p_at, wi);
    uint32_t rq[2];                          // the lane's row of fragment 0, both halves of its 128 bytes
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = wj + C::row_in(threadIdx.x & 15);
        rq[h] = q_at + row * 128 + (((threadIdx.x >> 4 & 3) + h * 4) ^ C::mix(row)) * 16;
    }
    f32x4 acc[FI][FJ];
#pragma unroll
    for (int x = 0; x < FI; ++x)
#pragma unroll
        for (int y = 0; y < FJ; ++y) acc[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // a, the sizes in it and the spot count pairs of values
    typedef Load8<TI, THREADS> DP;
    typedef Load8<TJ / HALVES, THREADS> DQ;
    constexpr int PIECES = DP::kPieces + HALVES * DQ::kPieces;
    DP lp;
    DQ lq[HALVES];
    Scales<TI> ls;
    const char* const q = (const char*)a.q + (s.g.group > 0 ? (uint64_t)s.g.group * a.q_group * 2 : 0);
    // Rows end with a whole piece or, of whole words, inside one, whose place takes the row's last
    // 16 bytes: some of them twice, once too often, until `clean` has made them zeros.  Other rows
    // are copies with zeros behind.
    const int bytes = s.c_end * 2, end = (bytes & 3) || bytes < 16 ? (bytes + 15) / 16 * 16 : bytes;
    const bool cut = tiles > 0 && (end & 15);
    lp.start((const char*)a.p, a.p_ld * 2, s.i0, s.i_end, end);
#pragma unroll
    for (int h = 0; h < HALVES; ++h) lq[h].start(q + h * a.q_half * 2, a.q_ld * 2, s.j0, a.j, end);
    if constexpr (EIGHT) ls.template start<GATED>(a, s, s_at);
    int left = end - s.c0 * 2;               // bytes of a row
    const int last = left - (tiles - 1) * 128;      // those of the last tile
    const int from = piece_of() * 16;        // of the 128
    const int from_q = ((here() & 7) ^ C::mix(here() >> 3)) * 16;
    uint32_t at_p = (uint32_t)(here() >> 3) * (uint32_t)(a.p_ld * 2) + from + s.c0 * 2;
    uint32_t at_q = (uint32_t)(here() >> 3) * (uint32_t)(a.q_ld * 2) + from_q + s.c0 * 2;
    const uint32_t mine = (uint32_t)__builtin_amdgcn_readfirstlane(wave * 1024);
    // before the loads of a tile: aim(); after its P's and Q's: 128 bytes on
    const auto aim = [&]() {
        at_p = from >= left ? kReach : at_p + min(left - from - 16, 0);
        at_q = from_q >= left ? kReach : at_q + min(left - from_q - 16, 0);
        left -= 128;
    };
    constexpr int QS = HALVES * DQ::kPieces, PS = DP::kPieces;
    const auto load_p = [&](uint32_t place, int k) { lp.piece(k, at_p, p_at + place * PB + mine); };
    const auto load_q = [&](uint32_t place, int k) {
        const int h = k / DQ::kPieces;
        lq[h].piece(k % DQ::kPieces, at_q, q_at + place * QB + h * (QB / 2) + mine);
    };
    const int first = s.c0 / kDepth;         // block of the first tile
    // of this lane's rows, and of the wave's columns
    const uint32_t sp_at = s_at + (wi + (threadIdx.x & 15)) * 16;
    const uint32_t sq_at = s_at + TI * 16 + (GATED ? 0 : wj / 128) * 16;
    // A tile's fragments of Q are in registers throughout, those of P one block row ahead.  So Q's
    // place is free early on: behind a barrier at block row MID the loads of the tile STAGES on
    // go into it, and P's behind one two block rows before the end, when the last of them are
    // read and the next tile has arrived.  (Both at once, in the second place, wait for each
    // other.)  The last two rows are multiplied column by column, and after each column the
    // next tile's fragment of Q takes the place of this one's.
    constexpr int MID = FI > 2 ? FI / 4 : 0, SPAN = FI > 2 ? FI - 2 - MID : 1;
    Frag fq[FJ], fp[FI > 4 ? 4 : FI * 2];
    float sq[HALVES], sp[FI], sq_next[HALVES], sp_next[FI];
    const auto read_p = [&](int slot, int x) {
        fp[slot] = frag_of(rp.template fragment<u32x4>(x, 0), rp.template fragment<u32x4>(x, 1));
    };
    const auto read_q = [&](int y) {
        u32x4 v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) v[h] = *(const BLK_LDS u32x4*)(uintptr_t)(rq[h] + C::row(y) * 128);
        fq[y] = frag_of(v[0], v[1]);
    };
    const auto read_scales = [&](int t) {
        const uint32_t at = (uint32_t)((t >> 2 & 1) * Scales<TI>::kBytes + (t & 3) * 4);
#pragma unroll
        for (int h = 0; h < HALVES; ++h) sq_next[h] = *(const BLK_LDS float*)(uintptr_t)(sq_at + at + h * 16);
#pragma unroll
        for (int x = 0; x < FI; ++x) sp_next[x] = *(const BLK_LDS float*)(uintptr_t)(sp_at + at + x * 256);
    };
    const auto use_scales = [&]() {
#pragma unroll
        for (int h = 0; h < HALVES; ++h) sq[h] = sq_next[h];
#pragma unroll
        for (int x = 0; x < FI; ++x) sp[x] = sp_next[x];
    };
    // Whether all scales of the four blocks from tile t on are powers of two: a lane looks at
    // every fourth of its rows.
    const auto powers = [&](int t) {
        const uint32_t at = (uint32_t)((t >> 2 & 1) * Scales<TI>::kBytes);
        const int lane = threadIdx.x & 63;
        uint32_t bad = 0;
#pragma unroll
        for (int h = 0; h < HALVES; ++h) bad |= not_power(*(const BLK_LDS u32x4*)(uintptr_t)(sq_at + at + h * 16));
#pragma unroll
        for (int x = 0; x < FI; x += 4) {
            const int block = (x + (lane >> 4)) % FI;
            const uint32_t not_this = not_power(*(const BLK_LDS u32x4*)(uintptr_t)(sp_at + at + block * 256));
            bad |= s.i0 + wi + block * 16 + (lane & 15) < s.i_end ? not_this : 0;
        }
        return __all(bad == 0);
    };
    constexpr int SLOTS = FI > 4 ? 4 : FI * 2, HELD = 3;
    int place = 0;
    // The last tile of rows that end inside a piece: the words of it that the piece before has too.
    const auto clean = [&](Frag& f) {
        const int piece = (int)(threadIdx.x >> 4 & 3);
#pragma unroll
        for (int w = 0; w < 8; ++w)
            if (w % 4 < 3) f[w] = piece + w / 4 * 4 == last >> 4 && w % 4 * 4 < 16 - (last & 15) ? 0 : f[w];
    };
    const auto tile = [&](auto power_, auto cut_, int t) {
        constexpr bool POWER = decltype(power_)::value, CUT = decltype(cut_)::value;
        if constexpr (CUT)
#pragma unroll
            for (int y = 0; y < FJ; ++y) clean(fq[y]);
        // Sums that are to be multiplied wait for HELD more products: what follows a product at once
        // would wait for it (8192 x 8192 x 8192 459 us instead of 473, 1024 x 4096 x 4096, where eight
        // waves hide it too, 26 either way; with two or four of them less).
        constexpr int LATER = FI * FJ > HELD ? HELD : 1;
        f32x4 held[LATER];
        const auto add_held = [&](int n) {          // of the tile's n-th product
            const int late = n - (FI - 2) * FJ, x = late < 0 ? n / FJ : FI - 2 + (late & 1), y = late < 0 ? n % FJ : late >> 1;
            const float f = sp[x] * sq[y / (FJ / HALVES)];
            acc[x][y] = __builtin_elementwise_fma(f32x4{f, f, f, f}, held[n % LATER], acc[x][y]);
        };
        const auto multiply = [&](int x, int y, float s) {
            const int half = y / (FJ / HALVES);
            if constexpr (!EIGHT) {
                typedef typename Mma<T>::V V;
                const Frag q = fq[y], p = fp[x % SLOTS];
                acc[x][y] = Mma<T>::run(__builtin_bit_cast(V, __builtin_shufflevector(q, q, 0, 1, 2, 3)),
                                        __builtin_bit_cast(V, __builtin_shufflevector(p, p, 0, 1, 2, 3)), acc[x][y]);
                acc[x][y] = Mma<T>::run(__builtin_bit_cast(V, __builtin_shufflevector(q, q, 4, 5, 6, 7)),
                                        __builtin_bit_cast(V, __builtin_shufflevector(p, p, 4, 5, 6, 7)), acc[x][y]);
            } else if constexpr (POWER) {
                acc[x][y] = mma8_scaled(fq[y], fp[x % SLOTS], acc[x][y], exponent_of(sq[half]), exponent_of(s));
            } else {
                const int n = x < FI - 2 ? x * FJ + y : (FI - 2) * FJ + y * 2 + x - (FI - 2);
                const f32x4 sum = mma8(fq[y], fp[x % SLOTS]);
                if (n >= LATER) add_held(n - LATER);
                held[n % LATER] = sum;
            }
        };
        // (no branches between the products: they are moved down behind them, and what they read
        // is held until then)
        if (EIGHT && (t & 3) == 0) ls.load(first + t + 4, (t >> 2 & 1) ^ 1);
        aim();
#pragma unroll
        for (int x = 0; x < FI - 2; ++x) {
            if (x == MID) all_read();
            if (x >= MID)
#pragma unroll
                for (int k = (x - MID) * QS / SPAN; k < (x - MID + 1) * QS / SPAN; ++k) load_q(place, k);
            read_p((x + 1) % SLOTS, x + 1);
            if (x == FI - 3) read_p((x + 2) % SLOTS, x + 2);
            if constexpr (CUT) clean(fp[x % SLOTS]);
#pragma unroll
            for (int y = 0; y < FJ; ++y) multiply(x, y, sp[x]);
            keep_order();
        }
        arrived<PIECES * (STAGES - 2) + (FI > 2 ? QS : 0)>();
        const int to = place;
        const bool wrap = place == STAGES - 1;
        rp.move(wrap ? -(STAGES - 1) * PB : PB);
        rq[0] += wrap ? -(STAGES - 1) * QB : QB;
        rq[1] += wrap ? -(STAGES - 1) * QB : QB;
        place = wrap ? 0 : place + 1;
        if constexpr (EIGHT) read_scales(t + 1);
        read_p(FI % SLOTS, 0);
        if constexpr (FI == 2) read_p(3, 1);
        if constexpr (CUT) {
            clean(fp[(FI - 2) % SLOTS]);
            clean(fp[(FI - 1) % SLOTS]);
        }
#pragma unroll
        for (int y = 0; y < FJ; ++y) {
            multiply(FI - 2, y, sp[FI - 2]);
            multiply(FI - 1, y, sp[FI - 1]);
#pragma unroll
            for (int k = y * PS / FJ; k < (y + 1) * PS / FJ; ++k) load_p(to, k);
            if (FI == 2)
#pragma unroll
                for (int k = y * QS / FJ; k < (y + 1) * QS / FJ; ++k) load_q(to, k);
            read_q(y);
            keep_order();
        }
        at_p += 128;
        at_q += 128;
        if constexpr (FI % SLOTS != 0) {
            fp[0] = fp[FI % SLOTS];
            if constexpr (FI == 2) fp[1] = fp[3];
        }
        if constexpr (EIGHT && !POWER)
#pragma unroll
            for (int n = FI * FJ - LATER; n < FI * FJ; ++n) add_held(n);
        if constexpr (EIGHT) use_scales();
    };
    if (tiles > 0) {
        if constexpr (EIGHT) ls.load(first, 0);
#pragma unroll
        for (int t = 0; t < STAGES; ++t) {
            aim();
#pragma unroll
            for (int k = 0; k < PS; ++k) load_p(t, k);
#pragma unroll
            for (int k = 0; k < QS; ++k) load_q(t, k);
            at_p += 128;
            at_q += 128;
        }
        arrived<PIECES * (STAGES - 1)>();
#pragma unroll
        for (int y = 0; y < FJ; ++y) read_q(y);
        read_p(0, 0);
        if constexpr (FI == 2) read_p(1, 1);
        if constexpr (EIGHT) {
            read_scales(0);
            use_scales();
        }
    }
    const int touch = TOUCH && a.residual && a.splits == 1 && s.parts == 1 ? max(tiles - 3, 0) : tiles;
    const auto ahead = [&](int t) {
        if constexpr (TOUCH)
            if (t == touch) touch_residual<T, TI, TJ, THREADS>(a, s, s_at + SCALES);
    };
    const int whole = cut ? tiles - 1 : tiles;
    int t = 0;
    if constexpr (EIGHT)                     // as long as all scales are powers of two, and the rest
        for (; t < whole && ((t & 3) != 0 || powers(t)); ++t) {
            ahead(t);
            tile(std::true_type(), std::false_type(), t);
        }
    for (; t < whole; ++t) {
        ahead(t);
        tile(std::false_type(), std::false_type(), t);
    }
    for (; t < tiles; ++t) {                 // once at most; as a loop nothing of it is moved down into the epilogue
        ahead(t);
        tile(std::false_type(), std::true_type(), t);
    }
    arrived<0>();                            // the loads past the end as well
    write_direct<T, TI, TJ, WI, WJ, FI, FJ, GATED>(a, s, room, acc);
}

// 128 x 128 with four stages, one workgroup a compute unit, is launched with eight waves: with four, one
// a SIMD, nothing hides a wave's waits, and the compiler keeps sums in registers that the vector
// units cannot reach (1024 x 4096 x 4096, four waves: gated in 16 bits 48 us, in 8 bits at scales that
// are no powers of two 42; so 36 and 29; at powers of two 26 and 27).
template <typename T, bool EIGHT, int TI, int TJ, int WI, int WJ, int STAGES, bool GATED>
static void launch_tile(const GemmArgs& a, hipStream_t s) {
    const unsigned grid = (unsigned)a.tiles_i * a.tiles_j * a.splits;
    tile_kernel<T, EIGHT, TI, TJ, WI, WJ, STAGES, GATED><<<grid + (unsigned)a.slots, 64 * WI * WJ, 0, s>>>(a);
}

}  // namespace blk
