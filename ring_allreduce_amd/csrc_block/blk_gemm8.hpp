// blk_gemm8.hpp -- products of 8-bit operands (e4m3) with a scale for each block of 128:
// block_linear8's, and block_gated's of such operands.
//
//   out[i][j] = sum over blocks b of sx(i, b) sw(j / 128, b) sum over c in b of x8(i, c) w8(j, c)
//
// The inner sums are the matrix instruction's own, 16 x 16 x 128: one block of the contraction
// each.  The products of both scales come on top on the vector units, a multiply-add a
// result, in 32 bits.
//
// The instruction is exact to 32 bits but for one thing: before it adds eight neighbouring
// products it aligns them, and cuts each at 2^-13 of the power of two of the largest.  (As
// measured: beside 2^16, 2^3 and above is kept, 2^2 lost; 8 bits further on all is kept.  The
// older 16 x 16 x 32 instruction does the same.)  Of 128 products of normal values that is an
// error of 2^-16.2 of the result at the root of the mean square, where e4m3 operands are 2^-5 off
// what they stand for and a bf16 result 2^-9.  Products without it are those of the values as
// bf16, at half the rate.
#pragma once

#include "blk_gemm.hpp"

namespace blk {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// 16 rows of Q by 16 of P, 128 deep, from nothing.  A lane's 32 bytes are 32 of a row's 128, the
// same ones of both operands; which ones does not matter to the sum.
__device__ __forceinline__ f32x4 mma8(u32x4 q0, u32x4 q1, u32x4 p0, u32x4 p1) {
    const i32x8 q = {(int)q0[0], (int)q0[1], (int)q0[2], (int)q0[3], (int)q1[0], (int)q1[1], (int)q1[2], (int)q1[3]};
    const i32x8 p = {(int)p0[0], (int)p0[1], (int)p0[2], (int)p0[3], (int)p1[0], (int)p1[1], (int)p1[2], (int)p1[3]};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(q, p, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

// ------------------------------------------------------------------- the tiles --
//
// The tiles of the 16-bit products, with two 8-bit values in the place of one of 16: a tile is
// 128 bytes deep, one block.  The scales of four blocks at a time go to LDS beside the
// operands: 16 bytes of a row for each of P's rows, and of up to two blocks of Q's.
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
            const int b = s.j0 / 128, r = GATED ? lane * a.q_rows + b : b + lane;
            at = lane < 2 && (GATED ? b < a.q_rows : r < a.q_rows) ? (uint32_t)(GATED ? lane * a.q_rows : lane) * line : kReach;
            const uint64_t each = (uint64_t)a.q_rows * (GATED ? 2 : 1), group = s.g.group > 0 ? s.g.group : 0;
            base = a.q_scale + (group * each + b) * a.blocks;
            bytes = (each - b) * line;
        }
        const uint64_t p = (uint64_t)uniform((const char*)base);
        rsrc = u32x4{(uint32_t)p, (uint32_t)(p >> 32) & 0xFFFF,
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)(bytes < kReach ? (uint32_t)bytes : kReach)), 0x00027000};
    }
    // blocks b .. b + 3 into place `which`
    __device__ __forceinline__ void load(int b, int which) const {
        if (mine)
            Direct<uint16_t, false, 64, 256, false>::issue(rsrc, at == kReach ? kReach : at + (uint32_t)b * 4, to + which * kBytes);
    }
};

template <typename T, int TI, int TJ, int WI, int WJ, int STAGES, bool GATED>
__global__ void __launch_bounds__(64 * WI * WJ, STAGES * (TI + TJ) * kDepth * 2 > 81920 && WI * WJ == 4 ? 1 : 2)
gemm8_kernel(const GemmArgs a) {
    constexpr int THREADS = 64 * WI * WJ, FI = TI / WI / 16, FJ = TJ / WJ / 16;
    constexpr int PB = Tile<false, TI>::kBytes, QB = Tile<false, TJ>::kBytes;
    constexpr uint32_t PLACES = STAGES * (PB + QB), ALL = PLACES + 2 * Scales<TI>::kBytes;
    constexpr uint32_t OUT = 2 * 16 * WI * (TJ + 4) * 4;   // write_out's place
    __shared__ __align__(PB) char lds[OUT > ALL ? OUT : ALL];
    BLK_LDS char* const room = (BLK_LDS char*)lds;
    const RowTiles rows = count_tiles(a, TI);
    Spot s;
    if (!find_spot<true, TI, GATED ? TJ / 2 : TJ>(a, rows, blockIdx.x, s)) return;
    const uint16_t* const p = (const uint16_t*)a.p;
    const uint16_t* const q = (const uint16_t*)a.q + (s.g.group > 0 ? (uint64_t)s.g.group * a.q_group : 0);
    const int wave = threadIdx.x >> 6, tiles = (s.c_end - s.c0 + kDepth - 1) / kDepth;
    const int wi = wave / WJ * (TI / WI), wj = wave % WJ * (TJ / WJ);
    Reader<false, TI> rp;
    Reader<false, TJ> rq;
    const uint32_t p_at = (uint32_t)(uintptr_t)room, q_at = p_at + STAGES * PB, s_at = p_at + PLACES;
    rp.start(p_at, wi);
    rq.start(q_at, wj);
    f32x4 acc[FI][FJ];
#pragma unroll
    for (int x = 0; x < FI; ++x)
#pragma unroll
        for (int y = 0; y < FJ; ++y) acc[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    typedef Direct<uint16_t, false, TI, THREADS, false> DP;
    typedef std::conditional_t<GATED, Twin<uint16_t, false, TJ, THREADS, false>, Direct<uint16_t, false, TJ, THREADS, false>> DQ;
    constexpr int PIECES = DP::kPieces + DQ::kPieces;
    DP lp;
    DQ lq;
    Scales<TI> ls;
    lp.start(p, a.p_ld, s.i0, s.i_end, s.c0, s.c_end);
    if constexpr (GATED) lq.start(q, a.q_half, a.q_ld, s.j0, a.j, s.c0, s.c_end);
    else lq.start(q, a.q_ld, s.j0, a.j, s.c0, s.c_end);
    ls.template start<GATED>(a, s, s_at);
    const int first = s.c0 / kDepth;         // block of the first tile
    const auto fetch = [&](int place) {
        lp.aim(p_at + place * PB);
        lq.aim(q_at + place * QB);
#pragma unroll
        for (int k = 0; k < DP::kPieces; ++k) lp.piece(k);
#pragma unroll
        for (int k = 0; k < DQ::kPieces; ++k) lq.piece(k);
    };
    if (tiles > 0) {
        ls.load(first, 0);
#pragma unroll
        for (int t = 0; t < STAGES - 1; ++t) fetch(t);
    }
    // of this lane's rows, and of the wave's columns
    const uint32_t sp_at = s_at + (wi + (threadIdx.x & 15)) * 16;
    const uint32_t sq_at = s_at + TI * 16 + (GATED ? wj / (TJ / 2) : wj / 128) * 16;
    int now = 0, next = STAGES - 1;
    for (int t = 0; t < tiles; ++t) {
        arrived<PIECES * (STAGES - 2)>();
        if ((t & 3) == 0) ls.load(first + t + 4, (t >> 2 & 1) ^ 1);
        fetch(next);
        next = next == STAGES - 1 ? 0 : next + 1;
        const uint32_t at = (t >> 2 & 1) * Scales<TI>::kBytes + (t & 3) * 4;
        u32x4 fq[FJ][2];
#pragma unroll
        for (int y = 0; y < FJ; ++y)
#pragma unroll
            for (int h = 0; h < 2; ++h) fq[y][h] = rq.template fragment<u32x4>(y, h);
        const float sq = *(const BLK_LDS float*)(uintptr_t)(sq_at + at);
#pragma unroll
        for (int x = 0; x < FI; ++x) {
            const u32x4 p0 = rp.template fragment<u32x4>(x, 0), p1 = rp.template fragment<u32x4>(x, 1);
            const float f = sq * *(const BLK_LDS float*)(uintptr_t)(sp_at + at + x * 256);
#pragma unroll
            for (int y = 0; y < FJ; ++y) {
                const f32x4 sum = mma8(fq[y][0], fq[y][1], p0, p1);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[x][y][e] = fmaf(f, sum[e], acc[x][y][e]);
            }
        }
        const uint32_t by_p = now == STAGES - 1 ? -(STAGES - 1) * PB : PB, by_q = now == STAGES - 1 ? -(STAGES - 1) * QB : QB;
        now = now == STAGES - 1 ? 0 : now + 1;
        rp.move(by_p);
        rq.move(by_q);
    }
    arrived<0>();                            // the loads past the end as well
    if constexpr (GATED) write_gated<T, TI, TJ, WI, WJ, FI, FJ>(a, s, room, acc);
    else write_out<T, true, TI, TJ, WI, WJ, FI, FJ>(a, s, room, acc);
}

// ------------------------------------------------------------ few rows: one pass --
//
// As the one-pass form of the 16-bit products: a wave's part is 256 deep, two blocks.
constexpr int kStreamDepth8 = 256;

template <typename T, int FI, int FJ, bool DIRECT, bool GATED>
__global__ void __launch_bounds__(64 * kStreamWaves) stream8_kernel(const GemmArgs a) {
    __shared__ f32x4 sums[kStreamWaves][FI * FJ][64];
    Range g;
    if (!find_tile(a, count_tiles(a, 16 * FI), (int)blockIdx.y, 16 * FI, g)) return;
    g.group = __builtin_amdgcn_readfirstlane(g.group);
    const int i0 = __builtin_amdgcn_readfirstlane(g.lo), i_end = __builtin_amdgcn_readfirstlane(g.hi);
    constexpr int HALVES = GATED ? 2 : 1, EACH = FJ / HALVES;
    const int j0 = (int)blockIdx.x * (16 * EACH), lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    int c_lo = 0, c_end = g.group < 0 ? 0 : a.c;
    if (a.splits > 1) {
        const int each = ((a.c + kStreamDepth8 - 1) / kStreamDepth8 + a.splits - 1) / a.splits * kStreamDepth8;
        c_lo = (int)min((int64_t)blockIdx.z * each, (int64_t)c_end);
        c_end = (int)min((int64_t)c_lo + each, (int64_t)c_end);
    }
    Strip<uint8_t, FI, DIRECT> sp;
    Strip<uint8_t, EACH, DIRECT> sq[HALVES];
    sp.start((const uint8_t*)a.p, a.p_ld, i0, i_end, c_end);
    const uint64_t group = g.group > 0 ? (uint64_t)g.group : 0;
    const float* q_scale[HALVES];
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
        sq[h].start((const uint8_t*)a.q + group * a.q_group + h * a.q_half, a.q_ld, j0, a.j, c_end);
        q_scale[h] = a.q_scale + ((group * HALVES + h) * a.q_rows + j0 / 128) * a.blocks;
    }
    const float* p_scale[FI];
#pragma unroll
    for (int x = 0; x < FI; ++x) p_scale[x] = a.p_scale + (uint64_t)max(min(i0 + x * 16 + (lane & 15), i_end - 1), 0) * a.blocks;
    f32x4 acc[FI][FJ];
#pragma unroll
    for (int x = 0; x < FI; ++x)
#pragma unroll
        for (int y = 0; y < FJ; ++y) acc[x][y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    struct Part {
        u32x4 p[4][FI], q[HALVES][4][EACH];
        float ps[2][FI], qs[2][HALVES];
    };
    const auto load = [&](Part& to, int c) {
#pragma unroll
        for (int h = 0; h < HALVES; ++h) sq[h].load(to.q[h], c);
        sp.load(to.p, c);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int block = min(c / 128 + b, a.blocks - 1);
#pragma unroll
            for (int x = 0; x < FI; ++x) to.ps[b][x] = p_scale[x][block];
#pragma unroll
            for (int h = 0; h < HALVES; ++h) to.qs[b][h] = q_scale[h][block];
        }
    };
    Part now, next;
    int c = c_lo + wave * kStreamDepth8;
    if (c < c_end) load(now, c);
    while (c < c_end) {
        c += kStreamWaves * kStreamDepth8;
        if (c < c_end) load(next, c);
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int x = 0; x < FI; ++x)
#pragma unroll
                for (int y = 0; y < FJ; ++y) {
                    const u32x4 (&q)[4][EACH] = now.q[y / EACH];
                    const f32x4 sum = mma8(q[b * 2][y % EACH], q[b * 2 + 1][y % EACH], now.p[b * 2][x], now.p[b * 2 + 1][x]);
                    const float f = now.ps[b][x] * now.qs[b][y / EACH];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[x][y][e] = fmaf(f, sum[e], acc[x][y][e]);
                }
        now = next;
    }
#pragma unroll
    for (int x = 0; x < FI; ++x)
#pragma unroll
        for (int y = 0; y < FJ; ++y) sums[wave][x * FJ + y][lane] = acc[x][y];
    __syncthreads();
    if constexpr (GATED) finish_stream<T, FI>(a, g.group, i0, i_end, j0, wave, sums);
    else finish_stream_plain<T, FI, FJ>(a, g.group, i0, i_end, j0, wave, sums);
}

// -------------------------------------------------------------------- launching --

template <typename T, int TI, int TJ, int WI, int WJ, int STAGES, bool GATED>
static void launch_tile8(const GemmArgs& a, hipStream_t s) {
    const unsigned grid = (unsigned)a.tiles_i * a.tiles_j * a.splits;
    gemm8_kernel<T, TI, TJ, WI, WJ, STAGES, GATED><<<grid + (unsigned)a.slots, 64 * WI * WJ, 0, s>>>(a);
}
template <typename T, int FI, bool GATED> static void launch_stream8(const GemmArgs& a, const GemmPlan& p, hipStream_t s) {
    const dim3 grid((unsigned)a.tiles_j, (unsigned)a.tiles_i, (unsigned)a.splits);
    const int threads = 64 * kStreamWaves;
    if constexpr (!GATED)
        if (p.narrow) {
            if (p.direct) stream8_kernel<T, FI, 1, true, false><<<grid, threads, 0, s>>>(a);
            else stream8_kernel<T, FI, 1, false, false><<<grid, threads, 0, s>>>(a);
            return;
        }
    if (p.direct) stream8_kernel<T, FI, 2, true, GATED><<<grid, threads, 0, s>>>(a);
    else stream8_kernel<T, FI, 2, false, GATED><<<grid, threads, 0, s>>>(a);
}

template <typename T, bool GATED> static rr_status_t launch_gemm8(const GemmArgs& a, const GemmPlan& p, hipStream_t s) {
    switch (p.tile) {
        case kStream16: launch_stream8<T, 1, GATED>(a, p, s); break;
        case kStream32: launch_stream8<T, 2, GATED>(a, p, s); break;
        case kStream64: launch_stream8<T, 4, GATED>(a, p, s); break;
        case kTile256:
            launch_tile8<T, 256, 256, 2, 4, 2, GATED>(a, s);
            if constexpr (!GATED)
                if (a.slots) join_last_kernel<T, true, 256, 256><<<dim3((unsigned)a.slots / 2, 8), 256, 0, s>>>(a);
            break;
        case kTile128:
            if (p.deep) launch_tile8<T, 128, 128, 2, 2, 4, GATED>(a, s);
            else launch_tile8<T, 128, 128, 2, 2, 2, GATED>(a, s);
            break;
        default:
            if (p.deep) launch_tile8<T, 64, 64, 2, 2, 4, GATED>(a, s);
            else launch_tile8<T, 64, 64, 2, 2, 2, GATED>(a, s);
    }
    if constexpr (GATED) {
        return join_gated<T>(a, s);
    } else {
        const rr_status_t st = launched();
        if (st != RR_OK || a.splits == 1) return st;
        join_kernel<T><<<(unsigned)ceil_div((uint64_t)a.rows * ceil_div(a.j, 4), 256), 256, 0, s>>>(a, 1);
        return launched();
    }
}

}  // namespace blk
