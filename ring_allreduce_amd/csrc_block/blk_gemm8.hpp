// blk_gemm8.hpp -- products of 8-bit operands (e4m3) with a scale for each block of 128:
// block_linear8's, and block_gated's of such operands.
//
//   out[i][j] = sum over blocks b of sx(i, b) sw(j / 128, b) sum over c in b of x8(i, c) w8(j, c)
//
// The inner sums are the matrix instruction's own, 16 x 16 x 128: one block of the contraction
// each; what it rounds, and both ways that the scales come on top, stand in blk_tile.hpp with
// the tiles.  Here: few rows, and the launches.
#pragma once

#include "blk_gated.hpp"

namespace blk {

// ------------------------------------------------------------ few rows: one pass --
//
// As the one-pass form of the 16-bit products: a wave's part is 256 deep, two blocks, and their
// scales, any fp32 ones, come on top on the vector units.  Bound by the read of the weights
// and, of few columns, by its start: 16 x 4096 x 4096 8.4 us (2.0 TB/s), 3 x 8192 x 8192 17.2
// (3.9 TB/s), 32 x 4096 x 4096 11.1; 256 uneven rows over 32 groups of 2 x 2048 x 4096, gated, 124
// (4.3 TB/s).  Of up to 16 rows two workgroups a compute unit, which leaves a lane 128 registers:
// rows at any byte with 32 columns (or 16 of each projection) keep 9 to 11 more in scratch memory.
// With one workgroup and nothing there groups take longer and single products less (256 uneven rows
// over 32 groups of 2 x 2048 x 4095 338 us instead of 325, plain 168 and 166; 16 x 2 x 4096 x 4095 25
// instead of 27).
constexpr int kStreamDepth8 = 256;

template <typename T, int FI, int FJ, bool DIRECT, bool GATED>
__global__ void __launch_bounds__(64 * kStreamWaves, FI == 1 ? 4 : 1) stream8_kernel(const GemmArgs a) {
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
            // (a part that ends after its first block has no second one: zeros, times zero)
            const int block = min(c / 128 + b, a.blocks - 1);
            const bool there = c / 128 + b < a.blocks;
#pragma unroll
            for (int x = 0; x < FI; ++x) to.ps[b][x] = there ? p_scale[x][block] : 0.0f;
#pragma unroll
            for (int h = 0; h < HALVES; ++h) to.qs[b][h] = there ? q_scale[h][block] : 0.0f;
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
                    const f32x4 sum = mma8(frag_of(q[b * 2][y % EACH], q[b * 2 + 1][y % EACH]), frag_of(now.p[b * 2][x], now.p[b * 2 + 1][x]));
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

// ------------------------------------------------------------------ one row: dots --
//
// As the dots of 16-bit rows: a wave goes along one row of the weights, or two, 1 KiB of each at a
// time, in memory's own order and at any alignment.  A lane's 16 values are in one block, whose
// scales come on top of their sum; everything in 32 bits.  8192 x 8192 weights that are in no
// cache take 16.1 us (4.2 TB/s), 4096 x 4096 6.1; two rows of x would take 20.7, which the one-pass
// form does in 17.
template <typename T, int R, bool GATED>
__global__ void __launch_bounds__(64 * kDotWaves) dot8_kernel(const GemmArgs a) {
    const int lane = threadIdx.x & 63;
    const int j0 = ((int)blockIdx.x * kDotWaves + (int)(threadIdx.x >> 6)) * (GATED ? 1 : R);
    if (j0 >= a.j) return;
    const uint8_t *const x = (const uint8_t*)a.p, *w[R];
    const float *const sx = a.p_scale, *sw[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int j = GATED ? j0 : min(j0 + r, a.j - 1);
        w[r] = (const uint8_t*)a.q + (GATED ? r * a.q_half : 0) + (uint64_t)j * a.q_ld;
        sw[r] = a.q_scale + ((uint64_t)(GATED ? r * a.q_rows : 0) + j / 128) * a.blocks;
    }
    float sum[R] = {};
    struct Part {
        u32x4 x, w[R];
        float sx, sw[R];
    };
    const auto load = [&](Part& to, int c) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            to.w[r] = load_raw(w[r] + c);
            to.sw[r] = sw[r][c / 128];
        }
        to.x = load_raw(x + c);
        to.sx = sx[c / 128];
    };
    const auto wide = [](u32x4 v, float (&to)[16]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[k], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[k], true);
            to[k * 4] = lo[0], to[k * 4 + 1] = lo[1], to[k * 4 + 2] = hi[0], to[k * 4 + 3] = hi[1];
        }
    };
    const auto add = [&](const Part& in) {
        float f[16];
        wide(in.x, f);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float v[16], part = 0.0f;
            wide(in.w[r], v);
#pragma unroll
            for (int e = 0; e < 16; ++e) part = fmaf(f[e], v[e], part);
            sum[r] = fmaf(in.sx * in.sw[r], part, sum[r]);
        }
    };
    constexpr int STEP = 64 * 16, AHEAD = 4;
    int c = 0;
    for (; c + AHEAD * STEP <= a.c; c += AHEAD * STEP) {
        Part in[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) load(in[u], c + u * STEP + lane * 16);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) add(in[u]);
    }
    const int whole = a.c / 16 * 16;
    for (c += lane * 16; c < whole; c += STEP) {
        Part in;
        load(in, c);
        add(in);
    }
    if (whole + lane < a.c) {
        const int at = whole + lane;
        const auto one = [](uint8_t v) { return __builtin_amdgcn_cvt_f32_fp8((int)v, 0); };
#pragma unroll
        for (int r = 0; r < R; ++r) sum[r] = fmaf(sx[at / 128] * sw[r][at / 128], one(x[at]) * one(w[r][at]), sum[r]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) sum[r] = lane_sum<64>(sum[r]);
    if constexpr (GATED) {
        float g[1] = {sum[0]}, u[1] = {sum[1]};
        if (lane == 0) finish_gated<T, 1>(a, 0, 0, j0, g, u);
    } else {
        float v[1] = {sum[0]};
#pragma unroll
        for (int r = 1; r < R; ++r) v[0] = lane == r ? sum[r] : v[0];
        if (lane < R && j0 + lane < a.j) finish<T, 1>(a, 0, 0, j0 + lane, v);
    }
}

// -------------------------------------------------------------------- launching --

template <typename T, int R, bool GATED> static void launch_dot8(const GemmArgs& a, hipStream_t s) {
    const unsigned grid = (unsigned)ceil_div(a.j, (uint64_t)(GATED ? 1 : R) * kDotWaves);
    dot8_kernel<T, R, GATED><<<grid, 64 * kDotWaves, 0, s>>>(a);
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
        case kDot:
            // two rows of the weights a wave where that leaves no compute unit empty
            if (GATED || a.j >= 2048) launch_dot8<T, 2, GATED>(a, s);
            else launch_dot8<T, GATED ? 2 : 1, GATED>(a, s);
            break;
        case kStream16: launch_stream8<T, 1, GATED>(a, p, s); break;
        case kStream32: launch_stream8<T, 2, GATED>(a, p, s); break;
        case kTile256:
            if constexpr (GATED) launch_gated_large<T, true>(a, s);
            else launch_tile<T, true, 256, 256, 2, 4, 2, false>(a, s);
            if constexpr (!GATED)
                if (a.slots) join_last_kernel<T, true, 256, 256><<<dim3((unsigned)a.slots / 2, 8), 256, 0, s>>>(a);
            break;
        case kTile128:
            if (p.deep) launch_tile<T, true, 128, 128, 2, 4, 4, GATED>(a, s);
            else launch_tile<T, true, 128, 128, 2, 2, 2, GATED>(a, s);
            break;
        default:
            if (p.deep) launch_tile<T, true, 64, 64, 2, 2, 4, GATED>(a, s);
            else launch_tile<T, true, 64, 64, 2, 2, 2, GATED>(a, s);
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
