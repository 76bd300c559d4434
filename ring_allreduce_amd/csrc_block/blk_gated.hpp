// blk_gated.hpp -- the launches of block_gated's forward product.
#pragma once

#include "blk_tile.hpp"

namespace blk {

// Adds the parts of the last round's tiles: 32 rows a workgroup, 8 columns of out a thread.
template <typename T, int TI, int TJ> __global__ void __launch_bounds__(256) join_last_gated_kernel(const GemmArgs a) {
    const RowTiles rows = count_tiles(a, TI);
    const unsigned tiles = (unsigned)rows.total * (unsigned)a.tiles_j;
    const unsigned whole = tiles / (unsigned)a.slots * (unsigned)a.slots, rest = tiles - whole;
    if (blockIdx.x >= rest || last_round_parts(rest, (unsigned)a.slots, a.steps) < 2) return;
    Spot s;
    if (!find_spot<true, TI, TJ / 2>(a, rows, whole + blockIdx.x, s)) return;
    constexpr int GROUPS = TJ / 16;
    const int col = (int)threadIdx.x % GROUPS * 8, j = s.j0 + col;
    if (j >= a.j && !a.z8) return;           // with z in 8 bits the row's threads stay together
    const Some<T, 8> g_bias = gated_bias_of<T, 8>(a, s.g.group, 0, j), u_bias = gated_bias_of<T, 8>(a, s.g.group, 1, j);
    for (int row = (int)(blockIdx.y * 32 + threadIdx.x / GROUPS), k = 0; k < 32; k += 256 / GROUPS, row += 256 / GROUPS) {
        const int i = s.i0 + row;
        if (i >= s.i_end) return;
        float v[2][8] = {};
        if (s.g.group >= 0)
            for (int p = 0; p < s.parts; ++p) {
                const float* from = a.part + ((uint64_t)s.tile * s.parts + p) * (TI * TJ) + row * TJ + col;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const f32x4 lo = *(const f32x4*)(from + h * (TJ / 2)), hi = *(const f32x4*)(from + h * (TJ / 2) + 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[h][e] += lo[e];
                        v[h][4 + e] += hi[e];
                    }
                }
            }
        if (a.z8) {                          // 16 threads have the row's block
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float r[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[h][e] = s.g.group < 0 ? 0.0f : v[h][e] + (float)(h ? u_bias : g_bias).e[e];
                    r[e] = j + e < a.j ? (float)(T)v[h][e] : 0.0f;
                }
                float size = largest_of(r);
#pragma unroll
                for (int d = 8; d > 0; d >>= 1) size = fmaxf(size, __shfl_xor(size, d));
                const float scale = scale_of(size);
                if (col == 0) a.z8_scale[((uint64_t)i * 2 + h) * a.q_rows + s.j0 / 128] = scale;
                if (j < a.j) store_eight(a.z8 + (uint64_t)i * a.z8_ld + (uint64_t)h * a.j + j, a.j - j, narrow(r, inverse_of(scale)));
            }
            act_values(a.act, v[0]);
            times(v[0], v[1]);
            if (j < a.j) store_some<T, 8>((T*)a.out + (uint64_t)i * a.out_ld + j, a.j - j, v[0]);
            continue;
        }
        finish_gated<T, 8>(a, s.g.group, a.j - j, v[0], v[1], g_bias, u_bias, (T*)a.z + (uint64_t)i * a.z_ld + j,
                           (T*)a.out + (uint64_t)i * a.out_ld + j);
    }
}

// Of 8-bit or 16-bit operands, in 256 x 256 tiles.
template <typename T, bool EIGHT> static void launch_gated_large(const GemmArgs& a, hipStream_t s) {
    launch_tile<T, EIGHT, 256, 256, 2, 4, 2, true>(a, s);
    if (a.slots) join_last_gated_kernel<T, 256, 256><<<dim3((unsigned)a.slots / 2, 8), 256, 0, s>>>(a);
}
template <typename T, int FI> static void launch_gated_stream(const GemmArgs& a, const GemmPlan& p, hipStream_t s) {
    const dim3 grid((unsigned)a.tiles_j, (unsigned)a.tiles_i, (unsigned)a.splits);
    if (p.direct) stream_kernel<T, FI, 2, true, true><<<grid, 64 * kStreamWaves, 0, s>>>(a);
    else stream_kernel<T, FI, 2, false, true><<<grid, 64 * kStreamWaves, 0, s>>>(a);
}
template <typename T> static rr_status_t join_gated(const GemmArgs& a, hipStream_t s) {
    const rr_status_t st = launched();
    if (st != RR_OK || a.splits == 1) return st;
    join_gated_kernel<T><<<(unsigned)ceil_div((uint64_t)a.rows * ceil_div(a.j, 4), 256), 256, 0, s>>>(a);
    return launched();
}
template <typename T> static rr_status_t launch_gated(const GemmArgs& a, const GemmPlan& p, hipStream_t s) {
    switch (p.tile) {
        case kDot:
            if (a.rows == 1) launch_dot<T, 1, 2, true>(a, s);
            else if (a.rows == 2) launch_dot<T, 2, 2, true>(a, s);
            else if (a.rows == 3) launch_dot<T, 3, 2, true>(a, s);
            else launch_dot<T, 4, 2, true>(a, s);
            break;
        case kStream16: launch_gated_stream<T, 1>(a, p, s); break;
        case kStream32: launch_gated_stream<T, 2>(a, p, s); break;
        case kStream64: launch_gated_stream<T, 4>(a, p, s); break;
        case kInner64:
            gemm_kernel<T, false, false, true, 64, 32, 2, 1, 3, 4, true>
                <<<(unsigned)a.tiles_i * a.tiles_j * a.splits, 512, 0, s>>>(a);
            break;
        case kTile256: launch_gated_large<T, false>(a, s); break;
        case kTile128:
            if (p.deep) launch_tile<T, false, 128, 128, 2, 4, 4, true>(a, s);
            else launch_tile<T, false, 128, 128, 2, 2, 2, true>(a, s);
            break;
        default:
            if (p.deep) launch_tile<T, false, 64, 64, 2, 2, 4, true>(a, s);
            else launch_tile<T, false, 64, 64, 2, 2, 2, true>(a, s);
    }
    return join_gated<T>(a, s);
}

}  // namespace blk
