// blk_quant.hip -- values to 8 bits with a scale for each block of 128, and back
// (block_quantize, block_dequantize).
//
// Bound by memory: e bytes in and 1 + 4 / 128 out a value, or the other way round.  16384 x 8192 in
// bf16, 407 MB: rows 77 us, 128 x 128 blocks 78, and back 80 (5.1 .. 5.3 TB/s; a copy of as many
// bytes takes 76).
#include "blk_product.hpp"

namespace blk {

typedef float f32x2 __attribute__((ext_vector_type(2)));

// The row of a piece, of `each` in a row; all matrices have less than 2^31 rows.
__device__ __forceinline__ uint64_t row_of(uint64_t piece, uint32_t each) {
    return piece >> 32 ? piece / each : (uint32_t)piece / each;
}

// 8 neighbouring columns in 32 bits.
template <typename T> struct Eight {
    static constexpr int RAWS = sizeof(T) / 2;
    u32x4 raw[RAWS];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int r = 0; r < RAWS; ++r) raw[r] = load_raw(p + r * Vec<T>::N);
    }
    __device__ __forceinline__ void load_some(const T* row, int at, int len) {
#pragma unroll
        for (int r = 0; r < RAWS; ++r)
            raw[r] = __builtin_bit_cast(u32x4, load_vec(row, at + r * Vec<T>::N, len));
    }
    __device__ __forceinline__ float value(int e) const {
        return (float)vec_of<T>(raw[e / Vec<T>::N]).e[e % Vec<T>::N];
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = value(e);
    }
    __device__ __forceinline__ float size() const {
        float v[8];
        values(v);
        return largest_of(v);
    }
    __device__ __forceinline__ u32x2 e4m3(float inverse) const {
        float v[8];
        values(v);
        return narrow(v, inverse);
    }
};

__device__ __forceinline__ float largest_of_16_lanes(float a) {
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) a = fmaxf(a, __shfl_xor(a, d));
    return a;
}

// 16 lanes a block of a row.
template <typename T> __global__ void __launch_bounds__(256) quantize_rows_kernel(const BlockArgs a) {
    const int lane = threadIdx.x & 15;
    const uint64_t all = a.groups * a.rows * (uint64_t)a.blocks;
    for (uint64_t id = (uint64_t)blockIdx.x * 16 + (threadIdx.x >> 4); id < all; id += (uint64_t)gridDim.x * 16) {
        const uint64_t line = row_of(id, (uint32_t)a.blocks);
        const int col = (int)(id - line * (uint32_t)a.blocks) * 128 + lane * 8;
        const uint64_t group = a.groups > 1 ? (uint32_t)line / (uint32_t)a.rows : 0, row = line - group * a.rows;
        const T* from = (const T*)a.wide + group * a.wide_group + row * a.wide_ld;
        Eight<T> v;
        if (col + 8 <= a.width) v.load(from + col);
        else v.load_some(from, col, a.width);
        const float scale = scale_of(largest_of_16_lanes(v.size()));
        if (col < a.width)
            store_eight(a.narrow + group * a.narrow_group + row * a.narrow_ld + col, a.width - col, v.e4m3(inverse_of(scale)));
        if (lane == 0) a.scales[id] = scale;
    }
}

// A workgroup a block of 128 x 128.
template <typename T> __global__ void __launch_bounds__(256) quantize_square_kernel(const BlockArgs a) {
    __shared__ float lds[4];
    const int lane = threadIdx.x & 15, y = threadIdx.x >> 4, high = (int)((a.rows + 127) / 128);
    const uint64_t line = blockIdx.x / (uint32_t)a.blocks, group = line / (uint32_t)high;
    const int col = (int)(blockIdx.x % (uint32_t)a.blocks) * 128 + lane * 8;
    const uint64_t row0 = (line - group * high) * 128;
    Eight<T> v[8];
    float size = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint64_t row = row0 + k * 16 + y;
        const T* from = (const T*)a.wide + group * a.wide_group + min(row, a.rows - 1) * a.wide_ld;
        if (col + 8 <= a.width) v[k].load(from + col);
        else v[k].load_some(from, col, a.width);
    }
    // rows past the end are the last one again
#pragma unroll
    for (int k = 0; k < 8; ++k) size = fmaxf(size, v[k].size());
    size = largest_of_16_lanes(size);
    size = fmaxf(size, __shfl_xor(size, 16));
    size = fmaxf(size, __shfl_xor(size, 32));
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = size;
    __syncthreads();
    size = fmaxf(fmaxf(lds[0], lds[1]), fmaxf(lds[2], lds[3]));
    const float scale = scale_of(size);
    if (threadIdx.x == 0) a.scales[blockIdx.x] = scale;
    if (col >= a.width) return;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint64_t row = row0 + k * 16 + y;
        if (row < a.rows)
            store_eight(a.narrow + group * a.narrow_group + row * a.narrow_ld + col, a.width - col, v[k].e4m3(inverse_of(scale)));
    }
}

template <typename T> __device__ __forceinline__ T rounded(float v) { return (T)v; }
// a finite value past the ends of fp16 is the end
template <> __device__ __forceinline__ f16 rounded<f16>(float v) {
    return (f16)(fabsf(v) < INFINITY ? fminf(fmaxf(v, -65504.0f), 65504.0f) : v);
}

// Eight columns a thread.  STREAM: what is written is not to stay in the caches, of which it would
// leave nothing else: 134 million values to bf16 take 80 us so and 100 otherwise.
template <typename T, bool STREAM> __global__ void __launch_bounds__(256) back_kernel(const BlockArgs a) {
    const uint32_t each = ((uint32_t)a.filled + 7) / 8;
    const uint64_t all = a.groups * a.rows * each, per = a.rows / a.part;
    for (uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x; id < all; id += (uint64_t)gridDim.x * 256) {
        const uint64_t line = row_of(id, each);
        const int col = (int)(id - line * each) * 8;
        const uint64_t group = a.groups > 1 ? (uint32_t)line / (uint32_t)a.rows : 0, row = line - group * a.rows;
        u32x2 q = {0, 0};
        float scale = 0.0f;
        if (col < a.width) {
            const uint8_t* from = a.narrow + group * a.narrow_group + row * a.narrow_ld + col;
            q = __builtin_bit_cast(u32x2, load_some<uint8_t, 8>(from, a.width - col));
            uint64_t block = line;
            if (a.high > 1) {
                const uint64_t part = per > 1 && row >= a.part;        // one or two of them
                block = (group * per + part) * ((a.part + 127) / 128) + (row - part * a.part) / 128;
            }
            scale = a.scales[block * (uint32_t)a.blocks + (uint32_t)col / 128];
        }
        float v[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[h], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[h], true);
            v[h * 4] = lo[0] * scale, v[h * 4 + 1] = lo[1] * scale, v[h * 4 + 2] = hi[0] * scale, v[h * 4 + 3] = hi[1] * scale;
        }
        T* const to = (T*)a.wide + group * a.wide_group + row * a.wide_ld + col;
        const int n = a.filled - col;
        if (n >= 8) {
#pragma unroll
            for (int h = 0; h < 8; h += Vec<T>::N) {
                Vec<T> o;
#pragma unroll
                for (int e = 0; e < Vec<T>::N; ++e) o.e[e] = rounded<T>(col + h + e < a.width ? v[h + e] : 0.0f);
                typedef u32x4 Any __attribute__((aligned(2)));
                if constexpr (STREAM) __builtin_nontemporal_store(__builtin_bit_cast(u32x4, o), (Any*)(to + h));
                else *(Any*)(to + h) = __builtin_bit_cast(u32x4, o);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) to[e] = rounded<T>(v[e]);
        }
    }
}

// 16 bytes a thread; both operands in one launch.
__global__ void __launch_bounds__(256) pack8_kernel(const Pack8Args all_parts) {
    const BlockArgs& a = all_parts.part[blockIdx.y];
    const uint32_t each = (uint32_t)a.filled / 16;
    const uint64_t all = a.groups * a.rows * each;
    for (uint64_t id = (uint64_t)blockIdx.x * 256 + threadIdx.x; id < all; id += (uint64_t)gridDim.x * 256) {
        const uint64_t line = row_of(id, each);
        const int col = (int)(id - line * each) * 16;
        const uint64_t group = a.groups > 1 ? (uint32_t)line / (uint32_t)a.rows : 0, row = line - group * a.rows;
        const uint8_t* from = a.narrow + group * a.narrow_group + row * a.narrow_ld + col;
        const Some<uint8_t, 16> v = load_some<uint8_t, 16>(from, a.width - col);
        *(u32x4*)((char*)a.wide + line * (uint32_t)a.filled + col) = __builtin_bit_cast(u32x4, v);
    }
}

// ------------------------------------------------------------------ host side --

static unsigned grid_of(uint64_t items, uint64_t each) {
    const uint64_t n = ceil_div(items, each);
    return (unsigned)(n < 8192 ? n : 8192);
}

template <typename T> static void launch_back_of(const BlockArgs& a, unsigned grid, bool stream, hipStream_t s) {
    if (stream) back_kernel<T, true><<<grid, 256, 0, s>>>(a);
    else back_kernel<T, false><<<grid, 256, 0, s>>>(a);
}

rr_status_t launch_back(const BlockArgs& a, int dt, hipStream_t s) {
    const uint64_t all = a.groups * a.rows * ceil_div((uint64_t)a.filled, 8);
    if (all == 0) return RR_OK;
    const unsigned grid = grid_of(all, 256);
    const bool stream = all * 8 * type_bytes(dt) > 128u << 20;      // half of the Infinity Cache
    switch (dt) {
        case RR_BF16: launch_back_of<bf16>(a, grid, stream, s); break;
        case RR_FP16: launch_back_of<f16>(a, grid, stream, s); break;
        default: launch_back_of<float>(a, grid, stream, s);
    }
    return launched();
}

rr_status_t launch_pack8(const Pack8Args& a, int parts, hipStream_t s) {
    uint64_t most = 0;
    for (int p = 0; p < parts; ++p) {
        const uint64_t all = a.part[p].groups * a.part[p].rows * ((uint32_t)a.part[p].filled / 16);
        most = all > most ? all : most;
    }
    if (most == 0) return RR_OK;
    pack8_kernel<<<dim3(grid_of(most, 256), (unsigned)parts), 256, 0, s>>>(a);
    return launched();
}

static rr_status_t check(const rr_quantize_t* a, bool back, BlockArgs& k) {
    if (!a || (a->square != 0 && a->square != 1) || !is_float_type(a->dt) || a->width < 1 || a->groups < 1)
        return RR_ERR_INVALID;
    if (a->width > kMaxSize || a->rows > kMaxSize || a->groups > kMaxSize || a->groups * a->rows > kMaxSize)
        return RR_ERR_UNSUPPORTED;
    const uint64_t e = type_bytes(a->dt), blocks = ceil_div(a->width, kBlock), high = a->square ? ceil_div(a->rows, kBlock) : a->rows;
    if (a->groups * high * blocks >= 1ull << 34) return RR_ERR_UNSUPPORTED;
    if (a->square && !back && a->groups * high * blocks > (1ull << 24) - 1) return RR_ERR_UNSUPPORTED;
    if (!rows_ok(a->x, a->rows, a->width, e) || !rows_ok(a->q, a->rows, a->width, 1)) return RR_ERR_INVALID;
    if (a->rows && (!a->scales || !aligned_to(a->scales, 4))) return RR_ERR_INVALID;
    if (a->x.ld > 1ull << 40 || a->q.ld > 1ull << 40 || a->x_stride > 1ull << 44 || a->q_stride > 1ull << 44)
        return RR_ERR_UNSUPPORTED;
    const uint64_t x_one = extent(a->rows, a->x.ld, a->width, 1), q_one = extent(a->rows, a->q.ld, a->width, 1);
    if (a->groups > 1 && ((back && a->x_stride < x_one) || (!back && a->q_stride < q_one))) return RR_ERR_INVALID;
    const uint64_t x_bytes = extent(a->groups, a->x_stride, x_one, e), q_bytes = extent(a->groups, a->q_stride, q_one, 1);
    const uint64_t s_bytes = a->groups * high * blocks * 4;
    if (overlap(a->x.data, x_bytes, a->q.data, q_bytes) || overlap(a->x.data, x_bytes, a->scales, s_bytes) ||
        overlap(a->q.data, q_bytes, a->scales, s_bytes))
        return RR_ERR_INVALID;
    k = {};
    k.wide = a->x.data;
    k.narrow = (uint8_t*)a->q.data;
    k.scales = a->scales;
    k.wide_ld = a->x.ld;
    k.wide_group = a->x_stride;
    k.narrow_ld = a->q.ld;
    k.narrow_group = a->q_stride;
    k.rows = a->rows;
    k.groups = a->groups;
    k.part = a->rows ? a->rows : 1;
    k.width = k.filled = (int32_t)a->width;
    k.blocks = (int32_t)blocks;
    k.high = a->square ? 128 : 1;
    return RR_OK;
}

template <typename T> static void launch_quantize(const BlockArgs& k, hipStream_t s) {
    if (k.high > 1)
        quantize_square_kernel<T><<<(unsigned)(k.groups * ceil_div(k.rows, kBlock) * k.blocks), 256, 0, s>>>(k);
    else
        quantize_rows_kernel<T><<<grid_of(k.groups * k.rows * k.blocks, 16), 256, 0, s>>>(k);
}

}  // namespace blk

using namespace blk;

extern "C" {

rr_status_t block_quantize(const rr_quantize_t* a, rr_stream_t stream) {
    BlockArgs k;
    const rr_status_t st = check(a, false, k);
    if (st != RR_OK || a->rows == 0) return st;
    if (a->dt == RR_BF16) launch_quantize<bf16>(k, (hipStream_t)stream);
    else if (a->dt == RR_FP16) launch_quantize<f16>(k, (hipStream_t)stream);
    else launch_quantize<float>(k, (hipStream_t)stream);
    return launched();
}

rr_status_t block_dequantize(const rr_quantize_t* a, rr_stream_t stream) {
    BlockArgs k;
    const rr_status_t st = check(a, true, k);
    if (st != RR_OK || a->rows == 0) return st;
    return launch_back(k, a->dt, (hipStream_t)stream);
}

}  // extern "C"
