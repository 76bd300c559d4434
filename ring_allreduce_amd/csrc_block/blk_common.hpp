// blk_common.hpp -- what the kernels of a block's operators share: element types,
// 16-byte row accesses of any alignment, activations, sums over a workgroup, and
// the host side's argument checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rr.h"

namespace blk {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16;
typedef _Float16 f16;

// ------------------------------------------------------------------ vectors --
// A Vec<T> is 16 bytes of a row: 4 fp32 or 8 bf16 / fp16 elements.  Rows may start
// at any element (odd lengths, views of wider tensors): the 16-byte access is
// declared with the element's alignment only, which gfx950 serves in one
// instruction; the last, partial vector of a row goes element by element.
template <typename T> struct Vec {
    static constexpr int N = 16 / (int)sizeof(T);
    T e[N];
};

template <typename T> struct __attribute__((packed, aligned(sizeof(T)))) Loose {
    u32x4 v;
};

template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* row, int at, int len) {
    Vec<T> r;
    if (at + Vec<T>::N <= len) {
        r = __builtin_bit_cast(Vec<T>, reinterpret_cast<const Loose<T>*>(row + at)->v);
    } else {
#pragma unroll
        for (int i = 0; i < Vec<T>::N; ++i) r.e[i] = at + i < len ? row[at + i] : (T)0.0f;
    }
    return r;
}

// A whole vector, and nothing else: behind a branch, a load is waited for before the next is
// sent (and the compiler takes it apart), which costs bandwidth-bound kernels half their rate.
template <typename T> __device__ __forceinline__ u32x4 load_raw(const T* p) {
    return reinterpret_cast<const Loose<T>*>(p)->v;
}
template <typename T> __device__ __forceinline__ Vec<T> vec_of(u32x4 v) {
    return __builtin_bit_cast(Vec<T>, v);
}
__device__ __forceinline__ u32x4 zero_unless(bool keep, u32x4 v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = keep ? v[i] : 0u;
    return v;
}
// v without its first `skip` bytes (a multiple of 2, 0 .. 16), zeros behind.
__device__ __forceinline__ u32x4 drop_first(u32x4 v, int skip) {
    const uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
    const int n = (skip & 7) * 8;
    const uint64_t low = n ? lo >> n | hi << (64 - n) : lo, high = hi >> n;
    const uint64_t a = skip >= 16 ? 0 : skip >= 8 ? high : low, b = skip >= 8 ? 0 : high;
    return u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
}

template <typename T>
__device__ __forceinline__ void store_vec(T* row, int at, int len, const Vec<T>& r) {
    u32x4 v = __builtin_bit_cast(u32x4, r);
    if (at + Vec<T>::N <= len) {
        reinterpret_cast<Loose<T>*>(row + at)->v = v;
    } else {
#pragma unroll 1
        for (; at < len; ++at) {
            row[at] = vec_of<T>(v).e[0];
            v = drop_first(v, (int)sizeof(T));
        }
    }
}

// -------------------------------------------------------------- activations --
// In 32 bits.  exp(-z) overflows to infinity for z below -88, where the logistic
// function is 0 to 32 bits: 1 / (1 + inf) = 0, and z * 0 is the right limit for
// every finite z.  The reciprocal is the hardware's, off by at most one step: a divide
// costs ten instructions a value, which the epilogue of a product has no room for (the
// SiLU of 8192 x 8192 outputs took 70 us with it).
__device__ __forceinline__ float logistic(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

// The normal distribution beyond a >= 0: *tail = 1 - Phi(a), off by 1.4e-6 of itself up to 5,
// where 1 - erf has lost all but a digit; returns exp(-a^2 / 2).  The tail is that times a
// polynomial in 1 / (1 + 0.3 a), fitted to the least largest relative error (9.7e-8) over 0
// .. 20; the rest is the rounding of a^2 / 2.  Without branches: the two ranges of erff, both
// taken by most waves, cost the GELU of 1001 x 1111 values 6 us behind its product.
__device__ __forceinline__ float normal_tail(float a, float* tail) {
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.3f * a);
    const float c[9] = {6.19887214e-06f, 0.119510077f, 0.121712074f, 0.0957123935f, 0.139562428f,
                        -0.0713275298f, 0.223317936f, -0.166166559f, 0.0376729406f};
    float q = c[8];
#pragma unroll
    for (int k = 7; k >= 0; --k) q = q * t + c[k];
    const float e = __expf(-0.5f * a * a);
    *tail = e * q;
    return e;
}
// |z|, at most 20, from where on the tail is 0 in 32 bits; NaN stays.  Infinities end here too:
// they get the limits, where z Phi(z) and z phi(z) themselves would be infinity times 0.
__device__ __forceinline__ float magnitude(float z) {
    const float a = fabsf(z);
    return a > 20.0f ? 20.0f : a;
}

template <int ACT> __device__ __forceinline__ float act_of(float z) {
    if constexpr (ACT == RR_ACT_RELU) return z > 0.0f || z != z ? z : 0.0f;
    if constexpr (ACT == RR_ACT_GELU) {        // z Phi(z), for either sign from the tail
        const float a = magnitude(z);
        float tail;
        normal_tail(a, &tail);
        return fmaxf(z, 0.0f) - a * tail;
    }
    if constexpr (ACT == RR_ACT_SILU) return z * logistic(z);
    if constexpr (ACT == RR_ACT_SIGMOID) return logistic(z);
    return z;
}

// d act / d z; 0 at the corner of relu.
template <int ACT> __device__ __forceinline__ float slope_of(float z) {
    if constexpr (ACT == RR_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == RR_ACT_GELU) {
        const float a = magnitude(z);
        float tail;
        const float e = normal_tail(a, &tail);
        return (z > 0.0f ? 1.0f - tail : tail) + copysignf(a, z) * e * 0.39894228040143268f;
    }
    if constexpr (ACT == RR_ACT_SILU) {
        const float q = logistic(z);
        return q * (1.0f + z * (1.0f - q));
    }
    if constexpr (ACT == RR_ACT_SIGMOID) {
        const float q = logistic(z);
        return q * (1.0f - q);
    }
    return 1.0f;
}

// Of N values at once, so that the choice of function is made once for all of them.
template <int ACT, int N> __device__ __forceinline__ void act_each(float (&v)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = act_of<ACT>(v[e]);
}
template <int ACT, int N> __device__ __forceinline__ void slope_each(float (&v)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = slope_of<ACT>(v[e]);
}
template <int N> __device__ __forceinline__ void act_values(int act, float (&v)[N]) {
    switch (act) {
        case RR_ACT_RELU: act_each<RR_ACT_RELU>(v); break;
        case RR_ACT_GELU: act_each<RR_ACT_GELU>(v); break;
        case RR_ACT_SILU: act_each<RR_ACT_SILU>(v); break;
        case RR_ACT_SIGMOID: act_each<RR_ACT_SIGMOID>(v); break;
        default: break;
    }
}
template <int N> __device__ __forceinline__ void act_slopes(int act, float (&v)[N]) {
    switch (act) {
        case RR_ACT_RELU: slope_each<RR_ACT_RELU>(v); break;
        case RR_ACT_GELU: slope_each<RR_ACT_GELU>(v); break;
        case RR_ACT_SILU: slope_each<RR_ACT_SILU>(v); break;
        case RR_ACT_SIGMOID: slope_each<RR_ACT_SIGMOID>(v); break;
        default: slope_each<RR_ACT_NONE>(v); break;
    }
}

// --------------------------------------------------------------------- sums --
// Sum over WIDTH neighbouring lanes (a power of two up to 64), to all of them.
template <int WIDTH> __device__ __forceinline__ float lane_sum(float v) {
#pragma unroll
    for (int d = WIDTH / 2; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// ----------------------------------------------------------------- the host --
inline uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }
inline bool is_float_type(int dt) { return dt == RR_FP32 || dt == RR_BF16 || dt == RR_FP16; }
inline uint64_t type_bytes(int dt) { return dt == RR_BF16 || dt == RR_FP16 ? 2 : 4; }
inline bool aligned_to(const void* p, uint64_t n) { return (uintptr_t)p % n == 0; }

// Whether [a, a + na) and [b, b + nb) share a byte.
inline bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
    if (!a || !b || !na || !nb) return false;
    return (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}

// Bytes that `rows` rows of `width` elements, `ld` elements apart, reach over.
inline uint64_t extent(uint64_t rows, uint64_t ld, uint64_t width, uint64_t bytes) {
    return rows ? ((rows - 1) * ld + width) * bytes : 0;
}

inline rr_status_t launched() { return hipGetLastError() == hipSuccess ? RR_OK : RR_ERR_HIP; }

// Compute units of the current device (0: the runtime gave no answer).
inline int compute_units() {
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 0;
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
        return 0;
    return n;
}

}  // namespace blk
