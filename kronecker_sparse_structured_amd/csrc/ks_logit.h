// ks_logit.h -- device helpers of the kernels that read rows of token logits.
#pragma once

#include <cstdint>

#include <hip/hip_runtime.h>

#include "ks_device.h"

namespace ks {

// log2 e in two parts: the fp32 value alone is 1.3e-8 too small, which a sum of
// terms near exp(-6) shows as 8e-8, the same way in every row
constexpr float kLog2e = 1.44269504088896340736f, kLog2eLow = 1.92596299e-8f;
constexpr float kLowest = -3.402823466e38f;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));   // elements in 16 bytes

template <typename T>
__device__ __forceinline__ void widen(u32x4 w, float (&x)[kVec<T>]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            x[i] = __uint_as_float(w[i]);
        } else {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    }
}

template <typename T>
__device__ __forceinline__ T narrow(float x) {
    if constexpr (sizeof(T) == 4) return x;
    else return to_bf16(x);
}

template <typename T>
__device__ __forceinline__ u32x4 pack(const float (&x)[kVec<T>]) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(x[i]);
        else w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    }
    return w;
}

// Elements before the first 128-byte line that starts at or after p, at most n.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int n) {
    const int bytes = static_cast<int>((128 - reinterpret_cast<uintptr_t>(p) % 128) % 128);
    return min(n, bytes / static_cast<int>(sizeof(T)));
}

__device__ __forceinline__ float exp_of(float d) {
    return __builtin_amdgcn_exp2f(__builtin_fmaf(d, kLog2e, d * kLog2eLow));
}

// Joins (m2, s2) to (m, s).
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
    const float top = fmaxf(m, m2);
    s = s * exp_of(m - top) + s2 * exp_of(m2 - top);
    m = top;
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
    return x;
}

}  // namespace ks
