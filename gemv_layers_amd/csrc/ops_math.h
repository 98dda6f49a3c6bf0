// The gated block's activation, and accesses at any element, shared by the 8-bit and training kernels
// (device side).
#pragma once

#include "common.h"

namespace glk {

// 1 / (1 + e^-g) in float32, within a few units of the last place. e^x = 2^n 2^f with n = round(x
// log2 e) and f = x log2 e - n from two fused multiply-adds with log2 e in two parts, so that f keeps
// its bits for large x; the hardware's exp2 and reciprocal do the rest, a third of the cycles of the
// library exponential and an IEEE division (the epilogue of a 256 x 256 gated tile evaluates 128 of
// these a SIMD lane). Beyond 150 the exponential is 0 or infinite whatever x is; the clamp keeps
// infinities out of f, and NaN comes back through the factor g that every use multiplies by.
__device__ __forceinline__ float op_sigmoid(float g) {
    constexpr float kHi = 0x1.715476p+0f, kLo = 0x1.4ae0cp-26f;  // log2 e
    const float x = __builtin_amdgcn_fmed3f(-g, -150.0f, 150.0f);
    const float n = rintf(x * kHi);
    const float f = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -n));
    const float e = __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
    return __builtin_amdgcn_rcpf(1.0f + e);
}

// silu(g) u
__device__ __forceinline__ float op_swiglu(float g, float u) { return g * op_sigmoid(g) * u; }

// eight bf16 values at any element: one 16-byte load, which needs no alignment
__device__ __forceinline__ u32x4 load8(const uint16_t* x) {
    typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
    return *reinterpret_cast<const u32x4_at2*>(x);
}
// stores the first `left` of eight bf16 values at any element: one 16-byte store where all count
__device__ __forceinline__ void store8(uint16_t* x, const u32x4& v, int left) {
    typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
    if (left >= 8) {
        *reinterpret_cast<u32x4_at2*>(x) = v;
    } else {
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < left) x[j] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
    }
}

}  // namespace glk
