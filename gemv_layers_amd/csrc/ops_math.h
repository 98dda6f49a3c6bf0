// The gated block's activation, and accesses at any element, shared by the 8-bit and training kernels
// (device side).
#pragma once

#include "common.h"

namespace glk {

// s = 1 / (1 + e^-g) in float32 as the product r p, within a few units of the last place. e^g = 2^n 2^f
// with n = round(g log2 e) and f = g log2 e - n from two fused multiply-adds with log2 e in two parts,
// so that f keeps its bits for large g; then s = p / (2^-f + p) with p = 2^n, and the hardware's exp2
// and reciprocal see arguments of ordinary size: a third of the cycles of the library exponential and
// an IEEE division (the epilogue of a 256 x 256 gated tile evaluates 128 of these a SIMD lane). Below
// g = -87.3 s itself is under float32's normal range, where a reciprocal may come out as zero; as r and
// p it loses nothing, and g s, which is still normal down to g = -91.6, is (g r) p. The clamp keeps
// infinities out of f: past it p is 0 or s is 1 whatever g is. NaN comes back through the factor g that
// every use multiplies by.
struct OpSigmoid {
    float r, p;
};
__device__ __forceinline__ OpSigmoid op_sigmoid(float g) {
    constexpr float kHi = 0x1.715476p+0f, kLo = 0x1.4ae0cp-26f;  // log2 e
    const float x = __builtin_amdgcn_fmed3f(g, -150.0f, 30.0f);
    const float n = rintf(x * kHi);
    const float f = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -n));
    const float p = __builtin_amdgcn_ldexpf(1.0f, (int)n);
    return OpSigmoid{__builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(-f) + p), p};
}

// silu(g) u
__device__ __forceinline__ float op_swiglu(float g, float u) {
    const OpSigmoid s = op_sigmoid(g);
    return g * s.r * s.p * u;
}

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
