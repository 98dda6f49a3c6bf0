// Symmetric 8-bit codes of bf16 rows, shared by the kernels that make them (device side).
//
// s = max|x| / 127 in float32 and q = round(x / s) for each row. The maximum is an integer one over
// the magnitude bits of bf16, whose order is that of the values, infinities and NaN last: no value is
// lost to a comparison with NaN. The codes are those of the correctly rounded float32 quotient x / s,
// from one multiplication by 127 / max|x|: with bf16 x, 127 x / max|x| = k + 1/2 means 254 x = (2 k + 1)
// max|x|, so 127 divides 2 k + 1 (then |x| = max|x| / 2, whose code is divided out once a row) or the
// mantissa of max|x| (then s and the factor are powers of two and nothing rounds). Any other x is
// off half-way by 1 / (254 * 255) of its size at least, 100 times the float32 roundings of either way.
#pragma once

#include "common.h"

namespace glk {

struct CodeScale {
    float s, inv;     // the row's scale, and 127 / max|x|
    float half, qh;   // max|x| / 2, and the magnitude of its code
    bool divide;      // a row so small that the scale may be subnormal: every code by division
    bool none;        // a row of zeros, or with an infinity or NaN: codes 0
};
__device__ __forceinline__ CodeScale code_scale(uint32_t amax_bits) {
    const float amax = __builtin_bit_cast(float, amax_bits << 16);
    CodeScale c;
    c.none = amax_bits == 0 || amax_bits >= 0x7F80u;
    c.s = amax_bits >= 0x7F80u ? __builtin_nanf("") : amax / 127.0f;
    c.divide = amax < 0x1p-60f;
    c.inv = 127.0f / amax;
    c.half = 0.5f * amax;
    c.qh = rintf(c.half / c.s);
    return c;
}
__device__ __forceinline__ int code_of(float x, const CodeScale& c) {
    if (c.none) return 0;
    if (c.divide) return (int)rintf(x / c.s);
    const float q = rintf(x * c.inv);
    return (int)(fabsf(x) == c.half ? copysignf(c.qh, x) : q);
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    return v;
}

// the largest magnitude bits of eight bf16 values
__device__ __forceinline__ uint32_t magnitude8(const u32x4& v, uint32_t m) {
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, max(v[j] & 0x7FFFu, (v[j] >> 16) & 0x7FFFu));
    return m;
}
// their codes, in order
__device__ __forceinline__ u32x2 codes8(const u32x4& v, const CodeScale& c) {
    u32x2 w = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float e = (j & 1) ? bf16_hi(v[j >> 1]) : bf16_lo(v[j >> 1]);
        w[j >> 2] |= ((uint32_t)code_of(e, c) & 0xFFu) << (8 * (j & 3));
    }
    return w;
}
// eight bf16 values from `left` (1 .. 7) of them, the rest zeros, element by element
__device__ __forceinline__ u32x4 load_some(const uint16_t* x, int left) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 7; ++j)
        if (j < left) w[j >> 1] |= (uint32_t)x[j] << (16 * (j & 1));
    return u32x4{w[0], w[1], w[2], w[3]};
}
}  // namespace glk
