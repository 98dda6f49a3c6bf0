// e4m3 codes (OCP FP8, largest magnitude 448, no infinities) and their scales, shared by the kernels that make
// and read them (device side).
//
// A block's scale is S = amax / 448 in float32 and its codes are e4m3(448 x / amax), rounded to nearest, ties
// to even: the quotient of the exact values, which the correctly rounded float32 quotient of 448 x and amax
// rounds to as well, as is shown here. With bf16 x and amax, 448 x has at most 11 significant bits (448 = 7 *
// 64), and half-way between two codes lies h = j 2^i with odd j < 32. The quotient equals h only if 448 x = h
// amax, where float32 holds it exactly; else |448 x - h amax| is a whole multiple of the products' last bit,
// and both have at most 13 bits: it is off by 2^-13 of its size at least, 1000 times a float32 rounding. From
// q = 448 x * (1 / amax), off by 2^-22, one step q + (448 x - q amax) / amax gives h itself where the quotient
// is h, and stays on its side of h elsewhere.
// The largest code is 448 x / amax <= 448, so nothing saturates. A scale is 2^-126 at least (codes e4m3(x 2^126),
// exact products): below, float32 scales would lose bits. Blocks of zeros get S = 0; with an infinity or a NaN
// S = NaN and codes 0, so that every output made from them is NaN.
#pragma once

#include "codes.h"
#include "common.h"

namespace glk {

struct F8Scale {
    float s;          // the block's scale
    float inv, amax;  // 1 / amax and amax, scaled (see below)
    float up;         // factor of x
};
// Scaled by a power of two so that neither 448 x overflows nor 1 / amax is subnormal: x and amax times `up` / 448.
__device__ __forceinline__ F8Scale f8_scale(uint32_t amax_bits) {
    const float amax = __builtin_bit_cast(float, amax_bits << 16);
    F8Scale c;
    if (amax_bits == 0 || amax_bits >= 0x7F80u) {  // codes 0
        c.s = amax_bits ? __builtin_nanf("") : 0.f;
        c.inv = 0.f;
        c.amax = 0.f;
        c.up = 0.f;
    } else if (amax < 448.f * 0x1p-126f) {  // S = 2^-126: codes of x 2^126
        c.s = 0x1p-126f;
        c.inv = 1.f;
        c.amax = 1.f;
        c.up = 0x1p126f;
    } else {
        const float e = amax >= 1.f ? 0x1p-64f : 0x1p64f;
        c.s = amax / 448.f;
        c.amax = amax * e;
        c.inv = 1.f / c.amax;
        c.up = 448.f * e;
    }
    return c;
}
// 448 x / amax (float32, see above); x finite, or c.up = 0
__device__ __forceinline__ float f8_quotient(float x, const F8Scale& c) {
    const float n = x * c.up;
    const float q = n * c.inv;
    return __builtin_fmaf(__builtin_fmaf(-q, c.amax, n), c.inv, q);
}
// the codes of four values, in order (v_cvt_pk_fp8_f32: nearest, ties to even)
__device__ __forceinline__ uint32_t f8_codes4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
// the codes of eight bf16 values (of which infinities and NaN only where c.up = 0), in order
__device__ __forceinline__ u32x2 f8_codes8(const u32x4& v, const F8Scale& c) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = f8_quotient((j & 1) ? bf16_hi(v[j >> 1]) : bf16_lo(v[j >> 1]), c);
    const u32x2 w = {f8_codes4(q[0], q[1], q[2], q[3]), f8_codes4(q[4], q[5], q[6], q[7])};
    return c.up == 0.f ? u32x2{0, 0} : w;
}
// the largest of the 16 lanes of a row of lanes, in all of them
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
#define GLK_ROR(n) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + n, 0xF, 0xF, false))
    GLK_ROR(8);
    GLK_ROR(4);
    GLK_ROR(2);
    GLK_ROR(1);
#undef GLK_ROR
    return v;
}

// A scale as m 2^(e - 127), e from 0 to 254: its exponent field, and 1 <= |m| < 2 for a normal one (zeros, infinities and
// NaN are m themselves). The product of two scales may be outside float32's range, or among its subnormal numbers, where an
// output is inside: a block's sum is taken times the powers of two first, which is exact, and then times m m', below 4.
// Where the product of the scales is a normal number the result is the sum times that, bit for bit.
struct F8Factor {
    float m;
    int e;
};
__device__ __forceinline__ F8Factor f8_factor(float s) {
    const int e = min(__builtin_amdgcn_ubfe(__builtin_bit_cast(uint32_t, s), 23, 8), 254u);
    return {__builtin_ldexpf(s, 127 - e), e};
}
// whether `product`, of scales a and w, is zero, subnormal or infinite though neither of them is zero
__device__ __forceinline__ bool f8_far_product(float a, float w, float product) {
    return __builtin_amdgcn_classf(product, 0x2F4) && a != 0.f && w != 0.f;
}

// the value of a code
__device__ __forceinline__ float f8_value(uint8_t code) { return __builtin_amdgcn_cvt_f32_fp8((int)code, 0); }

}  // namespace glk
