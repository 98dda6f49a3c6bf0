// General kernel of the 8-bit and training products, for operands that the matrix kernels do not
// take (unaligned pointers, leading dimensions or widths without the needed multiples, extents
// beyond their 32-bit offsets). Element-wise bounds-checked loads through LDS; each thread keeps a
// 4 x 4 block of sums, float32 FMAs for bf16 and 32-bit integer multiply-adds for codes, whose
// sums are exact. A gated product keeps a second block for the up half. It is bound by its
// scalar multiply-adds, not by memory, and is not tuned further.

#include "common.h"
#include "ops.h"
#include "ops_math.h"

namespace glk {

template <bool I8>
struct Elem {
    using Store = uint16_t;
    using Acc = float;
    static __device__ __forceinline__ Acc load(const void* p, int64_t i) {
        return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
    }
    static __device__ __forceinline__ Acc fma(Acc a, Acc b, Acc c) { return __builtin_fmaf(a, b, c); }
};
template <>
struct Elem<true> {
    using Store = int8_t;
    using Acc = int;
    static __device__ __forceinline__ Acc load(const void* p, int64_t i) { return static_cast<const int8_t*>(p)[i]; }
    static __device__ __forceinline__ Acc fma(Acc a, Acc b, Acc c) { return a * b + c; }
};

template <int MODE, bool GLU>
__global__ void __launch_bounds__(256) op_generic_kernel(OpArgs p, int64_t tiles_n) {
    constexpr int T = 64, KS = 16;
    using E = Elem<MODE == kOpI8>;
    using Acc = typename E::Acc;
    constexpr bool A_CONTIG = MODE != kOpAtb;
    constexpr bool B_CONTIG = MODE == kOpI8 || MODE == kOpAbt;
    __shared__ Acc sa[KS][T + 1];
    __shared__ Acc sb[KS][T + 1];
    __shared__ Acc su[GLU ? KS : 1][T + 1];
    const int tid = threadIdx.x;
    const int tx = tid & 15, ty = tid >> 4;
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * T, n0 = (int64_t)(blockIdx.x % tiles_n) * T;
    Acc acc[4][4] = {}, accu[4][4] = {};
    for (int64_t k0 = 0; k0 < p.K; k0 += KS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = tid + 256 * i;
            // neighbouring threads read neighbouring elements of the contiguous index
            const int ka = A_CONTIG ? e & (KS - 1) : e >> 6, ma = A_CONTIG ? e >> 4 : e & 63;
            const int kb = B_CONTIG ? e & (KS - 1) : e >> 6, nb = B_CONTIG ? e >> 4 : e & 63;
            const int64_t m = m0 + ma, n = n0 + nb;
            sa[ka][ma] = (m < p.M && k0 + ka < p.K)
                             ? E::load(p.A, A_CONTIG ? m * p.lda + k0 + ka : (k0 + ka) * p.lda + m)
                             : Acc(0);
            const bool ok = n < p.N && k0 + kb < p.K;
            sb[kb][nb] = ok ? E::load(p.B, B_CONTIG ? n * p.ldb + k0 + kb : (k0 + kb) * p.ldb + n) : Acc(0);
            if constexpr (GLU)
                su[kb][nb] = ok ? E::load(p.B, B_CONTIG ? (p.N + n) * p.ldb + k0 + kb : (k0 + kb) * p.ldb + p.N + n)
                                : Acc(0);
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            Acc a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = sa[kk][ty * 4 + i];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = sb[kk][tx * 4 + j];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = E::fma(a[i], b[j], acc[i][j]);
            if constexpr (GLU) {
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = su[kk][tx * 4 + j];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) accu[i][j] = E::fma(a[i], b[j], accu[i][j]);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        if (m >= p.M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tx * 4 + j;
            if (n >= p.N) continue;
            float g = (float)acc[i][j], u = GLU ? (float)accu[i][j] : 0.f;
            if constexpr (MODE == kOpI8) {
                g = g * p.sa[m] * p.sb[n];
                if constexpr (GLU) u = u * p.sa[m] * p.sb[p.N + n];
            }
            if constexpr (MODE == kOpTrain) {
                p.GU[m * p.ldgu + n] = __builtin_bit_cast(uint16_t, (__bf16)g);
                p.GU[m * p.ldgu + p.N + n] = __builtin_bit_cast(uint16_t, (__bf16)u);
            }
            const float h = GLU ? op_swiglu(g, u) : g;
            p.C[m * p.ldc + n] = __builtin_bit_cast(uint16_t, (__bf16)h);
        }
    }
}

hipError_t launch_op_generic(int mode, bool glu, const OpArgs& a, hipStream_t s) {
    const int64_t tn = (a.N - 1) / 64 + 1, tm = (a.M - 1) / 64 + 1;
    if (tm > 0xFFFFFF / tn) return hipErrorInvalidValue;
    const unsigned grid = (unsigned)(tm * tn);
    if (mode == kOpI8 && glu)
        op_generic_kernel<kOpI8, true><<<grid, 256, 0, s>>>(a, tn);
    else if (mode == kOpI8)
        op_generic_kernel<kOpI8, false><<<grid, 256, 0, s>>>(a, tn);
    else if (mode == kOpAbt)
        op_generic_kernel<kOpAbt, false><<<grid, 256, 0, s>>>(a, tn);
    else if (mode == kOpAtb)
        op_generic_kernel<kOpAtb, false><<<grid, 256, 0, s>>>(a, tn);
    else
        op_generic_kernel<kOpTrain, true><<<grid, 256, 0, s>>>(a, tn);
    return hipGetLastError();
}

}  // namespace glk
