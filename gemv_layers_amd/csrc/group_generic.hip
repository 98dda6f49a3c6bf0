// General kernel of the products grouped by expert and of the 8-bit floating-point products, for operands
// that the matrix kernels do not take (unaligned pointers, leading dimensions or widths without the needed
// multiples, extents beyond their 32-bit offsets). Element-wise bounds-checked loads through LDS; each thread
// keeps a 4 x 4 block of float32 sums, and for codes a second one over the current block of 128 k, whose
// scales are applied at its end. Bound by its scalar multiply-adds and not tuned further.

#include "common.h"
#include "f8.h"
#include "group.h"
#include "ops.h"
#include "plan.h"

namespace glk {

template <int MODE>
__global__ void __launch_bounds__(256) group_generic_kernel(OpArgs p, GroupArgs g, int tiles_n) {
    constexpr int T = 64, KS = 16;
    constexpr bool F8 = MODE == kOpF8;
    constexpr bool A_CONTIG = MODE != kOpAtb;
    constexpr bool B_CONTIG = MODE == kOpF8 || MODE == kOpAbt;
    __shared__ float sa[KS][T + 1];
    __shared__ float sb[KS][T + 1];
    // the group's operands; `M` rows of C, `K` of the summed index
    int64_t M, K = p.K, m0, n0, group = 0, first = 0;
    if constexpr (MODE == kOpAtb) {
        const int per = (int)((p.M - 1) / T + 1) * tiles_n;
        group = blockIdx.x / per;
        const int tile = blockIdx.x % per;
        int at, rows;
        group_rows(g, (int)group, &at, &rows);
        first = at;
        M = p.M;
        K = rows;
        m0 = (int64_t)(tile / tiles_n) * T;
        n0 = (int64_t)(tile % tiles_n) * T;
    } else {
        GroupSpan s;
        if (!find_span(g, T, tiles_n, EvenUnits{(int)blockIdx.x, 1}, &s)) return;
        group = max(s.group, 0);
        first = s.first;
        M = s.rows;
        if (s.group < 0) K = 0;
        m0 = (int64_t)(s.unit / tiles_n) * T;
        n0 = (int64_t)(s.unit % tiles_n) * T;
    }
    using E = std::conditional_t<F8, uint8_t, uint16_t>;
    const E* A = static_cast<const E*>(p.A) + first * p.lda;
    const E* B = static_cast<const E*>(p.B) + (MODE == kOpAtb ? first * p.ldb : group * g.stride_b);
    uint16_t* C = p.C + (MODE == kOpAtb ? group * g.stride_c : first * p.ldc);
    auto load = [](const E* x, int64_t i) {
        if constexpr (F8)
            return f8_value(x[i]);
        else
            return __builtin_bit_cast(float, (uint32_t)x[i] << 16);
    };
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    float acc[4][4] = {}, sum[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += KS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = tid + 256 * i;
            // neighbouring threads read neighbouring elements of the contiguous index
            const int ka = A_CONTIG ? e & (KS - 1) : e >> 6, ma = A_CONTIG ? e >> 4 : e & 63;
            const int kb = B_CONTIG ? e & (KS - 1) : e >> 6, nb = B_CONTIG ? e >> 4 : e & 63;
            const int64_t m = m0 + ma, n = n0 + nb;
            sa[ka][ma] = m < M && k0 + ka < K ? load(A, A_CONTIG ? m * p.lda + k0 + ka : (k0 + ka) * p.lda + m) : 0.f;
            sb[kb][nb] = n < p.N && k0 + kb < K ? load(B, B_CONTIG ? n * p.ldb + k0 + kb : (k0 + kb) * p.ldb + n) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            float a[4], b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = sa[kk][ty * 4 + i];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = sb[kk][tx * 4 + j];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_fmaf(a[i], b[j], acc[i][j]);
        }
        __syncthreads();
        if (F8 && ((k0 + KS) % 128 == 0 || k0 + KS >= K)) {
            const int64_t kb = k0 / 128;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t m = m0 + ty * 4 + i;
                const F8Factor a = f8_factor(m < M ? p.sa[kb * p.ldsa + first + m] : 0.f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t n = n0 + tx * 4 + j;
                    const F8Factor w = f8_factor(n < p.N ? p.sb[group * g.stride_sb + n / 128 * p.ldsb + kb] : 0.f);
                    sum[i][j] = __builtin_fmaf(__builtin_ldexpf(acc[i][j], a.e + w.e - 254), a.m * w.m, sum[i][j]);
                    acc[i][j] = 0.f;
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        if (m >= M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tx * 4 + j;
            if (n < p.N) C[m * p.ldc + n] = __builtin_bit_cast(uint16_t, (__bf16)(F8 ? sum[i][j] : acc[i][j]));
        }
    }
}

hipError_t launch_group_generic(int mode, const OpArgs& a, const GroupArgs& g, hipStream_t s) {
    const int64_t tn = (a.N - 1) / 64 + 1;
    const int64_t tm = mode == kOpAtb ? ((a.M - 1) / 64 + 1) * g.groups : most_row_tiles(g.rows, g.offsets ? g.groups : 0, 64);
    if (tm > 0xFFFFFF / tn) return hipErrorInvalidValue;
    const unsigned grid = (unsigned)(tm * tn);
    switch (mode) {
        case kOpAb: group_generic_kernel<kOpAb><<<grid, 256, 0, s>>>(a, g, (int)tn); break;
        case kOpAbt: group_generic_kernel<kOpAbt><<<grid, 256, 0, s>>>(a, g, (int)tn); break;
        case kOpAtb: group_generic_kernel<kOpAtb><<<grid, 256, 0, s>>>(a, g, (int)tn); break;
        case kOpF8: group_generic_kernel<kOpF8><<<grid, 256, 0, s>>>(a, g, (int)tn); break;
        default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace glk
