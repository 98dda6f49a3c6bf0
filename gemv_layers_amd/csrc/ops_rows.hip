// Row kernels of the 8-bit and training operators: one pass over memory each.
//
// Quantisation of rows (the arithmetic is in codes.h). A row stays in the registers of its workgroup
// between the maximum and the codes, so that memory is read once (2 bytes an element) and written
// once (1 byte). Few rows are bound by latency, a load, a reduction and a store, and take wide
// workgroups; many rows by memory. 16 rows of 4096 take 4.8 us, 4096 rows 12.0 us (4.2 TB/s; a copy
// reaches 6: each workgroup's load, reduction and store are in series). Rows may start at any element: the
// 16-byte loads need no alignment, and cost a quarter more without it (4096 x 4095: 15 us, where element
// by element it took 24). Rows of up to 65536 stay in registers (16 x 28672: 5.6 us
// against 35 in two passes).
//
// The gated block's gradient, element by element: reads dC, g and u, writes dg and du, 10 bytes an
// element. 4096 x 11008: 67 us, 6.7 TB/s.

#include "codes.h"
#include "common.h"
#include "ops.h"
#include "ops_math.h"

namespace glk {

// one row per workgroup of NW waves, NC 16-byte chunks per thread in registers
template <int NW, int NC>
__global__ void __launch_bounds__(64 * NW) i8_quantize_kernel(const uint16_t* __restrict__ X, int K, int64_t ldx,
                                                              int8_t* __restrict__ Q, int64_t ldq,
                                                              float* __restrict__ S) {
    __shared__ uint32_t part[NW];
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x;
    const uint16_t* x = X + r * ldx;
    u32x4 v[NC];
    uint32_t amax = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int k = 8 * (c * 64 * NW + tid);
        v[c] = u32x4{0, 0, 0, 0};
        if (k + 8 <= K) {
            v[c] = load8(x + k);
        } else if (k < K) {
            v[c] = load_some(x + k, K - k);
        }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) amax = magnitude8(v[c], amax);
    amax = wave_max(amax);
    if constexpr (NW > 1) {
        if ((tid & 63) == 0) part[tid >> 6] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NW; ++w) amax = max(amax, part[w]);
    }
    const CodeScale cs = code_scale(amax);
    if (tid == 0) S[r] = cs.s;
    int8_t* q = Q + r * ldq;
    const int64_t padded = min(ldq, (int64_t)(K + 15) / 16 * 16);
    const bool wide = ((reinterpret_cast<uintptr_t>(Q) | (uintptr_t)ldq) & 7) == 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int64_t k = 8 * ((int64_t)c * 64 * NW + tid);
        if (k >= padded) continue;
        const u32x2 w = codes8(v[c], cs);  // (elements past K are zero in v)
        if (wide && k + 8 <= padded) {
            *reinterpret_cast<u32x2*>(q + k) = w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k + j < padded) q[k + j] = (int8_t)(w[j >> 2] >> (8 * (j & 3)));
        }
    }
}

// longer rows than registers hold: two passes over the row, element by element
__global__ void __launch_bounds__(256) i8_quantize_any_kernel(const uint16_t* __restrict__ X, int64_t K, int64_t ldx,
                                                              int8_t* __restrict__ Q, int64_t ldq,
                                                              float* __restrict__ S) {
    __shared__ uint32_t part[4];
    const int tid = threadIdx.x;
    const int64_t r = blockIdx.x;
    const uint16_t* x = X + r * ldx;
    uint32_t amax = 0;
    for (int64_t k = tid; k < K; k += 256) amax = max(amax, (uint32_t)x[k] & 0x7FFFu);
    amax = wave_max(amax);
    if ((tid & 63) == 0) part[tid >> 6] = amax;
    __syncthreads();
    amax = max(max(part[0], part[1]), max(part[2], part[3]));
    const CodeScale cs = code_scale(amax);
    if (tid == 0) S[r] = cs.s;
    int8_t* q = Q + r * ldq;
    const int64_t padded = min(ldq, (K + 15) / 16 * 16);
    for (int64_t k = tid; k < padded; k += 256)
        q[k] = k < K ? (int8_t)code_of(__builtin_bit_cast(float, (uint32_t)x[k] << 16), cs) : (int8_t)0;
}

hipError_t launch_i8_quantize(const uint16_t* X, int64_t R, int64_t K, int64_t ldx, int8_t* Q, int64_t ldq,
                              float* S, hipStream_t s) {
    // a launch holds at most 2^32 - 1 threads: 2^24 - 1 rows of 256, 2^22 - 1 of 1024
    auto run = [&](auto kernel, int threads, auto k) {
        const int64_t most = int64_t(0xFFFFFFFF) / threads;
        for (int64_t r = 0; r < R; r += most)
            kernel<<<(unsigned)(R - r < most ? R - r : most), threads, 0, s>>>(X + r * ldx, k, ldx, Q + r * ldq, ldq,
                                                                            S + r);
    };
    // chunks of 8 elements, a padded row's among them
    const int64_t chunks = (K + 15) / 16 * 2;
    if (chunks > 1024 * 8)
        run(i8_quantize_any_kernel, 256, K);
    else if (chunks > 1024 * 4)
        run(i8_quantize_kernel<16, 8>, 1024, (int)K);
    else if (chunks > 1024 * 2)
        run(i8_quantize_kernel<16, 4>, 1024, (int)K);
    else if (chunks > 256 && R <= 512)
        run(i8_quantize_kernel<16, 2>, 1024, (int)K);
    else if (chunks <= 64)
        run(i8_quantize_kernel<1, 1>, 64, (int)K);
    else if (chunks <= 256)
        run(i8_quantize_kernel<4, 1>, 256, (int)K);
    else if (chunks <= 512)
        run(i8_quantize_kernel<4, 2>, 256, (int)K);
    else if (chunks <= 1024)
        run(i8_quantize_kernel<4, 4>, 256, (int)K);
    else
        run(i8_quantize_kernel<4, 8>, 256, (int)K);
    return hipGetLastError();
}

// ---- the gated block's gradient -------------------------------------------------------------------

// du = d silu(g), dg = d u s (1 + g (1 - s)) with s = sigmoid(g), in float32
__device__ __forceinline__ void swiglu_grad1(float d, float g, float u, float& dg, float& du) {
    const OpSigmoid sig = op_sigmoid(g);
    du = d * (g * sig.r * sig.p);
    dg = d * u * (sig.r * (1.0f + g * (1.0f - sig.r * sig.p)) * sig.p);
}

// dGU may be GU itself: every element is read by the thread that writes it, before it does. VEC: eight
// elements a thread. I: the type that counts them (the division by a row's length costs a 64-bit index
// more than the rest of a small call).
template <bool VEC, class I>
__global__ void __launch_bounds__(256) swiglu_grad_kernel(const uint16_t* __restrict__ dC, int64_t lddc,
                                                          const uint16_t* GU, int64_t ldgu, uint16_t* dGU,
                                                          int64_t lddgu, I total, I per_row, int64_t N) {
    const I step = (I)gridDim.x * 256;
    for (I e = (I)blockIdx.x * 256 + threadIdx.x; e < total; e += step) {
        const I m = e / per_row;
        const int64_t n = (VEC ? 8 : 1) * (int64_t)(e - m * per_row);
        const uint16_t* pd = dC + m * lddc + n;
        const uint16_t* pg = GU + m * ldgu + n;
        uint16_t* po = dGU + m * lddgu + n;
        if constexpr (VEC) {
            const u32x4 d = *reinterpret_cast<const u32x4*>(pd);
            const u32x4 g = *reinterpret_cast<const u32x4*>(pg);
            const u32x4 u = *reinterpret_cast<const u32x4*>(pg + N);
            u32x4 og, ou;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float g0, g1, u0, u1;
                swiglu_grad1(bf16_lo(d[j]), bf16_lo(g[j]), bf16_lo(u[j]), g0, u0);
                swiglu_grad1(bf16_hi(d[j]), bf16_hi(g[j]), bf16_hi(u[j]), g1, u1);
                og[j] = pack_bf16x2(g0, g1);
                ou[j] = pack_bf16x2(u0, u1);
            }
            *reinterpret_cast<u32x4*>(po) = og;
            *reinterpret_cast<u32x4*>(po + N) = ou;
        } else {
            auto wide = [](uint16_t h) { return __builtin_bit_cast(float, (uint32_t)h << 16); };
            float dg, du;
            swiglu_grad1(wide(*pd), wide(*pg), wide(pg[N]), dg, du);
            *po = __builtin_bit_cast(uint16_t, (__bf16)dg);
            po[N] = __builtin_bit_cast(uint16_t, (__bf16)du);
        }
    }
}

hipError_t launch_swiglu_grad(const uint16_t* dC, int64_t lddc, const uint16_t* GU, int64_t ldgu, uint16_t* dGU,
                              int64_t lddgu, int64_t M, int64_t N, hipStream_t s) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(dC) | reinterpret_cast<uintptr_t>(GU) | reinterpret_cast<uintptr_t>(dGU);
    const bool vec = (at & 15) == 0 && ((N | lddc | ldgu | lddgu) & 7) == 0;
    const int64_t per_row = vec ? N / 8 : N, total = M * per_row;
    const unsigned blocks = (unsigned)(total < (int64_t(1) << 28) ? (total + 255) / 256 : 1 << 20);
    auto run = [&](auto kernel, auto zero) {
        using I = decltype(zero);
        kernel<<<blocks, 256, 0, s>>>(dC, lddc, GU, ldgu, dGU, lddgu, (I)total, (I)per_row, N);
    };
    // (32-bit counting: the last index plus the grid's stride stays below 2^32)
    const bool small = total < (int64_t(1) << 31);
    if (vec && small)
        run(swiglu_grad_kernel<true, uint32_t>, uint32_t());
    else if (vec)
        run(swiglu_grad_kernel<true, int64_t>, int64_t());
    else if (small)
        run(swiglu_grad_kernel<false, uint32_t>, uint32_t());
    else
        run(swiglu_grad_kernel<false, int64_t>, int64_t());
    return hipGetLastError();
}

}  // namespace glk
