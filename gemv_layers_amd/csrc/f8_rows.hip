// Quantisation to e4m3 codes with a scale for each block of 128 (the arithmetic is in f8.h): activations by
// row and block of 128 columns, weights by 128 x 128 block. One pass over memory, 2 bytes read and 1 written
// an element.
//
// Activations: a wave takes 16 rows of one block of columns, 16 lanes a row and 16 bytes a lane, all loads
// before the first maximum, and a workgroup four neighbouring blocks, 1 KB of each row. Scales are stored
// block by block, as the products read them (16 rows are 64 neighbouring bytes).
// Weights: a workgroup takes a 128 x 128 block, which stays in its registers between the maximum and the codes.
//
// Bound by HBM from a few MB on, where a copy of 1 GiB reaches 5.1 to 6.1 TB/s: activations 8192 x 4096 19.2 us (5.3 TB/s),
// 4096 x 11008 25-29 (4.6-5.5), 4096 x 4096 11.6 (4.4); weights 4096 x 11008 25.1 (5.4), 11008 x 4096 26.6 (5.1), 4096 x 4096
// 11.9 (4.2), 8 of 11008 x 4096 205 (5.3). 16 x 11008 activations 2.4 to 3.0, the launch.

#include "common.h"
#include "f8.h"
#include "ops.h"
#include "ops_math.h"

namespace glk {

// eight bf16 values from x + k of a row of K
__device__ __forceinline__ u32x4 f8_load(const uint16_t* x, int64_t k, int64_t K) {
    if (k + 8 <= K) return load8(x + k);
    if (k < K) return load_some(x + k, (int)(K - k));
    return u32x4{0, 0, 0, 0};
}
// their codes to q + k of a row of `padded` bytes
__device__ __forceinline__ void f8_store(uint8_t* q, int64_t k, int64_t padded, const u32x2& w, bool wide) {
    if (wide && k + 8 <= padded) {
        *reinterpret_cast<u32x2*>(q + k) = w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k + j < padded) q[k + j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
    }
}
// the bytes of a row that are written: up to a multiple of 16 where the rows have room
__device__ __forceinline__ int64_t f8_padded(int64_t K, int64_t ldq) { return min(ldq, (K + 15) / 16 * 16); }

// IT: groups of four rows a wave
template <int IT>
__global__ void __launch_bounds__(256) f8_quantize_kernel(const uint16_t* __restrict__ X, int64_t R, int64_t K,
                                                          int64_t ldx, uint8_t* __restrict__ Q, int64_t ldq,
                                                          float* __restrict__ S, int64_t lds, int groups_k) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t r0 = (int64_t)(blockIdx.x / groups_k) * (4 * IT) + (lane >> 4);
    const int64_t block = (int64_t)(blockIdx.x % groups_k) * 4 + wave, k = block * 128 + 8 * (lane & 15);
    if (block * 128 >= K) return;
    u32x4 v[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int64_t r = r0 + 4 * i;
        v[i] = r < R ? f8_load(X + r * ldx, k, K) : u32x4{0, 0, 0, 0};
    }
    const int64_t padded = f8_padded(K, ldq);
    const bool wide = ((reinterpret_cast<uintptr_t>(Q) | (uintptr_t)ldq) & 7) == 0;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int64_t r = r0 + 4 * i;
        const F8Scale c = f8_scale(row_max(magnitude8(v[i], 0)));
        if (r >= R) continue;
        f8_store(Q + r * ldq, k, padded, f8_codes8(v[i], c), wide);
        if ((lane & 15) == 0) S[block * lds + r] = c.s;
    }
}

__global__ void __launch_bounds__(256) f8_quantize_weight_kernel(F8WeightArgs p, int64_t nb, int64_t kb) {
    __shared__ uint32_t part[4];
    const int tid = threadIdx.x;
    const int64_t id = blockIdx.x, b = id % kb, n0 = id / kb % nb * 128, e = id / kb / nb;
    const uint16_t* W = p.W + e * p.stride_w;
    uint8_t* Q = p.Q + e * p.stride_q;
    const int64_t r0 = n0 + (tid >> 4), k = b * 128 + 8 * (tid & 15);
    u32x4 v[8];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 16 * i;
        v[i] = r < p.N ? f8_load(W + r * p.ldw, k, p.K) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = magnitude8(v[i], amax);
    amax = wave_max(amax);
    if ((tid & 63) == 0) part[tid >> 6] = amax;
    __syncthreads();
    const F8Scale c = f8_scale(max(max(part[0], part[1]), max(part[2], part[3])));
    if (tid == 0) p.S[e * p.stride_s + n0 / 128 * p.lds + b] = c.s;
    const int64_t padded = f8_padded(p.K, p.ldq);
    const bool wide = ((reinterpret_cast<uintptr_t>(Q) | (uintptr_t)p.ldq) & 7) == 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 16 * i;
        if (r < p.N) f8_store(Q + r * p.ldq, k, padded, f8_codes8(v[i], c), wide);
    }
}

// a launch holds at most 2^32 - 1 threads: 2^24 - 1 workgroups of 256
constexpr int64_t kMostGroups = (int64_t(1) << 24) - 1;

hipError_t launch_f8_quantize(const uint16_t* X, int64_t R, int64_t K, int64_t ldx, uint8_t* Q, int64_t ldq, float* S,
                              int64_t lds, hipStream_t s) {
    const int64_t groups_k = (K + 511) / 512;
    auto run = [&](auto kernel, int64_t rows) {  // rows a workgroup
        const int64_t most = kMostGroups / groups_k * rows;
        for (int64_t r = 0; r < R; r += most) {
            const int64_t n = R - r < most ? R - r : most;
            kernel<<<(unsigned)((n + rows - 1) / rows * groups_k), 256, 0, s>>>(X + r * ldx, n, K, ldx, Q + r * ldq, ldq,
                                                                             S + r, lds, (int)groups_k);
        }
    };
    if (groups_k > kMostGroups) return hipErrorInvalidValue;
    if (R * groups_k <= 2048)
        run(f8_quantize_kernel<1>, 4);
    else
        run(f8_quantize_kernel<4>, 16);
    return hipGetLastError();
}

hipError_t launch_f8_quantize_weight(const F8WeightArgs& a, hipStream_t s) {
    const int64_t nb = (a.N + 127) / 128, kb = (a.K + 127) / 128, per = nb * kb;
    if (per > kMostGroups) return hipErrorInvalidValue;
    const int64_t most = kMostGroups / per;  // matrices a launch
    for (int64_t e = 0; e < a.E; e += most) {
        F8WeightArgs p = a;
        p.E = a.E - e < most ? a.E - e : most;
        p.W += e * a.stride_w;
        p.Q += e * a.stride_q;
        p.S += e * a.stride_s;
        f8_quantize_weight_kernel<<<(unsigned)(p.E * per), 256, 0, s>>>(p, nb, kb);
    }
    return hipGetLastError();
}

}  // namespace glk
