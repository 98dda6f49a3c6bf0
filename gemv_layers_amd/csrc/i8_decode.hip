// 8-bit products of few tokens (M <= 64) for gfx950: C = (Aq Wq^T) sa sw, or its gated form, with each
// byte of the weight read once.
//
// The product is a stream of weight codes. A row of W holds the summed index contiguous, so the 16
// bytes that v_mfma_i32_16x16x64_i8 wants of a lane (row l % 16, codes 16 (l / 16) .. + 15 of a 64-code
// k-step) are 16 contiguous bytes of memory: weights go from HBM to registers in operand order, with
// no LDS and no barrier in the loop. A workgroup takes TN tiles of 16 weight rows (for the gated form
// TN / 2 gate tiles and the up tiles of the same outputs) and one of `pieces` ranges of K; its NW
// waves take contiguous parts of the range and keep D k-steps of weight and activation loads in
// flight. The waves' 32-bit sums meet in LDS, the pieces' in the workspace, where the last arriver
// adds them and returns its counter to zero; integer sums are exact, so the result does not depend
// on the split. Rows past M and N load nothing and store nothing.
//
// FUSED (M = 1): the activations come as bf16, and every workgroup quantises the row itself, with its
// first weight loads already in flight, into LDS, where the loop reads the codes. That is 2 K bytes
// more through the L1 for each workgroup, against a launch and a round trip to memory (us, fused
// against two launches: 11008 x 4096 11.3 and 13.1, 4096 x 11008 12.3 and 13.7, gated 11008 x 4096 18.3 and
// 21.1, 1000 x 1000 4.8 and 7.1; with two rows it lost, 13.6 and 13.2, 15.1 and 13.9).
//
// Bound by the weight's bytes from HBM: one row through 11008 x 4096 codes, 45 MB, takes 10.2 us a call,
// 4.4 TB/s, where a kernel that only reads as many takes 9.3. Non-temporal weight loads cost 1.7 us of
// it, eight tiles a workgroup at 64 rows 25.7 us against 18.5.

#include "codes.h"
#include "common.h"
#include "ops.h"
#include "ops_math.h"

namespace glk {

__device__ __forceinline__ i32x4 i8_mfma(const u32x4& w, const u32x4& a, const i32x4& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, a), c, 0, 0, 0);
}

template <int MT, int TN>
struct I8Stage {
    u32x4 w[TN], a[MT];
};

// Quantises the row p.A16 into `codes` (`pitch` bytes, zeros past K); returns its scale.
template <int NW>
__device__ __forceinline__ float quantise_row(const I8DecodeArgs& p, char* codes, int pitch, uint32_t* part) {
    constexpr int NC = kI8FusedK / (8 * 64 * NW);  // chunks of 8 values a thread
    const int tid = threadIdx.x;
    u32x4 v[NC];
    uint32_t amax = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int k = 8 * (c * 64 * NW + tid);
        v[c] = u32x4{0, 0, 0, 0};
        if (k + 8 <= p.K)
            v[c] = load8(p.A16 + k);
        else if (k < p.K)
            v[c] = load_some(p.A16 + k, p.K - k);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) amax = magnitude8(v[c], amax);
    amax = wave_max(amax);
    if ((tid & 63) == 0) part[tid >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) amax = max(amax, part[w]);
    const CodeScale cs = code_scale(amax);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int k = 8 * (c * 64 * NW + tid);
        if (k < pitch) *reinterpret_cast<u32x2*>(codes + k) = codes8(v[c], cs);
    }
    __syncthreads();
    return cs.s;
}

template <int MT, int TN, int NW, int D, bool GLU, bool FUSED>
__global__ void __launch_bounds__(64 * NW) i8_decode_kernel(I8DecodeArgs p) {
    static_assert(!FUSED || MT == 1, "one row");
    constexpr int NJ = TN * MT;               // 16 x 16 blocks of sums
    constexpr int TO = GLU ? TN / 2 : TN;     // tiles of outputs
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int group = __builtin_amdgcn_readfirstlane((int)blockIdx.x / p.pieces);
    const int piece = (int)blockIdx.x - group * p.pieces;
    // k-steps of this wave, from an even one (a 128-byte line) to an even one
    const int steps = (p.K + 63) / 64, unit = piece * NW + wave, units = p.pieces * NW;
    const int pairs = (steps + 1) / 2;
    const int wb = __builtin_amdgcn_readfirstlane(2 * (int)((int64_t)pairs * unit / units));
    const int we = __builtin_amdgcn_readfirstlane(min(steps, 2 * (int)((int64_t)pairs * (unit + 1) / units)));

    const int i16 = lane & 15, g16 = lane >> 4;
    const int n0 = group * TO * 16;           // first output column
    __amdgpu_buffer_rsrc_t rw[TN];
    uint32_t w_off[TN], a_off[MT];
#pragma unroll
    for (int t = 0; t < TN; ++t) {
        const int n = n0 + 16 * (t % TO);
        rw[t] = make_rsrc(p.W + ((int64_t)n + (t < TO ? 0 : p.N)) * p.ldw);
        w_off[t] = sel_off(n + i16 < p.N, (uint32_t)(i16 * p.ldw + 16 * g16));
    }
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.A);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        a_off[mt] = sel_off(16 * mt + i16 < p.M, (uint32_t)((16 * mt + i16) * p.lda + 16 * g16));

    // (offsets of rows outside stay outside when a step's bytes are added: 2^31 - 16 + K < 2^32)
    char* codes = lds + NW * NJ * 1024;  // FUSED: the row's codes, whole k-steps, after the waves' sums
    __shared__ uint32_t s_part[NW];
    auto load = [&](I8Stage<MT, TN>& st, int s) {
        const bool in = s < we && 64 * s + 16 * g16 < p.K;
#pragma unroll
        for (int t = 0; t < TN; ++t) st.w[t] = buf_load16(rw[t], sel_off(in, w_off[t] + 64u * s));
        if constexpr (!FUSED) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) st.a[mt] = buf_load16(ra, sel_off(in, a_off[mt] + 64u * s));
        }
    };
    i32x4 acc[TN][MT];
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[t][mt] = i32x4{};
    // the codes past K in a row's last 16 bytes are the caller's padding: cleared in A
    const int tail = !FUSED && (p.K & 15) ? steps - 1 : -1;
    auto compute = [&](I8Stage<MT, TN>& st, int s) {
        if constexpr (FUSED) {
            st.a[0] = u32x4{0, 0, 0, 0};
            if (i16 == 0 && s < we) st.a[0] = *reinterpret_cast<const u32x4*>(codes + 64 * s + 16 * g16);
        }
        if (s == tail) {
            const int n = p.K - 64 * s - 16 * g16;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int b = n - 4 * w;
                const uint32_t mask = b >= 4 ? 0xFFFFFFFFu : (b <= 0 ? 0u : (1u << (8 * b)) - 1u);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) st.a[mt][w] &= mask;
            }
        }
#pragma unroll
        for (int t = 0; t < TN; ++t)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) acc[t][mt] = i8_mfma(st.w[t], st.a[mt], acc[t][mt]);
    };
    I8Stage<MT, TN> st[D];
#pragma unroll
    for (int j = 0; j < D; ++j) load(st[j], wb + j);
    float row_scale = 0.f;
    if constexpr (FUSED) row_scale = quantise_row<NW>(p, codes, 64 * steps, s_part);
    for (int s = wb; s < we; s += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            compute(st[j], s + j);
            load(st[j], s + j + D);
        }
    }

    // ---- the waves' sums --------------------------------------------------------------------------
    i32x4* red = reinterpret_cast<i32x4*>(lds);
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) red[((wave * TN + t) * MT + mt) * 64 + lane] = acc[t][mt];
    __syncthreads();
    // block q of outputs (tile q / MT, rows 16 (q % MT) ..): its wave sums it, gate and up together
    constexpr int NQ = TO * MT, QW = (NQ + NW - 1) / NW, H = GLU ? 2 : 1;
    i32x4 sum[QW][H];
#pragma unroll
    for (int e = 0; e < QW; ++e)
#pragma unroll
        for (int h = 0; h < H; ++h) {
            i32x4 x = i32x4{};
            const int q = e * NW + wave;
            if (q < NQ) {
#pragma unroll
                for (int w = 0; w < NW; ++w) x += red[(w * NJ + h * NQ + q) * 64 + lane];
            }
            sum[e][h] = x;
        }
    // lane l holds columns 4 (l / 16) .. + 3 of row l % 16
    auto store_c = [&](int q, const i32x4 (&v)[H]) {
        const int m = 16 * (q % MT) + i16, n = n0 + 16 * (q / MT) + 4 * g16;
        if (m >= p.M || n >= p.N) return;
        const float sa = FUSED ? row_scale : p.sa[m];
        f32x4 y;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int c = min(n + r, p.N - 1);
            y[r] = (float)v[0][r] * sa * p.sb[c];
            if constexpr (GLU) y[r] = op_swiglu(y[r], (float)v[H - 1][r] * sa * p.sb[(int64_t)p.N + c]);
        }
        const u32x2 o = {pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
        uint16_t* c = p.C + (int64_t)m * p.ldc + n;
        if (n + 4 <= p.N) {  // at any element: the store needs no alignment
            typedef uint32_t u32x2_at2 __attribute__((ext_vector_type(2), aligned(2)));
            *reinterpret_cast<u32x2_at2*>(c) = o;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (n + r < p.N) c[r] = (uint16_t)(o[r >> 1] >> (16 * (r & 1)));
        }
    };
    if (p.pieces == 1) {
#pragma unroll
        for (int e = 0; e < QW; ++e)
            if (e * NW + wave < NQ) store_c(e * NW + wave, sum[e]);
        return;
    }
    // ---- the pieces' sums: at device scope, added by the last arriver ------------------------------
    constexpr uint32_t kSlot = NJ * 1024;
    const __amdgpu_buffer_rsrc_t ws = make_rsrc(p.ws + (size_t)group * p.pieces * (kSlot / 4));
    auto at = [&](int pc, int h, int q) { return (uint32_t)pc * kSlot + (uint32_t)(((h * NQ + q) * 64 + lane) * 16); };
#pragma unroll
    for (int e = 0; e < QW; ++e)
#pragma unroll
        for (int h = 0; h < H; ++h)
            if (e * NW + wave < NQ) buf_store16_dev(ws, at(piece, h, e * NW + wave), __builtin_bit_cast(u32x4, sum[e][h]));
    wait_all_memory();
    __syncthreads();
    volatile uint32_t& last_flag = *reinterpret_cast<volatile uint32_t*>(lds);
    if (tid == 0) last_flag = (counter_arrive(&p.counters[group]) == (uint32_t)(p.pieces - 1)) ? 1u : 0u;
    __syncthreads();
    if (!last_flag) return;
    if (tid == 0) counter_reset(&p.counters[group]);
#pragma unroll
    for (int e = 0; e < QW; ++e) {
        const int q = e * NW + wave;
        if (q >= NQ) continue;
        for (int b0 = 0; b0 < p.pieces; b0 += 4) {  // four pieces' loads in flight before their adds
            u32x4 v[4][H];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int h = 0; h < H; ++h)
                    v[u][h] = buf_load16_dev(ws, sel_off(b0 + u < p.pieces && b0 + u != piece, at(b0 + u, h, q)));
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int h = 0; h < H; ++h) sum[e][h] += __builtin_bit_cast(i32x4, v[u][h]);
        }
        store_c(q, sum[e]);
    }
}

// k-steps in flight per wave: 16 KB of weights a workgroup of four waves with one tile or two, a
// step less of four tiles, whose activations are as many loads again
static constexpr int depth(int tn) { return tn == 4 ? 2 : 4; }

// calls f with the kernel and its LDS bytes for a shape that the planner makes, else returns an error
template <int MT, bool FUSED, class F>
static hipError_t with_kernel(bool glu, int tn, int nw, F f) {
#define GLK_DECODE(TN, NW, GLU)           \
    if (glu == GLU && tn == TN && nw == NW) \
        return f(i8_decode_kernel<MT, TN, NW, depth(TN), GLU, FUSED>, NW * TN * MT * 1024);
    GLK_DECODE(1, 4, false)
    GLK_DECODE(1, 8, false)
    GLK_DECODE(2, 4, true)
    if constexpr (MT == 1 && !FUSED) {
        GLK_DECODE(4, 4, false)
    } else if constexpr (!FUSED) {
        GLK_DECODE(2, 4, false)
        GLK_DECODE(4, 8, false)
        GLK_DECODE(4, 4, true)
    }
#undef GLK_DECODE
    return hipErrorInvalidValue;
}

hipError_t launch_i8_decode(bool glu, int mt, int tn, int nw, const I8DecodeArgs& a, int grid, hipStream_t s) {
    auto run = [&](void (*k)(I8DecodeArgs), int lds) {
        if (a.A16) lds += (a.K + 63) / 64 * 64;
        k<<<grid, 64 * nw, lds, s>>>(a);
        return hipGetLastError();
    };
    if (a.A16) return mt == 1 ? with_kernel<1, true>(glu, tn, nw, run) : hipErrorInvalidValue;
    switch (mt) {
        case 1: return with_kernel<1, false>(glu, tn, nw, run);
        case 2: return with_kernel<2, false>(glu, tn, nw, run);
        case 3: return with_kernel<3, false>(glu, tn, nw, run);
        case 4: return with_kernel<4, false>(glu, tn, nw, run);
        default: return hipErrorInvalidValue;
    }
}

// (the others ask for at most 64 KB: the fused ones 24 KB with the codes of a row of kI8FusedK)
hipError_t configure_i8_decode() {
    auto set = [](void (*k)(I8DecodeArgs), int lds) {
        return hipFuncSetAttribute((const void*)k, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    };
    hipError_t e = with_kernel<2, false>(false, 4, 8, set);
    if (e == hipSuccess) e = with_kernel<3, false>(false, 4, 8, set);
    if (e == hipSuccess) e = with_kernel<4, false>(false, 4, 8, set);
    return e;
}

}  // namespace glk
