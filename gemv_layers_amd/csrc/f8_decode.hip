// 8-bit floating-point products of few rows for gfx950, plain (at most 64 rows) or grouped (few rows a group), with
// each byte of a weight read once for every 16, 32 or 64 rows.
//
// As in the integer form (i8_decode.hip) the product is a stream of weight codes, from HBM to registers in operand
// order, with no LDS and no barrier in the loop: a workgroup takes TN tiles of 16 weight rows, all rows of a row tile
// and one of `pieces` ranges of K; its NW waves take contiguous parts of the range and keep D blocks of 128 k of
// weights, activations and scales in flight (lane l: row l % 16, codes 16 (l / 16) .. + 15 of each 64). A block's codes are
// widened to bf16, which holds each of them, for four v_mfma_f32_16x16x32_bf16 a tile: its sum is a float32 one, as the
// general kernel's is, and is added times the two scales. (The 8-bit instruction, one a tile, cuts small products, as f8_tile.hip
// says, and has twice the rate, which a stream does not need: us with it and as here, 1 x 11008 x 4096 12.0 and 12.1, 16 x
// 4096 x 11008 14.5 and 14.6, 32 x 4096 x 11008 17.2 and 16.7, 64 x 11008 x 4096 23.0 and 24.4.) The waves' sums meet in LDS and
// the pieces' in the workspace, added in order: the same bits on every run. Rows past the group's and columns past N load nothing
// and store nothing.
//
// FUSED (one row): the activations come as bf16 and every workgroup quantises the row itself, with its first weight
// loads already in flight, into LDS, where the loop reads codes and scales.
//
// Bound by the weight's stream and the launch. Here and below and in the planner, us a call with weights that come from HBM; in
// brackets with two 45 MB weights in turn, which the 256 MB cache behind the L2s holds: 1 x 11008 x 4096 11.9 (10.5, as a
// bare read of them), 16 x 4096 x 11008 14.4 (13.1), where 256 workgroups, one a CU, of 16 columns over all of K read as many
// bytes of activations through the caches as of weights; 64 x 11008 x 4096 24.6 (21.4) and 64 x 4096 x 11008 24.0 (21.0), 16 products
// of 16 x 16 for each 8 KB of weights and 8 of activations in 172 and 256 workgroups; 64 rows in 41 of 64 groups, 4096 to
// 1376, 42.6 (231 MB, 5.4 TB/s). At a copy's 6.0 TB/s 45 MB take 7.5.

#include "f8.h"
#include "group.h"
#include "ops.h"
#include "ops_math.h"

namespace glk {

template <int MT, int TN>
struct F8Stage {
    u32x4 w[TN][2], a[MT][2];
    float sa[MT], sw;
};

// a block's codes of a lane as bf16, exactly: eight of each half h and quarter q at [2 h + q]
__device__ __forceinline__ void f8_widen(const u32x4 (&v)[2], bf16x8 (&x)[4]) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u32x4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = (int)v[i >> 1][2 * (i & 1) + (j >> 1)];
            const bf16x2 p = (j & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.f, true)
                                     : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.f, false);
            w[j] = __builtin_bit_cast(uint32_t, p);
        }
        x[i] = __builtin_bit_cast(bf16x8, w);
    }
}

// Quantises the row p.A16 into `codes` (whole blocks, zeros past K) and `scales`.
template <int NW>
__device__ __forceinline__ void f8_quantise_row(const F8DecodeArgs& p, char* codes, float* scales, int blocks) {
    constexpr int NC = kF8FusedK / (8 * 64 * NW);  // chunks of 8 values a thread
    const int tid = threadIdx.x;
    u32x4 v[NC];
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
    for (int c = 0; c < NC; ++c) {
        const int k = 8 * (c * 64 * NW + tid);
        const F8Scale s = f8_scale(row_max(magnitude8(v[c], 0)));  // 16 lanes are a block
        if (k < 128 * blocks) {
            *reinterpret_cast<u32x2*>(codes + k) = f8_codes8(v[c], s);
            if ((tid & 15) == 0) scales[k >> 7] = s.s;
        }
    }
    __syncthreads();
}

template <int MT, int TN, int NW, int D, bool FUSED>
__global__ void __launch_bounds__(64 * NW) f8_decode_kernel(F8DecodeArgs p, GroupArgs g) {
    static_assert(!FUSED || MT == 1, "one row");
    constexpr int NJ = TN * MT;  // 16 x 16 blocks of sums
    extern __shared__ __attribute__((aligned(16))) char lds[];
    GroupSpan span;
    if (!find_span(g, 16 * MT, p.strips * p.pieces, EvenUnits{(int)blockIdx.x, p.nxcd}, &span)) return;
    const int tid = threadIdx.x, lane = tid & 63;
    auto uni = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    const int wave = uni(tid >> 6);
    // row tiles of one strip and piece next to each other: they share its weights
    const int in = uni(span.unit / span.tiles), tile = span.unit - in * span.tiles;
    const int strip = uni(in / p.pieces), piece = in - strip * p.pieces;
    const int group = max(span.group, 0);
    const int64_t first = span.first + 16 * MT * tile;  // the row tile's first row
    const int rows = min(span.rows - 16 * MT * tile, 16 * MT);
    const int K = span.group < 0 ? 0 : p.K;
    // blocks of this wave
    const int blocks = (K + 127) / 128, unit = piece * NW + wave, units = p.pieces * NW;
    const int wb = uni((int)((int64_t)blocks * unit / units)), we = uni((int)((int64_t)blocks * (unit + 1) / units));

    const int i16 = lane & 15, g16 = lane >> 4;
    const int n0 = strip * TN * 16;  // first output column
    const uint8_t* W = p.W + group * g.stride_b;
    __amdgpu_buffer_rsrc_t rw[TN];
    uint32_t w_off[TN], a_off[MT];
#pragma unroll
    for (int t = 0; t < TN; ++t) {
        rw[t] = make_rsrc(W + (int64_t)(n0 + 16 * t) * p.ldw);
        w_off[t] = sel_off(n0 + 16 * t + i16 < p.N, (uint32_t)(i16 * p.ldw + 16 * g16));
    }
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.A + first * p.lda);
    const float* sa[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int r = 16 * mt + i16;
        a_off[mt] = sel_off(r < rows, (uint32_t)(r * p.lda + 16 * g16));
        sa[mt] = p.sa + first + min(r, rows - 1);
    }
    // the TN tiles lie within 128 columns
    const float* sw = p.sb + group * g.stride_sb + n0 / 128 * p.ldsb;

    // (offsets of rows outside stay outside when a block's bytes are added: 2^31 - 16 + K < 2^32)
    char* codes = lds + NW * NJ * 1024;  // FUSED: the row's codes, whole blocks, after the waves' sums, then its scales
    float* scales = reinterpret_cast<float*>(codes + 128 * blocks);
    auto load = [&](F8Stage<MT, TN>& st, int b) {
        const int at = min(b, max(we - 1, 0));  // (scales past the wave's blocks: any, not used)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = 128 * b + 64 * h;
            const bool ok = b < we && k + 16 * g16 < K;
#pragma unroll
            for (int t = 0; t < TN; ++t) st.w[t][h] = buf_load16(rw[t], sel_off(ok, w_off[t] + (uint32_t)k));
            if constexpr (!FUSED) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) st.a[mt][h] = buf_load16(ra, sel_off(ok, a_off[mt] + (uint32_t)k));
            }
        }
        if (we > wb) {
            st.sw = sw[at];
            if constexpr (!FUSED) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) st.sa[mt] = sa[mt][at * p.ldsa];
            }
        }
    };
    f32x4 acc[TN][MT];
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[t][mt] = f32x4{0.f, 0.f, 0.f, 0.f};
    // the codes past K in a row's last 16 bytes are the caller's padding, which may hold NaN: cleared in both
    const int tail = K & 15 ? blocks - 1 : -1;
    auto compute = [&](F8Stage<MT, TN>& st, int b) {
        if (b >= we) return;
        if constexpr (FUSED) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                st.a[0][h] = u32x4{0, 0, 0, 0};
                if (i16 == 0) st.a[0][h] = *reinterpret_cast<const u32x4*>(codes + 128 * b + 64 * h + 16 * g16);
            }
            st.sa[0] = scales[b];
        }
        if (b == tail) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int n = K - 128 * b - 64 * h - 16 * g16 - 4 * w;
                    const uint32_t mask = n >= 4 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
#pragma unroll
                    for (int t = 0; t < TN; ++t) st.w[t][h][w] &= mask;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) st.a[mt][h][w] &= mask;
                }
        }
        bf16x8 a[MT][4];
        // the scales' powers of two are applied to the sums first (F8Factor): always, or, where that would be 64 instructions
        // a block, only where a product of scales asks for it (us: 64 x 11008 x 4096 21.1 without, 22.6 always, 21.5 so; 8 x
        // 4096 x 4096 6.0, 6.1, 6.5)
        constexpr bool ASK = MT * TN >= 16;
        float m[MT];
        bool far = !ASK;
        const F8Factor fw = f8_factor(st.sw);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            f8_widen(st.a[mt], a[mt]);
            m[mt] = st.sa[mt] * st.sw;
            if constexpr (ASK) far |= f8_far_product(st.sa[mt], st.sw, m[mt]);
        }
        if constexpr (ASK) far = __ballot(far) != 0;
        if (far) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) m[mt] = f8_factor(st.sa[mt]).m * fw.m;
        }
#pragma unroll
        for (int t = 0; t < TN; ++t) {
            bf16x8 w[4];
            f8_widen(st.w[t], w);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < 4; ++i) x = mfma16(w[i], a[mt][i], x);
                if (far) {
                    const int e = f8_factor(st.sa[mt]).e + fw.e - 254;
#pragma unroll
                    for (int r = 0; r < 4; ++r) x[r] = __builtin_ldexpf(x[r], e);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[t][mt][r] = __builtin_fmaf(x[r], m[mt], acc[t][mt][r]);
            }
        }
    };
    F8Stage<MT, TN> st[D];
#pragma unroll
    for (int j = 0; j < D; ++j) load(st[j], wb + j);
    if constexpr (FUSED) f8_quantise_row<NW>(p, codes, scales, blocks);
    for (int b = wb; b < we; b += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            compute(st[j], b + j);
            load(st[j], b + j + D);
        }
    }

    // ---- the waves' sums, in order ------------------------------------------------------------------
    f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) red[((wave * TN + t) * MT + mt) * 64 + lane] = acc[t][mt];
    __syncthreads();
    // block q of outputs (tile q / MT, rows 16 (q % MT) ..): its wave sums it
    constexpr int QW = (NJ + NW - 1) / NW;
    f32x4 sum[QW];
#pragma unroll
    for (int e = 0; e < QW; ++e) {
        sum[e] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int q = e * NW + wave;
        if (q < NJ) {
#pragma unroll
            for (int w = 0; w < NW; ++w) sum[e] += red[(w * NJ + q) * 64 + lane];
        }
    }
    // lane l holds columns 4 (l / 16) .. + 3 of row l % 16
    auto store_c = [&](int q, const f32x4& y) {
        const int m = 16 * (q % MT) + i16, n = n0 + 16 * (q / MT) + 4 * g16;
        if (m >= rows || n >= p.N) return;
        const u32x2 o = {pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
        uint16_t* c = p.C + (first + m) * p.ldc + n;
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
            if (e * NW + wave < NJ) store_c(e * NW + wave, sum[e]);
        return;
    }
    // ---- the pieces' sums: at device scope, added in order by the last arriver ----------------------
    const int place = (span.tile + tile) * p.strips + strip;
    constexpr uint32_t kSlot = NJ * 1024;
    const __amdgpu_buffer_rsrc_t ws = make_rsrc(p.ws + (size_t)place * p.pieces * (kSlot / 4));
    auto at = [&](int pc, int q) { return (uint32_t)pc * kSlot + (uint32_t)((q * 64 + lane) * 16); };
#pragma unroll
    for (int e = 0; e < QW; ++e)
        if (e * NW + wave < NJ) buf_store16_dev(ws, at(piece, e * NW + wave), f4_bits(sum[e]));
    wait_all_memory();
    __syncthreads();
    volatile uint32_t& last_flag = *reinterpret_cast<volatile uint32_t*>(lds);
    if (tid == 0) last_flag = (counter_arrive(&p.counters[place]) == (uint32_t)(p.pieces - 1)) ? 1u : 0u;
    __syncthreads();
    if (!last_flag) return;
    if (tid == 0) counter_reset(&p.counters[place]);
#pragma unroll
    for (int e = 0; e < QW; ++e) {
        const int q = e * NW + wave;
        if (q >= NJ) continue;
        f32x4 all = {0.f, 0.f, 0.f, 0.f};
        for (int b0 = 0; b0 < p.pieces; b0 += 4) {  // four pieces' loads in flight before their adds
            u32x4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                v[u] = buf_load16_dev(ws, sel_off(b0 + u < p.pieces && b0 + u != piece, at(b0 + u, q)));
#pragma unroll
            for (int u = 0; u < 4; ++u) all += b0 + u == piece ? sum[e] : bits_f4(v[u]);
        }
        store_c(q, all);
    }
}

static constexpr int kWaves = 4;

// Blocks of 128 k in flight per wave: two, and three where a wave has 16 or more and its row and weight tiles are few
// (us with two and three: 41 of 64 groups of 1376 x 4096, 8 blocks a wave, 46.4 and 49.4, 1 x 11008 x 4096, 8 blocks, 11.9 and 12.6; 16 x
// 4096 x 11008, 21 blocks, 15.8 and 14.5, 1 x 4096 x 11008 15.0 and 12.8; four were as three, five slower).
static bool deep(const F8DecodeArgs& a, int mt, int tn) { return mt * tn < 8 && a.K / 128 >= 16 * kWaves * a.pieces; }

// the kernel of a shape that the planner makes, and its LDS bytes, or null
struct F8Decode {
    void (*kernel)(F8DecodeArgs, GroupArgs);
    int lds;
};
template <int MT, int TN, bool FUSED = false>
static F8Decode of(bool deep) {
    constexpr int lds = kWaves * TN * MT * 1024;
    if constexpr (MT * TN < 8)
        if (deep) return {f8_decode_kernel<MT, TN, kWaves, 3, FUSED>, lds};
    return {f8_decode_kernel<MT, TN, kWaves, 2, FUSED>, lds};
}
static F8Decode find(int mt, int tn, bool fused, bool deep) {
    if (fused) return mt != 1 ? F8Decode{} : tn == 1 ? of<1, 1, true>(deep) : tn == 2 ? of<1, 2, true>(deep) : F8Decode{};
    switch (mt * 8 + tn) {
        case 9: return of<1, 1>(deep);
        case 10: return of<1, 2>(deep);
        case 12: return of<1, 4>(deep);
        case 17: return of<2, 1>(deep);
        case 18: return of<2, 2>(deep);
        case 20: return of<2, 4>(deep);
        case 33: return of<4, 1>(deep);
        case 34: return of<4, 2>(deep);
        case 36: return of<4, 4>(deep);
        default: return {};
    }
}

// (at most 64 KB, which needs no setting: with the codes and scales of a row of kF8FusedK the fused ones 25 KB)
hipError_t launch_f8_decode(int mt, int tn, const F8DecodeArgs& a, const GroupArgs& g, int grid, hipStream_t s) {
    const F8Decode k = find(mt, tn, a.A16 != nullptr, deep(a, mt, tn));
    if (!k.kernel) return hipErrorInvalidValue;
    k.kernel<<<grid, 64 * kWaves, k.lds + (a.A16 ? (a.K + 127) / 128 * 132 : 0), s>>>(a, g);
    return hipGetLastError();
}

}  // namespace glk
