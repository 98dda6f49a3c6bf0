// Matrix kernels of the 8-bit and training products for gfx950, on MFMA tiles.
//
// One k-step is 64 bytes of the summed index: 64 codes or 32 bf16 values, one
// v_mfma_i32_16x16x64_i8 or v_mfma_f32_16x16x32_bf16 for each 16 x 16 output block (16 bytes of each
// operand per lane, the same cycles, the same accumulator layout). An operand comes in one of two
// forms, and every product is a pair of them:
//   contiguous: the summed index is contiguous in memory (codes; dC and B of dA = dC B^T). A slot of
//     its LDS ring holds half of the tile's rows, 128 bytes (two k-steps) of each, so that copies
//     read whole lines: with one k-step of all rows, 64-byte rows, every line crossed the L1 twice
//     (8-bit 4096 x 4096 x 11008: 152 us against 124). 16-byte chunk c of row r is stored at c ^
//     ((r >> 1) & 7): the 16 rows that one cycle of a ds_read_b128 serves cover all 64 banks.
//   strided: the summed index is the row (A and dC of dB = A^T dC; B of the forward). A slot holds one
//     k-step, 32 rows of R elements, and ds_read_b64_tr_b16 transposes 4 x 16 blocks on the way to
//     registers; the 32-byte column groups of row k are stored at group ^ s(k), s(k) = (k & 3) | ((k >>
//     1) & 4).
// Both take 64 R bytes a slot. Slots are filled HBM -> LDS without registers, in rings of 5 for each
// operand: 160 KB for the 256 x 256 tile, 80 KB (two workgroups a CU) for 128 x 128, 40 KB for 64 x 64.
//
// Schedules. 256 x 256 (op_pp_kernel): two groups of four waves, one of each group on every SIMD; in
// turn one group reads its operands and issues copies while the other runs 32 MFMAs back to back, and
// they swap at each barrier. 128 x 128 and 64 x 64 (op_small): four waves in step, operands double-buffered
// in registers, K split over idle CUs with partial sums in a workspace that the last arriver adds in
// order (the same bits on every run; integer sums are exact in any order).
//
// Epilogues round once to bf16, staged through LDS so that each row segment is written by one
// instruction. Codes: the 32-bit sum times the row's and the column's scale in float32, and for the
// gated form silu(g) u. Training forward: g and u, then silu(g) u from their float32 values.
// Codes past K in the last 16-byte chunk of a row are whatever the caller's padding holds: they are
// cleared in the A operand, which is enough, as 0 times any code is 0.
//
// Measured, 256 x 256 tiles, medians of the kernel once the clock has settled: 8-bit 4096 x 4096 x 11008
// 127 us, 2.9 POP/s of the 4.0 that the matrix cores reach on random codes in registers; dA = dC B^T 4096
// x 4096 x 22016 484 us, 1.53 PFLOP/s of 2.0; of dB = A^T dC 4096 x 22016 x 4096 the 1280 tiles of its full
// waves 558 us, 1.23, and as many of the forward 542 us, 1.27 (after an idle spell 130, 486, 577 and 578). What bounds them, from timing-only
// copies that leave one part out (us, in that order, the whole 124, 470, 556, and 666 for the forward's
// 1376 tiles): without the copies 105, 362, 443, 478; without the operand reads 113, 469, 451, 641;
// without the MFMAs 84, 430, 360, 474; the operand reads alone 59, 187, 280, 273. dA waits
// mostly for its copies (32 KB a k-step from the L2 into each CU); in the others copies and MFMAs weigh
// alike, and in dB the reads too: a transposing read of a k-step's operands takes 0.44 us, a plain one 0.27.
// Where the copied lines come from does not matter (all tiles on the same panels: dA 459, dB 552), nor
// do wave priorities, copies issued before the reads, or tile rows walked in groups of 8 for 4 (all
// within 1%). Four waves of 128 x 128, which read a third less from LDS, gained nothing (dB 597-608
// against 599).

#include <type_traits>

#include "common.h"
#include "ops.h"
#include "ops_math.h"

namespace glk {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;

template <int BM_, int BN_, int WM, int WN, int MODE>
struct OpTile {
    static constexpr int BM = BM_, BN = BN_;
    static constexpr bool I8 = MODE == kOpI8;
    static constexpr bool A_CONTIG = MODE != kOpAtb;
    static constexpr bool B_CONTIG = MODE == kOpI8 || MODE == kOpAbt;
    static constexpr int ES = I8 ? 1 : 2;            // bytes per element
    static constexpr int KE = 64 / ES;               // elements per k-step
    static constexpr int SLOTS = 5;
    static constexpr int NW = WM * WN;
    static constexpr int WTM = BM / WM, WTN = BN / WN;
    static constexpr int TM = WTM / 16, TN = WTN / 16;
    static constexpr int A_BYTES = BM * 64, B_BYTES = BN * 64;  // one slot of each ring
    static constexpr int B_RING = SLOTS * A_BYTES;
    static constexpr int LDS_BYTES = SLOTS * (A_BYTES + B_BYTES);
    static constexpr int A_PW = A_BYTES / 1024 / NW;  // 1 KB copy instructions per wave and stage
    static constexpr int B_PW = B_BYTES / 1024 / NW;
    static constexpr int LOADS = A_PW + B_PW;
    using Acc = std::conditional_t<I8, i32x4, f32x4>;
    static_assert(A_PW * NW * 1024 == A_BYTES && B_PW * NW * 1024 == B_BYTES, "copies split evenly");
    static_assert(LDS_BYTES <= 160 * 1024, "LDS");
};

// strided operands of R columns: physical 32-byte column group of logical group u in row k (R = 64
// has four groups a row and two rows in the 256 bytes of all banks)
template <int R>
__device__ __forceinline__ int op_group(int u, int k) {
    return u ^ (R >= 128 ? ((k & 3) | ((k >> 1) & 4)) : (k & 3));
}

__device__ __forceinline__ f32x4 op_mfma(const u32x4& x, const u32x4& y, const f32x4& c) {
    return mfma16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c);
}
__device__ __forceinline__ i32x4 op_mfma(const u32x4& x, const u32x4& y, const i32x4& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, x), __builtin_bit_cast(i32x4, y), c, 0, 0, 0);
}

__device__ __forceinline__ int op_wrap(int slot) { return slot >= 5 ? slot - 5 : slot; }

// The copies of one operand (R rows or columns of the tile from r0, `rows` of them in all) by one
// wave: PW instructions of 1 KB for one slot. Issue number u fills slot u % 5: of a contiguous
// operand with half u & 1 of the rows, 128 bytes (two k-steps, u / 2) of each; of a strided one with
// the 32 rows of k-step u.
template <int R, int PW, bool CONTIG, int ES, bool GLU, int WT>
struct OpCopy {
    static constexpr int HALVES = CONTIG ? 2 : 1;
    uint32_t off[HALVES][PW];  // byte offset of the lane's 16 bytes, or kBufInvalid outside the matrix
    int chunk[PW];             // contiguous: byte of the lane's chunk in the 128-byte row
    const char* base[GLU && CONTIG ? HALVES * PW : 1];
    int64_t ld_bytes;
    int sum;                   // bytes (contiguous) or rows (strided) of the summed index

    // gated operands hold gate rows (columns) and, `up` of them later, the up ones; the tile's WT-wide
    // share of each wave is WT / 2 gate and the same WT / 2 up
    __device__ __forceinline__ void init(const void* p, int64_t ld, int64_t r0, int64_t rows, int up, int64_t k0,
                                         int k_count, int wave, int lane) {
        ld_bytes = ld * ES;
        sum = CONTIG ? k_count * ES : k_count;
        const char* at = static_cast<const char*>(p) + k0 * (CONTIG ? ES : ld_bytes);
#pragma unroll
        for (int i = 0; i < PW; ++i)  // row 8 idx + lane / 8, of which (row >> 1) & 7 is ...
            chunk[i] = 16 * ((lane & 7) ^ (4 * ((wave * PW + i) & 1) + (lane >> 4)));
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
#pragma unroll
            for (int i = 0; i < PW; ++i) {
                const int idx = wave * PW + i;
                if constexpr (CONTIG) {
                    const int q = h * (R / 2) + 8 * idx, r = q + (lane >> 3);
                    if constexpr (GLU) {  // 8 rows are all gate or all up: one base for the instruction
                        const int out = (q / WT) * (WT / 2) + q % (WT / 2);
                        const int64_t src = r0 + out + (q % WT < WT / 2 ? 0 : up);
                        base[h * PW + i] = at + src * ld_bytes;
                        off[h][i] = sel_off(r0 + out + (lane >> 3) < rows,
                                            (uint32_t)((lane >> 3) * (int)ld_bytes + chunk[i]));
                    } else {
                        off[h][i] = sel_off(r0 + r < rows, (uint32_t)(r * (int)ld_bytes + chunk[i]));
                    }
                } else {
                    constexpr int RPI = 512 / R, CH = R / 8;  // k rows per instruction, chunks per row
                    const int k = idx * RPI + lane / CH, pc = lane % CH;
                    const int col = 16 * op_group<R>(pc >> 1, k) + 8 * (pc & 1);
                    int src = col, out = col;
                    if constexpr (GLU) {
                        const int q = col % WT;
                        out = (col / WT) * (WT / 2) + q % (WT / 2);
                        src = out + (q < WT / 2 ? 0 : up);
                    }
                    off[h][i] = sel_off(r0 + out < rows, (uint32_t)(k * (int)ld_bytes + src * ES));
                }
            }
        if constexpr (!(GLU && CONTIG)) base[0] = at + (CONTIG ? r0 * ld_bytes : r0 * ES);
    }
    // issue number u with u & 1 == H (a constant where it matters) into the slot at LDS address `lds`
    template <int H>
    __device__ __forceinline__ void issue(int u, uint32_t lds, int wave) const {
        if constexpr (CONTIG) {
            const int at = (u >> 1) * 128, left = sum - at;  // left <= 0: zeros
            const int from = left > 0 ? at : 0;
#pragma unroll
            for (int i = 0; i < PW; ++i) {
                const i32x4 r = rsrc_words(base[GLU ? H * PW + i : 0] + from, kBufRecords);
                dma16(r, lds + (wave * PW + i) * 1024, sel_off(chunk[i] < left, off[H][i]));
            }
        } else {
            const int at = u * 32;
            const int krows = __builtin_amdgcn_readfirstlane(max(min(sum - at, 32), 0));
            const i32x4 r = rsrc_words(base[0] + (krows > 0 ? at : 0) * ld_bytes, (uint32_t)krows * (uint32_t)ld_bytes);
#pragma unroll
            for (int i = 0; i < PW; ++i) dma16(r, lds + (wave * PW + i) * 1024, off[0][i]);
        }
    }
};

// The operands of k-step t (t % 5 == slot, t & 1 == P) from one ring: T tiles of 16 rows (columns)
// from `w0`. Lane l gets row w0 + 16 i + (l & 15), bytes 16 (l >> 4) .. + 15 of the k-step.
template <int R, int T, bool CONTIG, int P>
__device__ __forceinline__ void op_read(const char* ring, int slot, int w0, int lane, u32x4 (&f)[T]) {
    const int j = lane & 15, G = lane >> 4;
    if constexpr (CONTIG) {
        const int at = op_wrap(slot + (w0 >= R / 2 ? 1 : 0) + (P ? 4 : 0));  // unit (t - P) + half
        const char* row = ring + at * (64 * R) + (w0 % (R / 2) + j) * 128 + 16 * ((4 * P + G) ^ (j >> 1));
#pragma unroll
        for (int i = 0; i < T; ++i) f[i] = *reinterpret_cast<const u32x4*>(row + i * 2048);
    } else {
        const char* stage = ring + slot * (64 * R);
#pragma unroll
        for (int i = 0; i < T; ++i) {
            i16x4 v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = 8 * G + 4 * h + (j >> 2);
                const char* at = stage + k * (2 * R) + 32 * op_group<R>((w0 >> 4) + i, k) + 8 * (j & 3);
                v[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)at);
            }
            const i16x8 x = {v[0][0], v[0][1], v[0][2], v[0][3], v[1][0], v[1][1], v[1][2], v[1][3]};
            f[i] = __builtin_bit_cast(u32x4, x);
        }
    }
}

// Waits until this wave's copies for the next k-step have landed, in a step (parity P) that issued
// A's slot and then B's. A strided operand's were issued three whole steps before this one's last; a
// contiguous one's second half in the step before, and only odd steps are followed by a new pair.
template <class T, int P>
__device__ __forceinline__ void op_wait() {
    if constexpr (T::A_CONTIG && T::B_CONTIG) {
        if constexpr (P == 1) wait_vmcnt<T::LOADS>();
    } else if constexpr (T::A_CONTIG) {
        if constexpr (P == 1)
            wait_vmcnt<T::LOADS + T::B_PW>();
        else
            wait_vmcnt<3 * T::LOADS>();
    } else {
        wait_vmcnt<3 * T::LOADS>();
    }
}

// clears the codes at `left` and after in a fragment of the last k-step
template <int T>
__device__ __forceinline__ void op_clear_tail(int left, int lane, u32x4 (&f)[T]) {
    const int n = left - 16 * (lane >> 4);  // codes of the lane's 16 that count
    u32x4 mask;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const int b = n - 4 * w;
        mask[w] = b >= 4 ? 0xFFFFFFFFu : (b <= 0 ? 0u : (1u << (8 * b)) - 1u);
    }
#pragma unroll
    for (int i = 0; i < T; ++i) f[i] &= mask;
}

struct OpPlace {
    int m0, n0, piece, tile;
};
// which tile, in grouped order over the XCDs' contiguous shares
template <int BM, int BNO>
__device__ __forceinline__ OpPlace op_place(const OpTileArgs& p, int block) {
    const int pieces = p.splits, ntiles = p.tiles_m * p.tiles_n;
    const int unit = xcd_remap(block, ntiles * pieces, p.nxcd);
    const int tile = unit / pieces;
    const int per_group = p.group_m * p.tiles_n;
    const int g = tile / per_group, first = g * p.group_m;
    const int gm = min(p.tiles_m - first, p.group_m);
    const int in = tile - g * per_group;
    // (uniform, but the divisions leave them in vector registers)
    auto uni = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    return OpPlace{uni((first + in % gm) * BM), uni((in / gm) * BNO), uni(unit - tile * pieces), uni(tile)};
}

// ---- epilogue ------------------------------------------------------------------------------------
// Lane layout of acc[ni][mi][r]: row wm WTM + 16 mi + (lane & 15), column wn WTN + 16 ni + 4 (lane >> 4) + r.
// Each wave rounds its block into an LDS area of its own (rows of RB bytes, 16-byte chunk c of row r
// at c ^ (r & (RB / 16 - 1))) and writes it out in whole row segments.

// Writes the wave's staged WTM x W block in 16-byte stores: `vec` aligned ones, else (rows of C without
// 16-byte alignment) ones at any address, and the row's last elements one by one (codes 2000 x 4001 x
// 1024 15.5 us, 18.2 with 2-byte stores).
template <int WTM, int W>
__device__ __forceinline__ void op_store_rows(const char* ob, uint16_t* C, int64_t ldc, int m0, int M, int n0, int N,
                                              int lane, bool vec) {
    constexpr int RB = W * 2, CPR = RB / 16, ROWS = 64 / CPR;
    if (vec) {
        const int lr = lane / CPR, lc = lane % CPR, n = n0 + lc * 8;
        const __amdgpu_buffer_rsrc_t rc = make_rsrc(C + (size_t)m0 * ldc);
#pragma unroll
        for (int s = 0; s < WTM / ROWS; ++s) {
            const int r = s * ROWS + lr;
            const u32x4 v = *reinterpret_cast<const u32x4*>(ob + r * RB + (lc ^ (r & (CPR - 1))) * 16);
            // non-temporal: written once, and far larger than the L2s when it is large
            __builtin_amdgcn_raw_buffer_store_b128(
                v, rc, m0 + r < M && n < N ? (uint32_t)(r * (int)ldc + n) * 2u : kBufInvalid, 0, kAuxNonTemporal);
        }
    } else {
        const int lr = lane / CPR, lc = lane % CPR, left = N - (n0 + lc * 8);
#pragma unroll
        for (int s = 0; s < WTM / ROWS; ++s) {
            const int r = s * ROWS + lr;
            const u32x4 v = *reinterpret_cast<const u32x4*>(ob + r * RB + (lc ^ (r & (CPR - 1))) * 16);
            if (m0 + r < M) store8(C + (size_t)(m0 + r) * ldc + n0 + lc * 8, v, left);
        }
    }
}

template <class T, int MODE, bool GLU>
__device__ __forceinline__ void op_epilogue(const OpTileArgs& p, char* lds, const OpPlace& at, int wave, int wm, int wn,
                                            int lane, typename T::Acc (&acc)[T::TN][T::TM]) {
    constexpr int TM = T::TM, TN = T::TN, TNO = GLU ? TN / 2 : TN, WTNO = TNO * 16;
    const int row = lane & 15, G = lane >> 4;
    const int mw = at.m0 + wm * T::WTM, nw = at.n0 + wn * WTNO;  // the wave's first row and output column
    char* ob = lds + wave * (T::WTM * T::WTN * 2);
    auto put = [&](auto width, int mi, int ni, const f32x4& h) {
        constexpr int RB = decltype(width)::value * 2;
        const int r = mi * 16 + row, byte = ni * 32 + G * 8;
        *reinterpret_cast<u32x2*>(ob + r * RB + (((byte >> 4) ^ (r & (RB / 16 - 1))) << 4) + (byte & 15)) =
            u32x2{pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3])};
    };
    using Full = std::integral_constant<int, T::WTN>;
    using Out = std::integral_constant<int, WTNO>;
    if constexpr (MODE == kOpI8) {
        float sa[TM];
#pragma unroll
        for (int mi = 0; mi < TM; ++mi) {
            const int m = mw + mi * 16 + row;
            sa[mi] = m < p.M ? p.sa[m] : 0.f;
        }
#pragma unroll
        for (int ni = 0; ni < TNO; ++ni) {
            f32x4 sg, su;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int n = nw + ni * 16 + 4 * G + r;
                sg[r] = n < p.N ? p.sb[n] : 0.f;
                if constexpr (GLU) su[r] = n < p.N ? p.sb[(int64_t)p.up + n] : 0.f;
            }
#pragma unroll
            for (int mi = 0; mi < TM; ++mi) {
                f32x4 h;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    h[r] = (float)acc[ni][mi][r] * sa[mi] * sg[r];
                    if constexpr (GLU) h[r] = op_swiglu(h[r], (float)acc[ni + TNO][mi][r] * sa[mi] * su[r]);
                }
                put(Out{}, mi, ni, h);
            }
        }
    } else {
        if constexpr (MODE == kOpTrain) {
#pragma unroll
            for (int mi = 0; mi < TM; ++mi)
#pragma unroll
                for (int ni = 0; ni < TN; ++ni) put(Full{}, mi, ni, acc[ni][mi]);
            // rows of WTNO gate and WTNO up values: two row segments
            constexpr int RB = T::WTN * 2, CPR = RB / 16, ROWS = 64 / CPR;
            const int lr = lane / CPR, lc = lane % CPR;
            const int n = nw + (lc % (CPR / 2)) * 8;
            const int64_t col = (lc < CPR / 2 ? 0 : (int64_t)p.up) + n;
            const __amdgpu_buffer_rsrc_t rg = make_rsrc(p.GU + (size_t)mw * p.ldgu);
#pragma unroll
            for (int s = 0; s < T::WTM / ROWS; ++s) {
                const int r = s * ROWS + lr;
                const u32x4 v = *reinterpret_cast<const u32x4*>(ob + r * RB + (lc ^ (r & (CPR - 1))) * 16);
                const bool ok = mw + r < p.M && n < p.N;
                __builtin_amdgcn_raw_buffer_store_b128(v, rg, ok ? (uint32_t)(r * p.ldgu + (int)col) * 2u : kBufInvalid,
                                                       0, kAuxNonTemporal);
            }
        }
#pragma unroll
        for (int mi = 0; mi < TM; ++mi)
#pragma unroll
            for (int ni = 0; ni < TNO; ++ni) {
                if constexpr (GLU)
                    {
                    f32x4 h;
#pragma unroll
                    for (int r = 0; r < 4; ++r) h[r] = op_swiglu(acc[ni][mi][r], acc[ni + TNO][mi][r]);
                    put(Out{}, mi, ni, h);
                }
                else
                    put(Out{}, mi, ni, acc[ni][mi]);
            }
    }
    op_store_rows<T::WTM, WTNO>(ob, p.C, p.ldc, mw, p.M, nw, p.N, lane, MODE != kOpI8 || p.vec != 0);
}

// ---- 256 x 256: two wave groups alternating memory and MFMA phases --------------------------------
// Phases are separated by workgroup barriers b1, b2, ...; group 0 runs the memory phase of step t
// before b(2 t + 1) and its MFMAs before b(2 t + 2), group 1 one barrier later, so every read of step
// t - 1 is over at b(2 t), before either group's memory phase of step t. That phase refills: a strided
// operand's slot of step t - 1 with step t + 4; a contiguous one's slot of unit t - 2 (of steps t - 2
// and t - 1 for even t, t - 3 and t - 2 for odd t) with unit t + 3. Each wave ends its memory phase
// waiting for its own copies that step t + 1 reads, and a barrier follows before any wave reads them.
template <int MODE, bool GLU>
__global__ void __attribute__((amdgpu_flat_work_group_size(512, 512), amdgpu_waves_per_eu(2, 2)))
op_pp_kernel(OpTileArgs p) {
    using T = OpTile<256, 256, 2, 4, MODE>;
    constexpr int TM = T::TM, TN = T::TN;
    // issue number of step t: t + 3 (contiguous) or t + 4 (strided)
    constexpr int A_AHEAD = T::A_CONTIG ? 3 : 4, B_AHEAD = T::B_CONTIG ? 3 : 4;
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int grp = wave >> 2, wm = grp, wn = wave & 3;
    const OpPlace at = op_place<256, GLU ? 128 : 256>(p, (int)blockIdx.x);
    const int nsteps = (p.K + T::KE - 1) / T::KE;

    OpCopy<256, T::A_PW, T::A_CONTIG, T::ES, false, T::WTM> ca;
    OpCopy<256, T::B_PW, T::B_CONTIG, T::ES, GLU, T::WTN> cb;
    ca.init(p.A, p.lda, at.m0, p.M, 0, 0, p.K, wave, lane);
    cb.init(p.B, p.ldb, at.n0, p.N, p.up, 0, p.K, wave, lane);
    const uint32_t ring = lds_addr(lds);
    auto issue_a = [&](auto h, int u, int slot) {
        ca.template issue<decltype(h)::value>(u, ring + slot * T::A_BYTES, wave);
    };
    auto issue_b = [&](auto h, int u, int slot) {
        cb.template issue<decltype(h)::value>(u, ring + T::B_RING + slot * T::B_BYTES, wave);
    };
    typename T::Acc acc[TN][TM];
#pragma unroll
    for (int ni = 0; ni < TN; ++ni)
#pragma unroll
        for (int mi = 0; mi < TM; ++mi) acc[ni][mi] = typename T::Acc{};
    auto phase_barrier = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    const int tail = (T::I8 && (p.K & 15)) ? nsteps - 1 : -1;
    using P0 = std::integral_constant<int, 0>;
    using P1 = std::integral_constant<int, 1>;

    // as steps -4 .. -1 would issue, in their order
    if (!T::A_CONTIG) issue_a(P0{}, 0, 0);
    if (!T::B_CONTIG) issue_b(P0{}, 0, 0);
    issue_a(P0{}, A_AHEAD - 3, A_AHEAD - 3);
    issue_b(P0{}, B_AHEAD - 3, B_AHEAD - 3);
    issue_a(P1{}, A_AHEAD - 2, A_AHEAD - 2);
    issue_b(P1{}, B_AHEAD - 2, B_AHEAD - 2);
    issue_a(P0{}, A_AHEAD - 1, A_AHEAD - 1);
    issue_b(P0{}, B_AHEAD - 1, B_AHEAD - 1);
    op_wait<T, 1>();
    lds_barrier();
    if (grp == 1) phase_barrier();
    int slot = 0;
    auto step = [&](int t, auto par) {
        constexpr int P = decltype(par)::value;
        using H = std::integral_constant<int, 1 - P>;  // parity of t + 3; strided copies have no halves
        u32x4 fa[TM], fb[TN];
        op_read<256, TM, T::A_CONTIG, P>(lds, slot, wm * T::WTM, lane, fa);
        op_read<256, TN, T::B_CONTIG, P>(lds + T::B_RING, slot, wn * T::WTN, lane, fb);
        issue_a(H{}, t + A_AHEAD, op_wrap(slot + A_AHEAD));
        issue_b(H{}, t + B_AHEAD, op_wrap(slot + B_AHEAD));
        if constexpr (T::I8) {
            if (t == tail) op_clear_tail(p.K - t * T::KE, lane, fa);
        }
        op_wait<T, P>();
        wait_lgkmcnt0();
        phase_barrier();
#pragma unroll
        for (int ni = 0; ni < TN; ++ni)
#pragma unroll
            for (int mi = 0; mi < TM; ++mi) acc[ni][mi] = op_mfma(fb[ni], fa[mi], acc[ni][mi]);
        phase_barrier();
        slot = op_wrap(slot + 1);
    };
    int t = 0;
    for (; t + 1 < nsteps; t += 2) {
        step(t, P0{});
        step(t + 1, P1{});
    }
    if (t < nsteps) step(t, P0{});
    if (grp == 0) phase_barrier();
    wait_vmcnt<0>();  // the copies past K included
    lds_barrier();    // the rings are free for the output
    op_epilogue<T, MODE, GLU>(p, lds, at, wave, wm, wn, lane, acc);
}

// ---- 128 x 128 and 64 x 64, K split over idle CUs -------------------------------------------------------------
// Iteration i reads the operands of step i + 1 while the MFMAs of step i run. At its barrier the reads
// of step i, made in iteration i - 1, are over in every wave; after it, a strided operand's slot of
// step i takes step i + 5, and a contiguous one's slot of unit i - 1 (steps i - 1 and i for odd i, i - 2
// and i - 1 for even i) takes unit i + 4. Before the barrier the wave waits for its copies of step i + 1.
// What it has issued by then, up to i + 3 or i + 4, is what the other schedule's step i has, so op_wait
// counts the same.
//
// With one or two tiles a CU what bounds it is the latency of each k-step, not a rate: 509 x 2501 x 1003
// codes 7.7 us, the gated forward 300 x 520 x 328 6.1 us (64 x 64 tiles). It is not a want of bytes in
// flight: 64 x 64 rings of 7, 9 and 13 slots gave 64 x 4096 x 11008 codes 2% at best and cost the other
// small products 2 to 50%, as fewer workgroups fit a CU.
template <int BT, int MODE, bool GLU>
__device__ __forceinline__ void op_small(const OpTileArgs& p, int block, char* lds) {
    using T = OpTile<BT, BT, 2, 2, MODE>;
    constexpr int TM = T::TM, TN = T::TN;
    constexpr int A_AHEAD = T::A_CONTIG ? 4 : 5, B_AHEAD = T::B_CONTIG ? 4 : 5;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const OpPlace at = op_place<BT, GLU ? BT / 2 : BT>(p, block);
    const int total = (p.K + T::KE - 1) / T::KE;
    const int first = at.piece * p.kt_per_split;
    const int nsteps = max(min(total - first, p.kt_per_split), 0);
    const int count = max(min(p.K - first * T::KE, nsteps * T::KE), 0);  // of the summed index

    OpCopy<BT, T::A_PW, T::A_CONTIG, T::ES, false, T::WTM> ca;
    OpCopy<BT, T::B_PW, T::B_CONTIG, T::ES, GLU, T::WTN> cb;
    ca.init(p.A, p.lda, at.m0, p.M, 0, (int64_t)first * T::KE, count, wave, lane);
    cb.init(p.B, p.ldb, at.n0, p.N, p.up, (int64_t)first * T::KE, count, wave, lane);
    const uint32_t ring = lds_addr(lds);
    auto issue_a = [&](auto h, int u, int slot) {
        ca.template issue<decltype(h)::value>(u, ring + slot * T::A_BYTES, wave);
    };
    auto issue_b = [&](auto h, int u, int slot) {
        cb.template issue<decltype(h)::value>(u, ring + T::B_RING + slot * T::B_BYTES, wave);
    };
    typename T::Acc acc[TN][TM];
#pragma unroll
    for (int ni = 0; ni < TN; ++ni)
#pragma unroll
        for (int mi = 0; mi < TM; ++mi) acc[ni][mi] = typename T::Acc{};
    const int tail = (T::I8 && (count & 15)) ? nsteps - 1 : -1;
    auto read = [&](int s, auto par, int slot, u32x4 (&fa)[TM], u32x4 (&fb)[TN]) {
        constexpr int P = decltype(par)::value;
        op_read<BT, TM, T::A_CONTIG, P>(lds, slot, wm * T::WTM, lane, fa);
        op_read<BT, TN, T::B_CONTIG, P>(lds + T::B_RING, slot, wn * T::WTN, lane, fb);
        if constexpr (T::I8) {
            if (s == tail) op_clear_tail(count - s * T::KE, lane, fa);
        }
    };
    using P0 = std::integral_constant<int, 0>;
    using P1 = std::integral_constant<int, 1>;

    // as iterations -5 .. -1 would issue, in their order
    u32x4 fa0[TM], fb0[TN], fa1[TM], fb1[TN];
    if (!T::A_CONTIG) issue_a(P0{}, 0, 0);
    if (!T::B_CONTIG) issue_b(P0{}, 0, 0);
    issue_a(P0{}, A_AHEAD - 4, A_AHEAD - 4);
    issue_b(P0{}, B_AHEAD - 4, B_AHEAD - 4);
    issue_a(P1{}, A_AHEAD - 3, A_AHEAD - 3);
    issue_b(P1{}, B_AHEAD - 3, B_AHEAD - 3);
    issue_a(P0{}, A_AHEAD - 2, A_AHEAD - 2);
    issue_b(P0{}, B_AHEAD - 2, B_AHEAD - 2);
    issue_a(P1{}, A_AHEAD - 1, A_AHEAD - 1);
    issue_b(P1{}, B_AHEAD - 1, B_AHEAD - 1);
    if constexpr (T::A_CONTIG && T::B_CONTIG)
        wait_vmcnt<2 * T::LOADS>();            // units 0 and 1; 2 and 3 may be in flight
    else if constexpr (T::A_CONTIG)
        wait_vmcnt<2 * T::LOADS + T::B_PW>();  // A's units 0 and 1 (B's step 0 before them)
    else
        wait_vmcnt<4 * T::LOADS>();
    lds_barrier();
    read(0, P0{}, 0, fa0, fb0);
    int slot = 0;
    auto step = [&](int i, auto par, u32x4 (&fa)[TM], u32x4 (&fb)[TN], u32x4 (&na)[TM], u32x4 (&nb)[TN]) {
        constexpr int P = decltype(par)::value;
        using H = std::integral_constant<int, P>;  // parity of i + 4
        const int next = op_wrap(slot + 1);
        op_wait<T, P>();  // this wave's copies of step i + 1 landed
        lds_barrier();    // every wave's did, and step i's operands are in registers
        issue_a(H{}, i + A_AHEAD, op_wrap(slot + A_AHEAD));
        issue_b(H{}, i + B_AHEAD, op_wrap(slot + B_AHEAD));
        read(i + 1, std::integral_constant<int, 1 - P>{}, next, na, nb);
#pragma unroll
        for (int ni = 0; ni < TN; ++ni)
#pragma unroll
            for (int mi = 0; mi < TM; ++mi) acc[ni][mi] = op_mfma(fb[ni], fa[mi], acc[ni][mi]);
        slot = next;
    };
    int i = 0;
    for (; i + 1 < nsteps; i += 2) {
        step(i, P0{}, fa0, fb0, fa1, fb1);
        step(i + 1, P1{}, fa1, fb1, fa0, fb0);
    }
    if (i < nsteps) step(i, P0{}, fa0, fb0, fa1, fb1);
    wait_vmcnt<0>();
    lds_barrier();

    if (p.splits > 1) {
        volatile uint32_t& last_flag = *reinterpret_cast<volatile uint32_t*>(lds);
        constexpr uint32_t kSlot = BT * BT * 4;
        const __amdgpu_buffer_rsrc_t ws = make_rsrc(p.ws + (size_t)at.tile * p.splits * (BT * BT));
        auto slot_off = [&](int pc, int ni, int mi) {
            return (uint32_t)pc * kSlot + (uint32_t)((((wave * TN + ni) * TM + mi) * 64 + lane) * 16);
        };
#pragma unroll
        for (int ni = 0; ni < TN; ++ni)
#pragma unroll
            for (int mi = 0; mi < TM; ++mi)
                buf_store16_dev(ws, slot_off(at.piece, ni, mi), __builtin_bit_cast(u32x4, acc[ni][mi]));
        wait_all_memory();
        __syncthreads();
        if (threadIdx.x == 0)
            last_flag = (counter_arrive(&p.counters[at.tile]) == (uint32_t)(p.splits - 1)) ? 1u : 0u;
        __syncthreads();
        if (!last_flag) return;
        if (threadIdx.x == 0) counter_reset(&p.counters[at.tile]);
        typename T::Acc sum[TN][TM];
#pragma unroll
        for (int ni = 0; ni < TN; ++ni)
#pragma unroll
            for (int mi = 0; mi < TM; ++mi) sum[ni][mi] = typename T::Acc{};
        for (int pc = 0; pc < p.splits; ++pc) {  // in K order, its own piece from registers
            if (pc == at.piece) {
#pragma unroll
                for (int ni = 0; ni < TN; ++ni)
#pragma unroll
                    for (int mi = 0; mi < TM; ++mi) sum[ni][mi] += acc[ni][mi];
                continue;
            }
            u32x4 v[TN][TM];
#pragma unroll
            for (int ni = 0; ni < TN; ++ni)
#pragma unroll
                for (int mi = 0; mi < TM; ++mi) v[ni][mi] = buf_load16_dev(ws, slot_off(pc, ni, mi));
#pragma unroll
            for (int ni = 0; ni < TN; ++ni)
#pragma unroll
                for (int mi = 0; mi < TM; ++mi) sum[ni][mi] += __builtin_bit_cast(typename T::Acc, v[ni][mi]);
        }
#pragma unroll
        for (int ni = 0; ni < TN; ++ni)
#pragma unroll
            for (int mi = 0; mi < TM; ++mi) acc[ni][mi] = sum[ni][mi];
        __syncthreads();  // the flag has been read: its place is free for the output
    }
    op_epilogue<T, MODE, GLU>(p, lds, at, wave, wm, wn, lane, acc);
}

template <int BT, int MODE, bool GLU>
__global__ void __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(2, BT == 64 ? 4 : 2)))
op_small_kernel(OpTileArgs p) {
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    op_small<BT, MODE, GLU>(p, (int)blockIdx.x, lds);
}

// Both gradients of a product in one launch: dA = dC B^T first, dB = A^T dC after. They share dC and
// neither fills the card when it is small.
template <int BT>
__global__ void __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(2, BT == 64 ? 4 : 2)))
op_pair_kernel(OpTileArgs pa, OpTileArgs pb) {
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    const int first = pa.tiles_m * pa.tiles_n * pa.splits;
    if ((int)blockIdx.x < first)
        op_small<BT, kOpAbt, false>(pa, (int)blockIdx.x, lds);
    else
        op_small<BT, kOpAtb, false>(pb, (int)blockIdx.x - first, lds);
}

template <int MODE, bool GLU>
static hipError_t launch_mode(int tile, const OpTileArgs& a, int grid, hipStream_t s) {
    if (tile == 256) {
        if (a.splits != 1) return hipErrorInvalidValue;
        op_pp_kernel<MODE, GLU><<<grid, 512, OpTile<256, 256, 2, 4, MODE>::LDS_BYTES, s>>>(a);
    } else if (tile == 128) {
        op_small_kernel<128, MODE, GLU><<<grid, 256, OpTile<128, 128, 2, 2, MODE>::LDS_BYTES, s>>>(a);
    } else {
        op_small_kernel<64, MODE, GLU><<<grid, 256, OpTile<64, 64, 2, 2, MODE>::LDS_BYTES, s>>>(a);
    }
    return hipGetLastError();
}

hipError_t launch_op_tile(int mode, bool glu, int tile, const OpTileArgs& a, int grid, hipStream_t s) {
    switch (mode) {
        case kOpI8: return glu ? launch_mode<kOpI8, true>(tile, a, grid, s) : launch_mode<kOpI8, false>(tile, a, grid, s);
        case kOpAbt: return launch_mode<kOpAbt, false>(tile, a, grid, s);
        case kOpAtb: return launch_mode<kOpAtb, false>(tile, a, grid, s);
        case kOpTrain: return launch_mode<kOpTrain, true>(tile, a, grid, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_op_pair(int tile, const OpTileArgs& a, const OpTileArgs& b, int grid, hipStream_t s) {
    if (tile == 128)
        op_pair_kernel<128><<<grid, 256, OpTile<128, 128, 2, 2, kOpAbt>::LDS_BYTES, s>>>(a, b);
    else
        op_pair_kernel<64><<<grid, 256, OpTile<64, 64, 2, 2, kOpAbt>::LDS_BYTES, s>>>(a, b);
    return hipGetLastError();
}

static hipError_t set_lds(const void* kernel, int bytes) {
    return hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

// (the 64 x 64 kernels ask for 40 KB, which needs no setting)
template <int MODE, bool GLU>
static hipError_t configure_mode() {
    hipError_t e = set_lds((const void*)op_pp_kernel<MODE, GLU>, OpTile<256, 256, 2, 4, MODE>::LDS_BYTES);
    if (e == hipSuccess)
        e = set_lds((const void*)op_small_kernel<128, MODE, GLU>, OpTile<128, 128, 2, 2, MODE>::LDS_BYTES);
    return e;
}

hipError_t configure_op_kernels() {
    hipError_t e = configure_mode<kOpI8, false>();
    if (e == hipSuccess) e = configure_mode<kOpI8, true>();
    if (e == hipSuccess) e = configure_mode<kOpAbt, false>();
    if (e == hipSuccess) e = configure_mode<kOpAtb, false>();
    if (e == hipSuccess) e = configure_mode<kOpTrain, true>();
    if (e == hipSuccess) e = set_lds((const void*)op_pair_kernel<128>, OpTile<128, 128, 2, 2, kOpAbt>::LDS_BYTES);
    return e;
}

}  // namespace glk
