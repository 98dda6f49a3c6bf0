// Matrix kernels of the 8-bit floating-point products for gfx950: C = sum over blocks b of 128 k of (A W^T)_b
// sa[b][m] sw[n / 128][b], one weight or one for each group of rows.
//
// A block of the summed index is one v_mfma_f32_16x16x128_f8f6f4 for each 16 x 16 output block, started from
// zero; its four sums a lane are then added to the accumulators times the block's two scales: four float32 FMAs
// (16 cycles of the SIMD's vector unit) beside 32 cycles of its matrix core. Weights are the first operand, so
// that a lane's four sums belong to one row of C and take one factor.
//
// The instruction does not keep every bit of its 128 products: it aligns them in eights and cuts what lies below
// 2^-13 of the largest of eight (measured; a test pins it), so a block's sum is off by at most 7 * 2^-13 of the sum of
// magnitudes, and in the mean far less, cuts of either sign falling on random products: 1.3e-5 of the norm of normal
// products' sums, 5e-5 where magnitudes spread over 2^6, 2.4e-6 less of sums of one sign (float32 sums 1e-8 to 7e-8).
// That is a choice: all 8-bit instructions cut alike, and the 16-bit ones, on codes widened to bf16, sum in float32 at half
// the rate (3.9 and 2.0 PFLOP/s from registers): 4096 x 4096 x 11008 would take 184 us for its MFMAs alone, and takes 147 so.
// Products of few rows, which wait for their weights, have them (f8_decode.hip). Against 64 bits the products' error is
// 0.0017 of their norm, all of it the bf16 output's.
//
// 256 x 256 tiles: copies, LDS rings of 128-byte rows and the two alternating wave groups are those of op_pp in
// ops_tile.h for 64-byte steps of two contiguous operands, of which two make a block: a pair of steps reads the
// block's activations once (both 64-byte halves, the MFMA's 32 bytes a lane: any order of k serves that is the same
// in both operands), and in each step half of the wave's weights. Activations are read in a pair's first step alone, so
// their ring needs four slots for the five of the weights, and the scales fit beside them: those of the tile's rows come
// for each block by a copy of 4 bytes a lane, two blocks in turn, and the weight's, one number for each 128 columns that a
// wave's columns lie within, by a scalar load. 128 x 128 and 64 x 64 tiles: below.
// Codes past K in the last 16-byte chunk of a row are the caller's padding, which may hold NaN: cleared in both
// operands.
//
// us: 4096 x 4096 x 11008 146-150 (2.5 PFLOP/s; the integer form, without FMAs, 127), 8192^3 442 (2.5; a library product
// of one scale for all 2.76). What bounds it, by timing-only copies of the first at 147 that leave one part out: no copies 99,
// no MFMAs 96, no FMAs 123; copies alone 105, MFMAs and FMAs 113, MFMAs and barriers 84. Copies, L2 to LDS at 13 TB/s on
// all CUs, and products with their FMAs take like long and share issue slots: MFMAs are busy 0.60 of the time. (With the
// weight's scales from vector loads in the loop, and so a wait for all copies in every block, 3 us more.)

#include "f8.h"
#include "group_tile.h"

namespace glk {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// WM x WN waves; a wave's columns lie within 128
template <int BM_, int BN_, int WM, int WN>
struct F8Tile {
    static constexpr int BM = BM_, BN = BN_;
    static constexpr int NW = WM * WN;
    static constexpr int WTM = BM / WM, WTN = BN / WN;
    static constexpr int TM = WTM / 16, TN = WTN / 16, HN = TN / 2;  // HN weight tiles a step
    static constexpr int A_SLOTS = 4, B_SLOTS = 5;
    static constexpr int A_BYTES = BM * 64, B_BYTES = BN * 64;  // one slot: half of the rows, 128 bytes of each
    static constexpr int B_RING = A_SLOTS * A_BYTES;
    static constexpr int S_RING = B_RING + B_SLOTS * B_BYTES;  // scales: 256 bytes a wave and block, two blocks
    static constexpr int S_BYTES = NW * 256;
    static constexpr int S_ROWS = BM / NW;                     // rows whose scales a wave copies
    static constexpr int KEPT = S_RING + 2 * S_BYTES;          // F8Again
    static constexpr int LDS_BYTES = KEPT + 256;
    static constexpr int A_PW = A_BYTES / 1024 / NW, B_PW = B_BYTES / 1024 / NW;
    static constexpr int LOADS = A_PW + B_PW;
    using Acc = f32x4;
    static_assert(A_PW * NW * 1024 == A_BYTES && B_PW * NW * 1024 == B_BYTES, "copies split evenly");
    static_assert(WTN <= 128 && S_ROWS <= 64 && LDS_BYTES <= 160 * 1024, "layout");
};

using F8Tile256 = F8Tile<256, 256, 4, 2>;

// T tiles of 16 rows from `w0` (within one half of the R rows) of the block in units `unit` and unit + 1 of a
// ring of SLOTS: both 64-byte halves of the lane's k
template <int R, int SLOTS, int T>
__device__ __forceinline__ void f8_read(const char* ring, int unit_slot, int w0, int lane, u32x4 (&f)[T][2]) {
    const int j = lane & 15, G = lane >> 4;
    int at = unit_slot + (w0 >= R / 2 ? 1 : 0);
    at = at >= SLOTS ? at - SLOTS : at;
    const char* row = ring + at * (64 * R) + (w0 % (R / 2) + j) * 128;
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            f[i][h] = *reinterpret_cast<const u32x4*>(row + i * 2048 + 16 * ((4 * h + G) ^ (j >> 1)));
}

// clears the codes at `left` and after in a block's fragments
template <int T>
__device__ __forceinline__ void f8_clear_tail(int left, int lane, u32x4 (&f)[T][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int n = left - 64 * h - 16 * (lane >> 4);  // codes of the lane's 16 that count
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int b = n - 4 * w;
            const uint32_t mask = b >= 4 ? 0xFFFFFFFFu : (b <= 0 ? 0u : (1u << (8 * b)) - 1u);
#pragma unroll
            for (int i = 0; i < T; ++i) f[i][h][w] &= mask;
        }
    }
}

// A block's product; FAR, times 2^(e - 127) for byte 0 of ew (its weights' rows) and byte MI of ea (its activations').
template <bool FAR, int MI>
__device__ __forceinline__ f32x4 f8_mfma(const u32x4 (&w)[2], const u32x4 (&a)[2], int ew, int ea) {
    const i32x8 x = {(int)w[0][0], (int)w[0][1], (int)w[0][2], (int)w[0][3], (int)w[1][0], (int)w[1][1], (int)w[1][2], (int)w[1][3]};
    const i32x8 y = {(int)a[0][0], (int)a[0][1], (int)a[0][2], (int)a[0][3], (int)a[1][0], (int)a[1][1], (int)a[1][2], (int)a[1][3]};
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    if constexpr (FAR) return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, zero, 0, 0, 0, ew, MI, ea);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, zero, 0, 0, 0, 0, 0, 0);
}

// Each lane copies 4 bytes from descriptor + voff into LDS at lds_base + 4 * lane (as dma16).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma4(const i32x4& rsrc, uint32_t lds_base, uint32_t voff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(lds_base), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// The scales of a block for a wave's row tiles and columns: their products, or, FAR, products of their factors and the
// exponents (F8Factor), those of the rows a byte for each tile.
template <int TM, bool FAR>
struct F8BlockScales {
    static_assert(TM <= 4, "bytes of ea");
    float m[TM];
    int ea, ew;
};

// The scales of a tile: its rows' copied into LDS block by block, the weight's, one for all rows of the wave, by scalar
// loads a block ahead. (A vector load of it in the loop would be one that the compiler waits for, and as it cannot count the
// copies, which are inline assembly, it would wait for all of those too, in every block.)
template <class T>
struct F8Scales {
    typedef const __attribute__((address_space(4))) float* ScalarPtr;
    const float* sa;   // of the wave's rows to copy, block 0
    ScalarPtr sb;      // of the weight's 128 columns, block 0
    int64_t ldsa;
    uint32_t off;      // of the lane's row to copy
    int count;         // blocks
    float next;        // of the weight, for the block that is read next

    __device__ __forceinline__ void init(const F8TileArgs& p, const OpPlace& at, int first, int blocks, int wave, int wn,
                                         int lane) {
        const int row = wave * T::S_ROWS + lane;
        ldsa = p.ldsa;
        if (blocks == 0) first = 0;  // (a piece past the last block: block 0 is copied and not read)
        sa = p.sa + first * ldsa + at.m0;
        off = sel_off(lane < T::S_ROWS && at.m0 + row < p.M, (uint32_t)row * 4u);
        // (past N: any block of the weight, whose columns are not stored)
        const int nb = min((at.n0 + wn * T::WTN) / 128, (p.N - 1) / 128);
        sb = (ScalarPtr)(uintptr_t)(p.sb + nb * p.ldsb + first);
        count = blocks;
        next = sb[0];
    }
    // block b's into place `slot` of the ring
    __device__ __forceinline__ void issue(int b, uint32_t lds, int slot, int wave) const {
        const int from = b < count ? b : 0;  // (a block past the last: any, not read)
        dma4(rsrc_words(sa + from * ldsa, kBufRecords), lds + T::S_RING + slot * T::S_BYTES + wave * 256, off);
    }
    // those of block b, in place `slot`, for rows w0 + 16 mi + (lane & 15). Blocks are read in order.
    template <bool FAR>
    __device__ __forceinline__ void read(const char* lds, int b, int slot, int w0, int lane, F8BlockScales<T::TM, FAR>& s) {
        const float sw = next;
        next = sb[max(min(b + 1, count - 1), 0)];
        if constexpr (FAR) {
            s.ea = 0;
            s.ew = f8_factor(sw).e;
        }
#pragma unroll
        for (int mi = 0; mi < T::TM; ++mi) {
            const int r = w0 + 16 * mi;
            const float v = *reinterpret_cast<const float*>(lds + T::S_RING + slot * T::S_BYTES + (r / T::S_ROWS) * 256 +
                                                            (r % T::S_ROWS + (lane & 15)) * 4);
            if constexpr (FAR) {
                const F8Factor f = f8_factor(v);
                s.m[mi] = f.m * f8_factor(sw).m;
                s.ea |= f.e << (8 * mi);
            } else {
                s.m[mi] = v * sw;
            }
        }
    }
};

// Products of two scales that are no normal numbers, though neither scale is zero, spoil the sums of the tile that has them.
// It is multiplied again, FAR, with the scales' powers of two applied to the sums first, by the matrix instruction. That
// is found from the sums: terms of a product below 2^-126 are below 2^-100 a block, so that sums of 2^-60 and more are right; and
// a product that is infinite makes all sums of its row infinite or NaN. Only where a sum is neither, as in a row of zeros,
// are the tile's scales looked through, all of them in flight by eights (us without and with such a row in every tile: 4096
// x 4096 x 11008 152 and 154, 8192^3 428 and 442, 509 x 2501 x 1003 7.7 and 9.3). us as here, without a second run, and with the
// powers of two in every block: 4096 x 4096 x 11008 147, 145, 158, 8192^3 442, 435, 478, 509 x 2501 x 1003 7.7, 7.4, 7.8 (the
// second run's code costs that, not the look at the sums); with a test of every block's products and branches 4096 x 4096 x
// 11008 180.
// Whether the sums of a wave say so. Rows past M do not count, and columns past N, which nobody stores, are set to NaN.
template <class T>
__device__ __forceinline__ bool f8_suspect(const F8TileArgs& p, const OpPlace& at, int wm, int wn, int lane,
                                           f32x4 (&acc)[T::TN][T::TM]) {
    const int left = p.N - (at.n0 + wn * T::WTN);
    if (left <= 0) return false;
    if (left < T::WTN) {
#pragma unroll
        for (int ni = 0; ni < T::TN; ++ni)
#pragma unroll
            for (int mi = 0; mi < T::TM; ++mi)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (16 * ni + 4 * (lane >> 4) + r >= left) acc[ni][mi][r] = __builtin_nanf("");
    }
    bool bad = false;
#pragma unroll
    for (int mi = 0; mi < T::TM; ++mi) {
        // (of a NaN and a number these give the number: where one of a row's is NaN all are, or infinite)
        float low = __builtin_inff(), high = 0.f;
#pragma unroll
        for (int ni = 0; ni < T::TN; ++ni)
#pragma unroll
            for (int r = 0; r < 4; r += 2) {
                const float v0 = acc[ni][mi][r], v1 = acc[ni][mi][r + 1];
                asm("v_min3_f32 %0, %0, |%1|, |%2|" : "+v"(low) : "v"(v0), "v"(v1));
                if (ni == 0 && r == 0)
                    asm("v_max_f32 %0, |%1|, |%2|" : "=v"(high) : "v"(v0), "v"(v1));
                else
                    asm("v_max3_f32 %0, %0, |%1|, |%2|" : "+v"(high) : "v"(v0), "v"(v1));
            }
        bad |= at.m0 + wm * T::WTM + 16 * mi + (lane & 15) < p.M && !(low >= 0x1p-60f && high < __builtin_inff());
    }
    return __ballot(bad && 4 * (lane >> 4) < left) != 0;
}
// Whether any wave of the workgroup says yes. `word`: a place of its own for each call, in the waves' areas of the scales'
// ring, which the output does not use. A barrier.
template <class T>
__device__ __forceinline__ bool f8_any(bool yes, char* lds, int wave, int lane, int word) {
    *reinterpret_cast<uint32_t*>(lds + T::S_RING + 256 * wave + 4 * word) = yes;
    lds_barrier();
    return __ballot(*reinterpret_cast<const uint32_t*>(lds + T::S_RING + 256 * (lane % T::NW) + 4 * word) != 0) != 0;
}
// Whether a product of the tile's scales, `blocks` blocks from `first`, is no normal number and no zero for a zero scale.
// The whole workgroup calls it.
template <class T>
__device__ __forceinline__ bool f8_far_scales(const F8TileArgs& p, const OpPlace& at, int first, int blocks, char* lds,
                                              int wave, int lane) {
    constexpr int PARTS = 64 * T::NW / T::BM, U = 8;  // a thread takes one row and every PARTS-th block, U loads in flight
    constexpr int NB = (T::BN + 127) / 128;
    const int row = (int)threadIdx.x % T::BM, part = (int)threadIdx.x / T::BM, nb = at.n0 / 128;
    bool far = false;
    if (at.m0 + row < p.M) {
        const float* sa = p.sa + first * p.ldsa + at.m0 + row;
        for (int b0 = part; b0 < blocks; b0 += U * PARTS) {
            float a[U], w[NB][U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int b = b0 + u * PARTS;
                a[u] = b < blocks ? sa[b * p.ldsa] : 0.f;
#pragma unroll
                for (int j = 0; j < NB; ++j)  // (past N: the last block of columns)
                    w[j][u] = b < blocks ? p.sb[min(nb + j, (p.N - 1) / 128) * p.ldsb + first + b] : 0.f;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < NB; ++j) far |= f8_far_product(a[u], w[j][u], a[u] * w[j][u]);
        }
    }
    return f8_any<T>(__ballot(far) != 0, lds, wave, lane, 1);
}

// What a second run needs is not kept in registers through the first, which has none to spare. The 256 x 256 kernel puts
// it into LDS; the small ones, which that would cost 0.3 us of 7.5, read their arguments again and find the tile again.
struct F8Again {
    F8TileArgs p;
    OpPlace at;

    static __device__ __forceinline__ void keep(char* place, const F8TileArgs& p, const OpPlace& at) {
        static_assert(sizeof(F8Again) % 4 == 0 && sizeof(F8Again) <= 256, "fits its place");
        if (threadIdx.x == 0) *reinterpret_cast<F8Again*>(place) = F8Again{p, at};
    }
    static __device__ __forceinline__ F8Again kept(const char* place) {
        uint32_t from = lds_addr(place);
        asm volatile("" : "+v"(from) : : "memory");  // (not the values that were stored)
        F8Again k;
        uint32_t* to = reinterpret_cast<uint32_t*>(&k);
#pragma unroll
        for (unsigned i = 0; i < sizeof(F8Again) / 4; ++i) to[i] = ((const __attribute__((address_space(3))) uint32_t*)from)[i];
        return k.uniform();
    }
    // (p and g are the kernel's arguments, in this order)
    template <int BT>
    static __device__ __forceinline__ F8Again read() {
        constexpr unsigned N = sizeof(F8TileArgs) / 4, G = sizeof(GroupArgs) / 4;
        static_assert(sizeof(F8TileArgs) % alignof(GroupArgs) == 0, "as they lie in a kernel's argument segment");
        auto from = (const __attribute__((address_space(4))) uint32_t*)__builtin_amdgcn_kernarg_segment_ptr();
        asm volatile("" : "+s"(from));  // (not the values that were read before)
        F8Again k;
        GroupArgs g;
        uint32_t *p = reinterpret_cast<uint32_t*>(&k.p), *groups = reinterpret_cast<uint32_t*>(&g);
#pragma unroll
        for (unsigned i = 0; i < N; ++i) p[i] = from[i];
#pragma unroll
        for (unsigned i = 0; i < G; ++i) groups[i] = from[N + i];
        group_tile<kOpF8, BT>(k.p, g, (int)blockIdx.x, &k.at);
        return k.uniform();
    }

private:
    // (the copies' descriptors are to be in scalar registers)
    __device__ __forceinline__ F8Again uniform() const {
        F8Again k = *this;
        uint32_t* to = reinterpret_cast<uint32_t*>(&k);
#pragma unroll
        for (unsigned i = 0; i < sizeof(F8Again) / 4; ++i) to[i] = __builtin_amdgcn_readfirstlane(to[i]);
        return k;
    }
};

// acc += s (W A) for H weight tiles from tile FROM. Product j + 2 is issued before product j's sums are added,
// so that the FMAs read a result that is two MFMAs old and fit between their issues. (The empty statements and
// scheduling barriers hold that order: left alone, the compiler issues all MFMAs first and runs out of registers.)
template <class T, int FROM, int H, bool FAR>
__device__ __forceinline__ void f8_multiply(const u32x4 (&fb)[H][2], const u32x4 (&fa)[T::TM][2],
                                            const F8BlockScales<T::TM, FAR>& s, f32x4 (&acc)[T::TN][T::TM]) {
    constexpr int N = H * T::TM;
    f32x4 x[3];
    auto product = [&](int j) {
        const int mi = j % T::TM;  // (a constant of the unrolled loop)
        const u32x4(&w)[2] = fb[j / T::TM];
        const u32x4(&a)[2] = fa[mi];
        return mi == 0   ? f8_mfma<FAR, 0>(w, a, s.ew, s.ea)
               : mi == 1 ? f8_mfma<FAR, 1>(w, a, s.ew, s.ea)
               : mi == 2 ? f8_mfma<FAR, 2>(w, a, s.ew, s.ea)
                         : f8_mfma<FAR, 3>(w, a, s.ew, s.ea);
    };
    x[0] = product(0);
    x[1] = product(1);
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (j + 2 < N) x[(j + 2) % 3] = product(j + 2);
        __builtin_amdgcn_sched_barrier(0);
        const int ni = FROM + j / T::TM, mi = j % T::TM;
        float c[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) c[r] = __builtin_fmaf(x[j % 3][r], s.m[mi], acc[ni][mi][r]);
        asm volatile("" : "+v"(c[0]), "+v"(c[1]), "+v"(c[2]), "+v"(c[3]));
        acc[ni][mi] = f32x4{c[0], c[1], c[2], c[3]};
        __builtin_amdgcn_sched_barrier(0);
    }
}

// ---- 256 x 256: two wave groups alternating memory and MFMA phases (op_pp's schedule) ------------------
// Activations' unit u (half of the rows of block u / 2) is read in step u & ~1 alone, at the latest one step
// before op_pp frees its slot: step t refills the slot of unit t - 1 with unit t + 3. The scales of block b + 1
// are issued in the first step of block b, before that step's other copies, and awaited in its second.
template <bool FAR>
__device__ __forceinline__ void f8_pp_sums(const F8TileArgs& p, const OpPlace& at, char* lds,
                                           f32x4 (&acc)[F8Tile256::TN][F8Tile256::TM]) {
    using T = F8Tile256;
    int lane = threadIdx.x & 63;
    if (FAR) asm volatile("" : "+v"(lane));  // (nothing made from it is kept from the first run)
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int grp = wave >> 2, wm = wave & 3, wn = grp;
    const int blocks = (p.K + 127) / 128;

    OpCopy<256, T::A_PW, true, 1, false, T::WTM> ca;
    OpCopy<256, T::B_PW, true, 1, false, T::WTN> cb;
    ca.init(p.A, p.lda, at.m0, p.M, 0, 0, p.K, wave, lane);
    cb.init(p.B, p.ldb, at.n0, p.N, 0, 0, p.K, wave, lane);
    F8Scales<T> sc;
    sc.init(p, at, 0, blocks, wave, wn, lane);
    const uint32_t ring = lds_addr(lds);
    auto issue_a = [&](auto h, int u) { ca.template issue<decltype(h)::value>(u, ring + (u & 3) * T::A_BYTES, wave); };
    auto issue_b = [&](auto h, int u, int slot) {
        cb.template issue<decltype(h)::value>(u, ring + T::B_RING + slot * T::B_BYTES, wave);
    };
    auto phase_barrier = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    int tail = (p.K & 15) ? blocks - 1 : -1;
    asm volatile("" : "+s"(tail));
    using P0 = std::integral_constant<int, 0>;
    using P1 = std::integral_constant<int, 1>;

#pragma unroll
    for (int ni = 0; ni < T::TN; ++ni)
#pragma unroll
        for (int mi = 0; mi < T::TM; ++mi) acc[ni][mi] = f32x4{};
    sc.issue(0, ring, 0, wave);
    issue_a(P0{}, 0);
    issue_b(P0{}, 0, 0);
    issue_a(P1{}, 1);
    issue_b(P1{}, 1, 1);
    issue_a(P0{}, 2);
    issue_b(P0{}, 2, 2);
    wait_vmcnt<T::LOADS>();
    lds_barrier();
    if (grp == 1) phase_barrier();
    int slot = 0;  // of the weights' unit 2 b
    u32x4 fa[T::TM][2];
    F8BlockScales<T::TM, FAR> s;
#pragma clang loop unroll(disable)
    for (int b = 0; b < blocks; ++b) {
        {  // first step: all activations, the first weights
            u32x4 fb[T::HN][2];
            sc.read(lds, b, b & 1, wm * T::WTM, lane, s);
            f8_read<256, 4>(lds, (2 * b) & 3, wm * T::WTM, lane, fa);
            f8_read<256, 5>(lds + T::B_RING, slot, wn * T::WTN, lane, fb);
            sc.issue(b + 1, ring, (b + 1) & 1, wave);
            issue_a(P1{}, 2 * b + 3);
            issue_b(P1{}, 2 * b + 3, op_wrap(slot + 3));
            if (b == tail) {
                f8_clear_tail(p.K - 128 * b, lane, fa);
                f8_clear_tail(p.K - 128 * b, lane, fb);
            }
            wait_lgkmcnt0();
            phase_barrier();
            f8_multiply<T, 0, T::HN, FAR>(fb, fa, s, acc);
            phase_barrier();
        }
        {  // second step: the other weights
            u32x4 fb[T::HN][2];
            f8_read<256, 5>(lds + T::B_RING, slot, wn * T::WTN + T::WTN / 2, lane, fb);
            issue_a(P0{}, 2 * b + 4);
            issue_b(P0{}, 2 * b + 4, op_wrap(slot + 4));
            if (b == tail) f8_clear_tail(p.K - 128 * b, lane, fb);
            wait_vmcnt<T::LOADS>();
            wait_lgkmcnt0();
            phase_barrier();
            f8_multiply<T, T::HN, T::HN, FAR>(fb, fa, s, acc);
            phase_barrier();
        }
        slot = op_wrap(slot + 2);
    }
    if (grp == 0) phase_barrier();
    wait_vmcnt<0>();  // the copies past K included
}

__global__ void __attribute__((amdgpu_flat_work_group_size(512, 512), amdgpu_waves_per_eu(2, 2)))
f8_pp_kernel(F8TileArgs p, GroupArgs g) {
    using T = F8Tile256;
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    OpPlace at;
    if (!group_tile<kOpF8, 256>(p, g, (int)blockIdx.x, &at)) return;
    F8Again::keep(lds + T::KEPT, p, at);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave & 3, wn = wave >> 2;
    f32x4 acc[T::TN][T::TM];
    f8_pp_sums<false>(p, at, lds, acc);
    // (at f8_any's barrier the rings are free for the output)
    if (f8_any<T>(p.K > 0 && f8_suspect<T>(p, at, wm, wn, lane, acc), lds, wave, lane, 0)) {
        const F8Again k = F8Again::kept(lds + T::KEPT);
        if (f8_far_scales<T>(k.p, k.at, 0, (k.p.K + 127) / 128, lds, wave, lane)) {
            lds_barrier();
            f8_pp_sums<true>(k.p, k.at, lds, acc);
            lds_barrier();
        }
    }
    if (p.splits > 1 && !op_join_tile<T>(p, at, lds, wave, lane, acc)) return;
    op_epilogue<T, kOpF8, false>(p, lds, at, wave, wm, wn, lane, acc);
}

// ---- 128 x 128 and 64 x 64, K split over idle CUs --------------------------------------------------------
// Four waves in step, one step a block: iteration b multiplies block b, which is in registers, while block b + 1 comes
// to registers from LDS and block b + 2 to LDS, into the place of block b, whose reads are over in every wave at the
// iteration's barrier. Before it each wave waits for its copies of block b + 1. 34 KB for 64 x 64, four workgroups a CU,
// 66 KB for 128 x 128, two. us: 2048 x 4096 x 11008 91 (2.0 PFLOP/s), 1024 x 4096 x 4096 in two pieces 28, 509 x 2501 x 1003
// 7.7. As first made, against steps of half a block in op_small's rings: 91 and 114, 32.8 and 40.3 whole, 8.3 and 10.5; a third
// block of 64 x 64, three workgroups a CU: 38.8 and 9.0.
template <int BT>
struct F8Small : F8Tile<BT, BT, 2, 2> {
    using Base = F8Tile<BT, BT, 2, 2>;
    static constexpr int BLOCK = BT * 128;  // of either operand
    static constexpr int B_RING = 2 * BLOCK, S_RING = 4 * BLOCK;
    static constexpr int LDS_BYTES = S_RING + 2 * Base::S_BYTES;
    static constexpr int LOADS = 2 * Base::LOADS + 1;  // copies of a wave and block
};

// T tiles of 16 rows from `w0` of a block
template <int T>
__device__ __forceinline__ void f8_read_block(const char* block, int w0, int lane, u32x4 (&f)[T][2]) {
    const int j = lane & 15, G = lane >> 4;
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            f[i][h] = *reinterpret_cast<const u32x4*>(block + (w0 + 16 * i + j) * 128 + 16 * ((4 * h + G) ^ (j >> 1)));
}

// The blocks of a piece: the first, how many, and values of the summed index.
struct F8Piece {
    int first, blocks, count;
    __device__ __forceinline__ F8Piece(const F8TileArgs& p, const OpPlace& at) {
        const int total = (p.K + 127) / 128, per = p.kt_per_split / 2;
        first = at.piece * per;
        blocks = max(min(total - first, per), 0);
        count = max(min(p.K - first * 128, blocks * 128), 0);
    }
};

template <int BT, bool FAR>
__device__ __forceinline__ void f8_small_sums(const F8TileArgs& p, const OpPlace& at, char* lds,
                                              f32x4 (&acc)[F8Small<BT>::TN][F8Small<BT>::TM]) {
    using T = F8Small<BT>;
    int lane = threadIdx.x & 63;
    if (FAR) asm volatile("" : "+v"(lane));  // (nothing made from it is kept from the first run)
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const F8Piece piece(p, at);
    const int first = piece.first, blocks = piece.blocks, count = piece.count;

    OpCopy<BT, T::A_PW, true, 1, false, T::WTM> ca;
    OpCopy<BT, T::B_PW, true, 1, false, T::WTN> cb;
    ca.init(p.A, p.lda, at.m0, p.M, 0, (int64_t)first * 128, count, wave, lane);
    cb.init(p.B, p.ldb, at.n0, p.N, 0, (int64_t)first * 128, count, wave, lane);
    F8Scales<T> sc;
    sc.init(p, at, first, blocks, wave, wn, lane);
    const uint32_t ring = lds_addr(lds);
    auto issue = [&](int b, int slot) {
        sc.issue(b, ring, slot, wave);
        const uint32_t a = ring + slot * T::BLOCK, w = ring + T::B_RING + slot * T::BLOCK;
        ca.template issue<0>(2 * b, a, wave);
        ca.template issue<1>(2 * b + 1, a + T::BLOCK / 2, wave);
        cb.template issue<0>(2 * b, w, wave);
        cb.template issue<1>(2 * b + 1, w + T::BLOCK / 2, wave);
    };
    const int tail = (count & 15) ? blocks - 1 : -1;
#pragma unroll
    for (int ni = 0; ni < T::TN; ++ni)
#pragma unroll
        for (int mi = 0; mi < T::TM; ++mi) acc[ni][mi] = f32x4{};
    struct Operands {
        u32x4 a[T::TM][2], b[T::TN][2];
        F8BlockScales<T::TM, FAR> s;
    };
    auto read = [&](int b, int slot, Operands& x) {
        sc.read(lds, b, slot, wm * T::WTM, lane, x.s);
        f8_read_block(lds + slot * T::BLOCK, wm * T::WTM, lane, x.a);
        f8_read_block(lds + T::B_RING + slot * T::BLOCK, wn * T::WTN, lane, x.b);
        if (b == tail) {
            f8_clear_tail(count - 128 * b, lane, x.a);
            f8_clear_tail(count - 128 * b, lane, x.b);
        }
    };
    Operands x0, x1;
    issue(0, 0);
    issue(1, 1);
    wait_vmcnt<T::LOADS>();
    lds_barrier();
    read(0, 0, x0);
    auto step = [&](int b, int slot, Operands& x, Operands& next) {
        wait_vmcnt<0>();
        lds_barrier();
        issue(b + 2, slot);
        read(b + 1, slot ^ 1, next);
        f8_multiply<T, 0, T::TN, FAR>(x.b, x.a, x.s, acc);
    };
    int b = 0;
    for (; b + 1 < blocks; b += 2) {
        step(b, 0, x0, x1);
        step(b + 1, 1, x1, x0);
    }
    if (b < blocks) step(b, 0, x0, x1);
    wait_vmcnt<0>();
}

template <int BT>
__global__ void __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(2, BT == 64 ? 4 : 2)))
f8_small_kernel(F8TileArgs p, GroupArgs g) {
    using T = F8Small<BT>;
    extern __shared__ __attribute__((aligned(1024))) char lds[];
    OpPlace at;
    if (!group_tile<kOpF8, BT>(p, g, (int)blockIdx.x, &at)) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave >> 1, wn = wave & 1;
    f32x4 acc[T::TN][T::TM];
    f8_small_sums<BT, false>(p, at, lds, acc);
    // (at f8_any's barrier the rings are free for the output)
    if (f8_any<T>(F8Piece(p, at).blocks > 0 && f8_suspect<T>(p, at, wm, wn, lane, acc), lds, wave, lane, 0)) {
        const F8Again k = F8Again::read<BT>();
        const F8Piece piece(k.p, k.at);
        if (f8_far_scales<T>(k.p, k.at, piece.first, piece.blocks, lds, wave, lane)) {
            lds_barrier();
            f8_small_sums<BT, true>(k.p, k.at, lds, acc);
            lds_barrier();
        }
    }
    if (p.splits > 1 && !op_join<T>(p, at, lds, wave, lane, acc)) return;
    op_epilogue<T, kOpF8, false>(p, lds, at, wave, wm, wn, lane, acc);
}

hipError_t launch_f8_tile(int tile, const F8TileArgs& a, const GroupArgs& g, int grid, hipStream_t s) {
    if (tile == 256) {
        if (a.splits != 1) return hipErrorInvalidValue;
        f8_pp_kernel<<<grid, 512, F8Tile256::LDS_BYTES, s>>>(a, g);
    } else if (tile == 128) {
        f8_small_kernel<128><<<grid, 256, F8Small<128>::LDS_BYTES, s>>>(a, g);
    } else {
        f8_small_kernel<64><<<grid, 256, F8Small<64>::LDS_BYTES, s>>>(a, g);
    }
    return hipGetLastError();
}

// (the 64 x 64 kernel asks for 34 KB, which needs no setting)
hipError_t configure_f8_kernels() {
    hipError_t e = hipFuncSetAttribute((const void*)f8_pp_kernel, hipFuncAttributeMaxDynamicSharedMemorySize,
                                       F8Tile256::LDS_BYTES);
    if (e == hipSuccess)
        e = hipFuncSetAttribute((const void*)f8_small_kernel<128>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                F8Small<128>::LDS_BYTES);
    return e;
}

}  // namespace glk
