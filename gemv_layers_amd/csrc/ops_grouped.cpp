// Entry points of the products grouped by expert and of the 8-bit floating-point products (declared in
// include/gemm_bf16.h): argument checks on the host before any HIP call, planning, and dispatch onto the
// caller's stream. A plain 8-bit floating-point product is a grouped one whose rows are all of one group.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "abi.h"
#include "gemm_bf16.h"
#include "kernels.h"
#include "ops.h"

namespace {

using glk::GroupArgs;
using glk::guarded;
using glk::OpArgs;

constexpr int64_t kMaxRows = (int64_t(1) << 24) - 1;  // rows, or tiles, of 256 threads in a 32-bit grid
constexpr int64_t kMaxK = int64_t(1) << 30;

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
hipStream_t hip_stream(gemm_stream_t s) { return reinterpret_cast<hipStream_t>(s); }
int64_t blocks(int64_t n) { return n / 128 + (n % 128 != 0); }

const char* op_name(int mode, bool grouped) {
    switch (mode) {
        case glk::kOpF8: return grouped ? "f8_grouped" : "f8";
        case glk::kOpAbt: return "grouped_grad_a";
        case glk::kOpAtb: return "grouped_grad_b";
        default: return "grouped";
    }
}

// A product that is ready to launch: planned, its limits checked, its workspace at hand. A call prepares
// every product it makes before it launches anything, so that a refused one has written nothing.
struct Ready {
    enum Route { kZero, kGeneral, kTiles, kDecode } route = kZero;
    bool fused = false;  // kDecode: a.A holds one row of bf16
    int mode = 0;
    OpArgs a{};
    GroupArgs g{};
    glk::Plan p;
    glk::Workspace w;
};

// Whether the matrix kernels take these operands: 16-byte aligned rows, 32-bit offsets within a tile, and
// widths of 8 except along the rows of groups.
bool matrix_ok(int mode, const OpArgs& a, const GroupArgs& g) {
    const int64_t unit = mode == glk::kOpF8 ? 16 : 8;
    const int64_t max_ld = int64_t(1) << 20, max_dim = int64_t(1) << 26;
    if (misaligned(a.A, 16) || misaligned(a.B, 16) || (a.lda % unit) || (a.ldb % unit) || (g.stride_b % unit)) return false;
    if (a.lda > max_ld || a.ldb > max_ld || a.ldc > max_ld) return false;
    if (a.M > max_dim || a.N > max_dim || a.K > max_dim) return false;
    if (mode == glk::kOpF8) return true;  // (any width; C at any element)
    if (misaligned(a.C, 16) || (a.ldc % 8) || (g.stride_c % 8) || (a.N % 8)) return false;
    return mode == glk::kOpAtb ? a.M % 8 == 0 : a.K % 8 == 0;
}

// plans r's product on MFMA tiles, of `tile` rows and columns if that is not 0
int plan_tiles(int tile, const glk::DeviceInfo& dev, hipStream_t stream, Ready* r) {
    const bool f8 = r->mode == glk::kOpF8, summed = r->mode == glk::kOpAtb;
    // codes: planned as the bf16 product whose k-steps have the same bytes and matrix-core cycles
    glk::GroupShape shape{r->g.rows, r->g.offsets || summed ? r->g.groups : 0, r->a.M, r->a.N, f8 ? (r->a.K + 1) / 2 : r->a.K,
                          summed, f8, r->mode == glk::kOpAb};
    shape.tile = tile;
    r->route = Ready::kTiles;
    r->p = glk::make_group_plan(shape, dev);
    if (r->p.grid > glk::kMostThreads / r->p.threads) return GEMM_ERR_UNSUPPORTED;
    r->g.cus = dev.cus;
    r->g.tail = r->p.tail;
    r->g.slots = (int)r->p.counters;
    return r->p.ws_floats > 0 ? glk::stream_workspace(stream, &r->w) : GEMM_OK;
}

// One product on the current device with a non-empty C, operands checked. `fused`: one row of bf16 activations
// and a weight that the weight-streaming kernel takes. The rows of C (of kOpAtb those of
// all groups' C together) are written whole.
int prepare(int mode, const OpArgs& a, const GroupArgs& g, bool fused, hipStream_t stream, Ready* r) {
    int st = GEMM_OK;
    const glk::DeviceInfo* dev = glk::current_device(&st);
    if (!dev) return st;
    r->mode = mode;
    r->a = a;
    r->g = g;
    if (mode != glk::kOpAtb && (g.groups == 0 || a.K == 0)) {
        r->route = Ready::kZero;
        r->p = glk::make_plan(a.M, a.N, 0, *dev, false, 2, false);
        return GEMM_OK;
    }
    const int64_t groups = g.offsets ? g.groups : 0;
    const bool matrix = fused || matrix_ok(mode, a, g);
    r->fused = fused;
    if (mode == glk::kOpF8 && matrix && glk::f8_decode_pays(g.rows, groups)) {  // the weight-streaming kernel
        r->p = glk::make_f8_decode_plan(g.rows, a.N, a.K, groups, *dev);
        if (r->p.grid <= glk::kMostThreads / r->p.threads) {
            r->route = Ready::kDecode;
            return r->p.ws_floats > 0 ? glk::stream_workspace(stream, &r->w) : GEMM_OK;
        }
    }
    if (matrix) return plan_tiles(0, *dev, stream, r);
    // 64 x 64 tiles of 256 threads, 32-bit grids
    const int64_t row_tiles =
        mode == glk::kOpAtb ? ((a.M - 1) / 64 + 1) * g.groups : glk::most_row_tiles(g.rows, groups, 64);
    if (row_tiles > kMaxRows / ((a.N - 1) / 64 + 1)) return GEMM_ERR_UNSUPPORTED;
    r->route = Ready::kGeneral;
    r->p = glk::make_plan(a.M, a.N, a.K, *dev, false, 2, false);
    return GEMM_OK;
}

glk::OpPlan plan_of(const Ready& r) {
    return {op_name(r.mode, r.g.offsets != nullptr), r.p, r.a.M, r.a.N, r.mode == glk::kOpAtb ? r.g.rows : r.a.K};
}

glk::OpTileArgs tile_args(const Ready& r) {
    const OpArgs& a = r.a;
    glk::OpTileArgs t{};
    t.A = a.A;
    t.B = a.B;
    t.C = a.C;
    t.sa = a.sa;
    t.sb = a.sb;
    t.M = (int)a.M;
    t.N = (int)a.N;
    t.K = (int)a.K;
    t.lda = (int)a.lda;
    t.ldb = (int)a.ldb;
    t.ldc = (int)a.ldc;
    t.up = (int)a.N;
    t.vec = !misaligned(a.C, 16) && a.ldc % 8 == 0 && a.N % 8 == 0;
    t.tiles_m = (int)r.p.tiles_m;
    t.tiles_n = (int)r.p.tiles_n;
    t.group_m = r.p.group_m;
    t.nxcd = r.p.nxcd;
    t.splits = r.p.splits;
    t.kt_per_split = r.p.kt_per_split;
    t.ws = r.w.ws;
    t.counters = r.w.counters;
    return t;
}

glk::F8TileArgs f8_tile_args(const Ready& r) { return {tile_args(r), r.a.ldsa, r.a.ldsb}; }

int launch(const Ready& r, hipStream_t stream) {
    const OpArgs& a = r.a;
    hipError_t e = hipSuccess;
    switch (r.route) {
        case Ready::kZero:
            e = glk::launch_zero_c(a.C, a.M, a.N, a.ldc, stream);
            break;
        case Ready::kGeneral:
            e = glk::launch_group_generic(r.mode, a, r.g, stream);
            break;
        case Ready::kDecode: {
            const glk::F8DecodeArgs t{r.fused ? nullptr : static_cast<const uint8_t*>(a.A),
                                      r.fused ? static_cast<const uint16_t*>(a.A) : nullptr,
                                      static_cast<const uint8_t*>(a.B), a.C, a.sa, a.sb, (int)a.N, (int)a.K, (int)a.lda,
                                      (int)a.ldb, (int)a.ldc, r.p.strips, r.p.splits, r.p.nxcd, r.w.ws, r.w.counters, a.ldsa, a.ldsb};
            e = glk::launch_f8_decode(r.p.mtiles, r.p.strip / 16, t, r.g, (int)r.p.grid, stream);
            break;
        }
        case Ready::kTiles:
            e = r.mode == glk::kOpF8 ? glk::launch_f8_tile(r.p.bm, f8_tile_args(r), r.g, (int)r.p.grid, stream)
                                     : glk::launch_group_tile(r.mode, r.p.bm, tile_args(r), r.g, (int)r.p.grid, stream);
            break;
    }
    if (e != hipSuccess) return GEMM_ERR_HIP;
    glk::set_last_plan(plan_of(r));
    return GEMM_OK;
}

// Both gradients as one launch where each is a grid of the same small tiles: the second's partials follow the
// first's. Small ones whose tiles differ take dB's (1018 rows in 8 groups, 512 to 1376: 9.8 and 7.8 us alone with 64 x 64 and
// 128 x 128 tiles, 18.0 in two launches, 13.3 in one with 128 x 128, 15.1 with 64 x 64).
int launch_gradients(Ready a, Ready b, const glk::DeviceInfo& dev, hipStream_t stream) {
    if (a.route == Ready::kTiles && b.route == Ready::kTiles && a.p.bm < 256 && b.p.bm < 256 && a.p.bm != b.p.bm &&
        a.p.grid <= 4 * dev.cus && b.p.grid <= 4 * dev.cus) {
        const int st = plan_tiles(b.p.bm, dev, stream, &a);
        if (st != GEMM_OK) return st;
    }
    const glk::Plan &pa = a.p, &pb = b.p;
    const bool pair = a.route == Ready::kTiles && b.route == Ready::kTiles && pa.bm == pb.bm && pa.bm < 256 &&
                      pa.grid + pb.grid <= glk::kMostThreads / 256 && pa.ws_floats + pb.ws_floats <= dev.ws_floats &&
                      pa.counters + pb.counters <= dev.ws_counters;
    if (!pair) {
        const int st = launch(a, stream);
        return st == GEMM_OK ? launch(b, stream) : st;
    }
    if (pa.ws_floats > 0 && pb.ws_floats > 0) {
        b.w.ws = a.w.ws + pa.ws_floats;
        b.w.counters = a.w.counters + pa.counters;
    }
    if (glk::launch_group_pair(pa.bm, tile_args(a), a.g, (int)pa.grid, tile_args(b), b.g, (int)pb.grid, stream) != hipSuccess)
        return GEMM_ERR_HIP;
    glk::set_last_plan(plan_of(b), plan_of(a));
    return GEMM_OK;
}

// checks shared by all products of grouped rows
int check_groups(int64_t M, int64_t E, const int32_t* offsets) {
    if (M < 0 || E < 0) return GEMM_ERR_INVALID_ARG;
    if (M > 0 && E > 0 && (!offsets || misaligned(offsets, 4))) return GEMM_ERR_INVALID_ARG;
    if (M > kMaxRows || E > glk::kMaxGroups) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

// ---- 8-bit floating point ---------------------------------------------------------------------------

int quantize(int64_t R, int64_t K, const void* X, int64_t ldx, void* Q, int64_t ldq, float* S, int64_t lds,
             hipStream_t stream) {
    if (R < 0 || K < 0 || ldx < K || ldq < K || lds < R) return GEMM_ERR_INVALID_ARG;
    if (R > 0 && K > 0 && (!X || !Q || !S || misaligned(S, 4) || misaligned(X, 2))) return GEMM_ERR_INVALID_ARG;
    if (R > kMaxRows || K > kMaxK) return GEMM_ERR_UNSUPPORTED;
    if (R == 0 || K == 0) return GEMM_OK;
    int st = GEMM_OK;
    if (!glk::current_device(&st)) return st;
    return glk::launch_f8_quantize(static_cast<const uint16_t*>(X), R, K, ldx, static_cast<uint8_t*>(Q), ldq, S, lds,
                                   stream) == hipSuccess
               ? GEMM_OK
               : GEMM_ERR_HIP;
}

// an 8-bit weight of E groups and its scales
struct F8Weight {
    const void* q;
    int64_t ld, stride;
    const float* s;
    int64_t lds, stride_s;
};

// E groups with `offsets`, or (dense) one of all rows. `A` with rows of lda: codes, or bf16 to be quantised.
int check_f8(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const F8Weight& w, int64_t E, bool dense,
             const int32_t* offsets, const void* C, int64_t ldc) {
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
    const int st = dense ? (M > kMaxRows ? GEMM_ERR_UNSUPPORTED : GEMM_OK) : check_groups(M, E, offsets);
    if (st == GEMM_ERR_INVALID_ARG) return st;
    if (lda < K || w.ld < K || ldc < N || w.lds < blocks(K) || w.stride < 0 || w.stride_s < 0) return GEMM_ERR_INVALID_ARG;
    if (M > 0 && K > 0 && !A) return GEMM_ERR_INVALID_ARG;
    if (E > 0 && N > 0 && K > 0 && (!w.q || !w.s || misaligned(w.s, 4))) return GEMM_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && (!C || misaligned(C, 2))) return GEMM_ERR_INVALID_ARG;
    return K > kMaxK ? GEMM_ERR_UNSUPPORTED : st;
}

int f8_product(int64_t M, int64_t N, int64_t K, const void* Aq, int64_t lda, const float* Sa, int64_t ldsa,
               const F8Weight& w, int64_t E, bool dense, const int32_t* offsets, void* C, int64_t ldc,
               hipStream_t stream) {
    int st = check_f8(M, N, K, Aq, lda, w, E, dense, offsets, C, ldc);
    if (st == GEMM_ERR_INVALID_ARG) return st;
    if (ldsa < M || (M > 0 && K > 0 && (!Sa || misaligned(Sa, 4)))) return GEMM_ERR_INVALID_ARG;
    if (st != GEMM_OK || M == 0 || N == 0) return st;
    OpArgs a{Aq, w.q, static_cast<uint16_t*>(C), nullptr, Sa, w.s, M, N, K, lda, w.ld, ldc, 0};
    a.ldsa = ldsa;
    a.ldsb = w.lds;
    Ready r;
    st = prepare(glk::kOpF8, a, GroupArgs{dense ? nullptr : offsets, (int)E, (int)M, w.stride, 0, w.stride_s}, false, stream, &r);
    return st == GEMM_OK ? launch(r, stream) : st;
}

// M x K codes with rows padded to 16 bytes, then ceil(K / 128) x M scales
int64_t padded_codes(int64_t K) { return (K + 15) / 16 * 16; }
int64_t work_bytes_of(int64_t M, int64_t K) { return M * padded_codes(K) + 4 * M * blocks(K); }

int f8_product_bf16(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const F8Weight& w, int64_t E, bool dense,
                    const int32_t* offsets, void* C, int64_t ldc, void* work, int64_t work_bytes, hipStream_t stream) {
    int st = check_f8(M, N, K, A, lda, w, E, dense, offsets, C, ldc);
    if (st == GEMM_ERR_INVALID_ARG) return st;
    if (M > 0 && misaligned(A, 2)) return GEMM_ERR_INVALID_ARG;
    if (st != GEMM_OK || M == 0 || N == 0) return st;
    if (K > 0 && (!work || misaligned(work, 16) || work_bytes < work_bytes_of(M, K))) return GEMM_ERR_INVALID_ARG;
    OpArgs a{work, w.q, static_cast<uint16_t*>(C), nullptr, nullptr, w.s, M, N, K, padded_codes(K), w.ld, ldc, 0};
    const GroupArgs g{dense ? nullptr : offsets, (int)E, (int)M, w.stride, 0, w.stride_s};
    Ready r;
    // one row: quantised in the product's kernel (neither its alignment nor its leading dimension matters)
    if (dense && M == 1 && K > 0 && K <= glk::kF8FusedK && matrix_ok(glk::kOpF8, a, g)) {
        a.A = A;
        a.ldsb = w.lds;
        st = prepare(glk::kOpF8, a, g, true, stream, &r);
        return st == GEMM_OK ? launch(r, stream) : st;
    }
    float* sa = reinterpret_cast<float*>(static_cast<char*>(work) + M * a.lda);
    a.sa = sa;
    a.ldsa = M;
    a.ldsb = w.lds;
    st = prepare(glk::kOpF8, a, g, false, stream, &r);
    if (st == GEMM_OK && K > 0 && E > 0) st = quantize(M, K, A, lda, work, a.lda, sa, M, stream);
    return st == GEMM_OK ? launch(r, stream) : st;
}

}  // namespace

extern "C" {

int gemm_f8_quantize(int64_t R, int64_t K, const void* X, int64_t ldx, void* Q, int64_t ldq, float* S, int64_t lds,
                     gemm_stream_t stream) {
    return guarded([&] { return quantize(R, K, X, ldx, Q, ldq, S, lds, hip_stream(stream)); });
}

int gemm_f8_quantize_weight(int64_t E, int64_t N, int64_t K, const void* W, int64_t ldw, int64_t stride_w, void* Q,
                            int64_t ldq, int64_t stride_q, float* S, int64_t lds, int64_t stride_s,
                            gemm_stream_t stream) {
    return guarded([&]() -> int {
        if (E < 0 || N < 0 || K < 0 || ldw < K || ldq < K || lds < blocks(K)) return GEMM_ERR_INVALID_ARG;
        if (N > kMaxRows || K > kMaxK || E > glk::kMaxGroups) return GEMM_ERR_UNSUPPORTED;
        if (E == 0 || N == 0 || K == 0) return GEMM_OK;
        if (!W || !Q || !S || misaligned(W, 2) || misaligned(S, 4) || stride_w < 0) return GEMM_ERR_INVALID_ARG;
        // (outputs of different matrices do not meet)
        if (E > 1 && (stride_q / N < ldq || stride_s / blocks(N) < lds)) return GEMM_ERR_INVALID_ARG;
        if (blocks(N) > kMaxRows / blocks(K)) return GEMM_ERR_UNSUPPORTED;
        int st = GEMM_OK;
        if (!glk::current_device(&st)) return st;
        const glk::F8WeightArgs a{static_cast<const uint16_t*>(W), static_cast<uint8_t*>(Q), S, E, N, K, ldw, stride_w,
                                  ldq, stride_q, lds, stride_s};
        return glk::launch_f8_quantize_weight(a, hip_stream(stream)) == hipSuccess ? GEMM_OK : GEMM_ERR_HIP;
    });
}

int gemm_f8(int64_t M, int64_t N, int64_t K, const void* Aq, int64_t ldaq, const float* Sa, int64_t ldsa,
            const void* Wq, int64_t ldwq, const float* Sw, int64_t ldsw, void* C, int64_t ldc, gemm_stream_t stream) {
    return guarded([&] {
        return f8_product(M, N, K, Aq, ldaq, Sa, ldsa, F8Weight{Wq, ldwq, 0, Sw, ldsw, 0}, 1, true, nullptr, C, ldc,
                          hip_stream(stream));
    });
}

int gemm_f8_work_bytes(int64_t M, int64_t K, int64_t* bytes) {
    if (M < 0 || K < 0 || !bytes) return GEMM_ERR_INVALID_ARG;
    if (M > kMaxRows || K > kMaxK) return GEMM_ERR_UNSUPPORTED;
    *bytes = work_bytes_of(M, K);
    return GEMM_OK;
}

int gemm_f8_bf16(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* Wq, int64_t ldwq,
                 const float* Sw, int64_t ldsw, void* C, int64_t ldc, void* work, int64_t work_bytes,
                 gemm_stream_t stream) {
    return guarded([&] {
        return f8_product_bf16(M, N, K, A, lda, F8Weight{Wq, ldwq, 0, Sw, ldsw, 0}, 1, true, nullptr, C, ldc, work,
                               work_bytes, hip_stream(stream));
    });
}

int gemm_f8_grouped(int64_t M, int64_t N, int64_t K, int64_t E, const void* Aq, int64_t ldaq, const float* Sa,
                    int64_t ldsa, const void* Wq, int64_t ldwq, int64_t stride_wq, const float* Sw, int64_t ldsw,
                    int64_t stride_sw, const int32_t* offsets, void* C, int64_t ldc, gemm_stream_t stream) {
    return guarded([&] {
        return f8_product(M, N, K, Aq, ldaq, Sa, ldsa, F8Weight{Wq, ldwq, stride_wq, Sw, ldsw, stride_sw}, E, false,
                          offsets, C, ldc, hip_stream(stream));
    });
}

int gemm_f8_grouped_bf16(int64_t M, int64_t N, int64_t K, int64_t E, const void* A, int64_t lda, const void* Wq,
                         int64_t ldwq, int64_t stride_wq, const float* Sw, int64_t ldsw, int64_t stride_sw,
                         const int32_t* offsets, void* C, int64_t ldc, void* work, int64_t work_bytes,
                         gemm_stream_t stream) {
    return guarded([&] {
        return f8_product_bf16(M, N, K, A, lda, F8Weight{Wq, ldwq, stride_wq, Sw, ldsw, stride_sw}, E, false, offsets, C,
                               ldc, work, work_bytes, hip_stream(stream));
    });
}

int gemm_bf16_grouped(int64_t M, int64_t N, int64_t K, int64_t E, const void* A, int64_t lda, const void* B,
                      int64_t ldb, int64_t stride_b, const int32_t* offsets, void* C, int64_t ldc,
                      gemm_stream_t stream) {
    return guarded([&]() -> int {
        if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
        int st = check_groups(M, E, offsets);
        if (st == GEMM_ERR_INVALID_ARG) return st;
        if (lda < K || ldb < N || ldc < N || stride_b < 0) return GEMM_ERR_INVALID_ARG;
        if ((M > 0 && K > 0 && !A) || (E > 0 && K > 0 && N > 0 && !B) || (M > 0 && N > 0 && !C)) return GEMM_ERR_INVALID_ARG;
        if (misaligned(A, 2) || misaligned(B, 2) || misaligned(C, 2)) return GEMM_ERR_INVALID_ARG;
        if (K > kMaxK) return GEMM_ERR_UNSUPPORTED;
        if (st != GEMM_OK || M == 0 || N == 0) return st;
        const OpArgs a{A, B, static_cast<uint16_t*>(C), nullptr, nullptr, nullptr, M, N, K, lda, ldb, ldc, 0};
        Ready r;
        st = prepare(glk::kOpAb, a, GroupArgs{offsets, (int)E, (int)M, stride_b, 0, 0}, false, hip_stream(stream), &r);
        return st == GEMM_OK ? launch(r, hip_stream(stream)) : st;
    });
}

int gemm_bf16_grouped_bwd(int64_t M, int64_t N, int64_t K, int64_t E, const void* dC, int64_t lddc, const void* A,
                          int64_t lda, const void* B, int64_t ldb, int64_t stride_b, const int32_t* offsets, void* dA,
                          int64_t ldda, void* dB, int64_t lddb, int64_t stride_db, gemm_stream_t stream) {
    return guarded([&]() -> int {
        if (M < 0 || N < 0 || K < 0 || lddc < N || misaligned(dC, 2)) return GEMM_ERR_INVALID_ARG;
        int st = check_groups(M, E, offsets);
        if (st == GEMM_ERR_INVALID_ARG) return st;
        if ((dA || dB) && M > 0 && N > 0 && K > 0 && !dC) return GEMM_ERR_INVALID_ARG;
        if (dA && (ldb < N || ldda < K || stride_b < 0 || (E > 0 && K > 0 && N > 0 && !B))) return GEMM_ERR_INVALID_ARG;
        if (dB && (lda < K || lddb < N || (M > 0 && K > 0 && !A))) return GEMM_ERR_INVALID_ARG;
        if (dB && E > 1 && K > 0 && stride_db / K < lddb) return GEMM_ERR_INVALID_ARG;  // (the gradients do not meet)
        if ((dA && (misaligned(dA, 2) || misaligned(B, 2))) || (dB && (misaligned(dB, 2) || misaligned(A, 2))))
            return GEMM_ERR_INVALID_ARG;
        if (K > kMaxK || N > kMaxK) return GEMM_ERR_UNSUPPORTED;
        if (st != GEMM_OK) return st;
        const bool need_a = dA && M > 0 && K > 0, need_b = dB && E > 0 && K > 0 && N > 0;
        Ready ra, rb;
        if (need_a) {
            const OpArgs a{dC, B, static_cast<uint16_t*>(dA), nullptr, nullptr, nullptr, M, K, N, lddc, ldb, ldda, 0};
            st = prepare(glk::kOpAbt, a, GroupArgs{offsets, (int)E, (int)M, stride_b, 0, 0}, false, hip_stream(stream), &ra);
        }
        if (st == GEMM_OK && need_b) {
            const OpArgs b{A, dC, static_cast<uint16_t*>(dB), nullptr, nullptr, nullptr, K, N, 0, lda, lddc, lddb, 0};
            st = prepare(glk::kOpAtb, b, GroupArgs{offsets, (int)E, (int)M, 0, stride_db, 0}, false, hip_stream(stream), &rb);
        }
        if (st != GEMM_OK) return st;
        if (need_a && need_b) {
            const glk::DeviceInfo* dev = glk::current_device(&st);
            return dev ? launch_gradients(ra, rb, *dev, hip_stream(stream)) : st;
        }
        if (need_a) return launch(ra, hip_stream(stream));
        return need_b ? launch(rb, hip_stream(stream)) : GEMM_OK;
    });
}

}  // extern "C"
