// Entry points of the 8-bit and training products (declared in include/gemm_bf16.h): argument
// checks on the host before any HIP call, planning, and dispatch onto the caller's stream.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "abi.h"
#include "gemm_bf16.h"
#include "kernels.h"
#include "ops.h"

namespace {

using glk::guarded;
using glk::OpArgs;

constexpr int64_t kMaxCodesK = 131071;  // 128 * 128 * K < 2^31
constexpr int64_t kMaxRows = (int64_t(1) << 24) - 1;  // rows, or tiles, of 256 threads in a 32-bit grid

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

hipStream_t hip_stream(gemm_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

const char* op_name(int mode, bool glu) {
    switch (mode) {
        case glk::kOpI8: return glu ? "i8_swiglu" : "i8";
        case glk::kOpAbt: return "grad_a";
        case glk::kOpAtb: return "grad_b";
        default: return "swiglu_train";
    }
}

// Whether the matrix kernels take these operands: 16-byte aligned rows, 32-bit offsets within a tile.
// Codes need no multiple in any size, and C any rows; bf16 widths are multiples of 8, except along the
// summed index where it is the row index.
bool matrix_ok(int mode, bool glu, const OpArgs& a) {
    const int64_t unit = mode == glk::kOpI8 ? 16 : 8;
    const int64_t max_ld = int64_t(1) << 20, max_dim = int64_t(1) << 26;
    if (misaligned(a.A, 16) || misaligned(a.B, 16) || (a.lda % unit) || (a.ldb % unit)) return false;
    if (a.lda > max_ld || a.ldb > max_ld || a.ldc > max_ld || a.ldgu > max_ld) return false;
    if (a.M > max_dim || a.N > max_dim || a.K > max_dim) return false;
    if (mode == glk::kOpI8) return true;
    if (misaligned(a.C, 16) || (a.ldc % 8) || (a.N % 8)) return false;
    if (mode == glk::kOpTrain && (misaligned(a.GU, 16) || (a.ldgu % 8))) return false;
    return mode == glk::kOpAtb ? a.M % 8 == 0 : a.K % 8 == 0;
}

// The tile kernels' arguments for plan `p` over rows m0 .. m0 + M - 1 and columns n0 .. n0 + N - 1.
glk::OpTileArgs tile_args(int mode, const OpArgs& a, const glk::Plan& p, int64_t m0, int64_t M, int64_t n0, int64_t N,
                          const glk::Workspace& w) {
    const int64_t es = mode == glk::kOpI8 ? 1 : 2;
    const bool a_contig = mode != glk::kOpAtb, b_contig = mode == glk::kOpI8 || mode == glk::kOpAbt;
    glk::OpTileArgs t;
    t.A = static_cast<const char*>(a.A) + es * m0 * (a_contig ? a.lda : 1);
    t.B = static_cast<const char*>(a.B) + es * n0 * (b_contig ? a.ldb : 1);
    t.C = a.C + m0 * a.ldc + n0;
    t.GU = a.GU ? a.GU + m0 * a.ldgu + n0 : nullptr;
    t.sa = a.sa ? a.sa + m0 : nullptr;
    t.sb = a.sb ? a.sb + n0 : nullptr;
    t.M = (int)M;
    t.N = (int)N;
    t.K = (int)a.K;
    t.lda = (int)a.lda;
    t.ldb = (int)a.ldb;
    t.ldc = (int)a.ldc;
    t.ldgu = (int)a.ldgu;
    t.up = (int)a.N;
    t.vec = !misaligned(t.C, 16) && a.ldc % 8 == 0 && N % 8 == 0;
    t.tiles_m = (int)p.tiles_m;
    t.tiles_n = (int)p.tiles_n;
    t.group_m = p.group_m;
    t.nxcd = p.nxcd;
    t.splits = p.sched == glk::kSchedSplitK ? p.splits : 1;
    t.kt_per_split = p.kt_per_split;
    t.ws = w.ws;
    t.counters = w.counters;
    return t;
}

hipError_t launch_tiles(int mode, bool glu, const OpArgs& a, const glk::Plan& p, int64_t m0, int64_t M, int64_t n0,
                        int64_t N, const glk::Workspace& w, hipStream_t stream) {
    return glk::launch_op_tile(mode, glu, p.bm, tile_args(mode, a, p, m0, M, n0, N, w), (int)p.grid, stream);
}

// A product that is ready to launch: planned, its limits checked, its workspace at hand. A call prepares
// every product it makes before it launches anything, so that a refusal leaves its outputs, and inputs
// that it overwrites, as they were.
struct Ready {
    enum Route { kZero, kGeneral, kTiles, kDecode } route = kZero;
    int mode = 0;
    bool glu = false;
    bool fused = false;  // kDecode: a.A holds bf16
    OpArgs a{};
    glk::Plan p;
    glk::Workspace w;
};

// One product on the current device: M, N > 0, operands checked. `fused`: one row of bf16 activations
// and a weight that the weight-streaming kernel takes.
int prepare(int mode, bool glu, const OpArgs& a, bool fused, hipStream_t stream, Ready* r) {
    int st = GEMM_OK;
    const glk::DeviceInfo* dev = glk::current_device(&st);
    if (!dev) return st;
    r->mode = mode;
    r->glu = glu;
    r->fused = fused;
    r->a = a;
    const bool matrix = fused || (a.K > 0 && matrix_ok(mode, glu, a));
    if (mode == glk::kOpI8 && a.M <= 64 && matrix) {  // at most 64 rows: the weight-streaming kernel
        r->p = glk::make_i8_decode_plan(a.M, a.N, a.K, *dev, glu);
        if (fused || glk::i8_decode_fits(a.M, a.K, r->p)) {
            r->route = Ready::kDecode;
            return r->p.splits > 1 ? glk::stream_workspace(stream, &r->w) : GEMM_OK;
        }
    }
    if (a.K == 0) {
        r->route = Ready::kZero;
        r->p = glk::make_plan(a.M, a.N, 0, *dev, false, 2, glu);
    } else if (!matrix) {
        // 64 x 64 tiles of 256 threads, 32-bit grids
        if ((a.M - 1) / 64 + 1 > kMaxRows / ((a.N - 1) / 64 + 1)) return GEMM_ERR_UNSUPPORTED;
        r->route = Ready::kGeneral;
        r->p = glk::make_plan(a.M, a.N, a.K, *dev, false, 2, glu);
    } else {
        // codes: planned as the bf16 product whose k-steps have the same bytes and matrix-core cycles
        r->route = Ready::kTiles;
        r->p = glk::make_op_plan(a.M, a.N, mode == glk::kOpI8 ? (a.K + 1) / 2 : a.K, *dev, glu,
                                 mode == glk::kOpI8 || mode == glk::kOpAbt);
        if (r->p.grid > INT32_MAX) return GEMM_ERR_UNSUPPORTED;
        if (r->p.ws_floats > 0) return glk::stream_workspace(stream, &r->w);
    }
    return GEMM_OK;
}

glk::OpPlan plan_of(const Ready& r) { return {op_name(r.mode, r.glu), r.p, r.a.M, r.a.N, r.a.K}; }

int launch(const Ready& r, hipStream_t stream) {
    const OpArgs& a = r.a;
    const glk::Plan& p = r.p;
    hipError_t e = hipSuccess;
    switch (r.route) {
        case Ready::kDecode: {
            const glk::I8DecodeArgs t{r.fused ? nullptr : static_cast<const int8_t*>(a.A),
                                      r.fused ? static_cast<const uint16_t*>(a.A) : nullptr,
                                      static_cast<const int8_t*>(a.B), a.C, a.sa, a.sb, (int)a.M, (int)a.N, (int)a.K,
                                      (int)a.lda, (int)a.ldb, (int)a.ldc, p.splits,
                                      reinterpret_cast<int32_t*>(r.w.ws), r.w.counters};
            e = glk::launch_i8_decode(r.glu, p.mtiles, p.strip / 16, p.threads / 64, t, (int)p.grid, stream);
            break;
        }
        case Ready::kZero:
            e = glk::launch_zero_c(a.C, a.M, a.N, a.ldc, stream);
            if (e == hipSuccess && r.mode == glk::kOpTrain) e = glk::launch_zero_c(a.GU, a.M, 2 * a.N, a.ldgu, stream);
            break;
        case Ready::kGeneral:
            e = glk::launch_op_generic(r.mode, r.glu, a, stream);
            break;
        case Ready::kTiles: {
            const int64_t Mm = p.cut_axis == 2 ? p.cut_at : a.M, Nm = p.cut_axis == 1 ? p.cut_at : a.N;
            e = launch_tiles(r.mode, r.glu, a, p, 0, Mm, 0, Nm, r.w, stream);
            if (e == hipSuccess && p.cut_axis == 1)
                e = launch_tiles(r.mode, r.glu, a, p.rest[0], 0, a.M, Nm, a.N - Nm, r.w, stream);
            else if (e == hipSuccess && p.cut_axis == 2)
                e = launch_tiles(r.mode, r.glu, a, p.rest[0], Mm, a.M - Mm, 0, a.N, r.w, stream);
            break;
        }
    }
    if (e != hipSuccess) return GEMM_ERR_HIP;
    glk::set_last_plan(plan_of(r));
    return GEMM_OK;
}

// checks shared by the 8-bit products; `rows` of Wq are N or 2N
int check_i8(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* Wq, int64_t ldwq,
             const float* Sw, const void* C, int64_t ldc, bool glu) {
    if (M < 0 || N < 0 || K < 0 || (glu && N > INT64_MAX / 2)) return GEMM_ERR_INVALID_ARG;
    if (lda < K || ldwq < K || ldc < N) return GEMM_ERR_INVALID_ARG;
    if (M > 0 && K > 0 && !A) return GEMM_ERR_INVALID_ARG;
    if (N > 0 && ((K > 0 && !Wq) || !Sw || misaligned(Sw, 4))) return GEMM_ERR_INVALID_ARG;
    if (M > 0 && N > 0 && (!C || misaligned(C, 2))) return GEMM_ERR_INVALID_ARG;
    if (K > kMaxCodesK) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}

int i8_product(int64_t M, int64_t N, int64_t K, const void* Aq, int64_t ldaq, const float* Sa, const void* Wq,
               int64_t ldwq, const float* Sw, void* C, int64_t ldc, bool glu, hipStream_t stream) {
    int st = check_i8(M, N, K, Aq, ldaq, Wq, ldwq, Sw, C, ldc, glu);
    if (st != GEMM_OK) return st;
    if (M > 0 && (!Sa || misaligned(Sa, 4))) return GEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return GEMM_OK;
    Ready r;
    const OpArgs a{Aq, Wq, static_cast<uint16_t*>(C), nullptr, Sa, Sw, M, N, K, ldaq, ldwq, ldc, 0};
    st = prepare(glk::kOpI8, glu, a, false, stream, &r);
    return st == GEMM_OK ? launch(r, stream) : st;
}

int quantize(int64_t R, int64_t K, const void* X, int64_t ldx, void* Q, int64_t ldq, float* S, hipStream_t stream) {
    if (R < 0 || K < 0 || ldx < K || ldq < K) return GEMM_ERR_INVALID_ARG;
    if (R > 0 && (!S || misaligned(S, 4) || misaligned(X, 2))) return GEMM_ERR_INVALID_ARG;
    if (R > 0 && K > 0 && (!X || !Q)) return GEMM_ERR_INVALID_ARG;
    if (R > kMaxRows) return GEMM_ERR_UNSUPPORTED;
    if (R == 0) return GEMM_OK;
    int st = GEMM_OK;
    if (!glk::current_device(&st)) return st;
    return glk::launch_i8_quantize(static_cast<const uint16_t*>(X), R, K, ldx, static_cast<int8_t*>(Q), ldq, S,
                                   stream) == hipSuccess
               ? GEMM_OK
               : GEMM_ERR_HIP;
}

// M x K codes with rows padded to 16 bytes, then M scales
int64_t padded_codes(int64_t K) { return (K + 15) / 16 * 16; }
int64_t work_bytes_of(int64_t M, int64_t K) { return M * padded_codes(K) + 4 * M; }

int i8_product_bf16(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* Wq, int64_t ldwq,
                    const float* Sw, void* C, int64_t ldc, void* work, int64_t work_bytes, bool glu,
                    hipStream_t stream) {
    int st = check_i8(M, N, K, A, lda, Wq, ldwq, Sw, C, ldc, glu);
    if (st != GEMM_OK) return st;
    if (M > 0 && misaligned(A, 2)) return GEMM_ERR_INVALID_ARG;
    if (M > kMaxRows) return GEMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return GEMM_OK;
    if (!work || misaligned(work, 16) || work_bytes < work_bytes_of(M, K)) return GEMM_ERR_INVALID_ARG;
    Ready r;
    // one row: quantised in the product's kernel (neither its alignment nor its leading dimension matters)
    OpArgs a{nullptr, Wq, static_cast<uint16_t*>(C), nullptr, nullptr, Sw, M, N, K, 16, ldwq, ldc, 0};
    if (M == 1 && K > 0 && K <= glk::kI8FusedK && matrix_ok(glk::kOpI8, glu, a)) {
        a.A = A;
        st = prepare(glk::kOpI8, glu, a, true, stream, &r);
        return st == GEMM_OK ? launch(r, stream) : st;
    }
    a.A = work;
    a.lda = padded_codes(K);
    float* sa = reinterpret_cast<float*>(static_cast<char*>(work) + M * a.lda);
    a.sa = sa;
    st = prepare(glk::kOpI8, glu, a, false, stream, &r);
    if (st == GEMM_OK) st = quantize(M, K, A, lda, work, a.lda, sa, stream);
    return st == GEMM_OK ? launch(r, stream) : st;
}

// dA = D B^T and dB = A^T D for D (M x W), ready to launch
struct Gradients {
    bool need_a = false, need_b = false;
    bool pair = false;  // both in one launch
    Ready a, b;
};

// Both gradients as one launch where each is a grid of the same small tiles that leaves CUs idle, with
// the plans, and so the bits, of either alone (512^3: 4.8 and 5.5 us alone, 6.3 together; M = 509, N =
// 2752, K = 512: 9.3 and 7.6 alone, 11.5 together): the second's partials follow the first's.
void pair_gradients(const glk::DeviceInfo& dev, Gradients* g) {
    const glk::Plan &pa = g->a.p, &pb = g->b.p;
    if (g->a.route != Ready::kTiles || g->b.route != Ready::kTiles) return;
    if (pa.bm != pb.bm || pa.bm == 256 || pa.cut_axis || pb.cut_axis) return;
    if (pa.grid > dev.cus * int64_t(4) || pb.grid > dev.cus * int64_t(4)) return;
    if (pa.ws_floats + pb.ws_floats > dev.ws_floats || pa.counters + pb.counters > dev.ws_counters) return;
    g->pair = true;
    if (pb.ws_floats > 0 && pa.ws_floats > 0) {
        g->b.w.ws = g->a.w.ws + pa.ws_floats;
        g->b.w.counters = g->a.w.counters + pa.counters;
    }
}

// either gradient skipped when null
int prepare_gradients(int64_t M, int64_t W, int64_t K, const void* D, int64_t ldd, const void* A, int64_t lda,
                      const void* B, int64_t ldb, void* dA, int64_t ldda, void* dB, int64_t lddb, hipStream_t stream,
                      Gradients* g) {
    g->need_a = dA && M > 0 && K > 0;
    g->need_b = dB && K > 0 && W > 0;
    int st = GEMM_OK;
    if (g->need_a) {
        const OpArgs a{D, B, static_cast<uint16_t*>(dA), nullptr, nullptr, nullptr, M, K, W, ldd, ldb, ldda, 0};
        st = prepare(glk::kOpAbt, false, a, false, stream, &g->a);
    }
    if (st == GEMM_OK && g->need_b) {
        const OpArgs b{A, D, static_cast<uint16_t*>(dB), nullptr, nullptr, nullptr, K, W, M, lda, ldd, lddb, 0};
        st = prepare(glk::kOpAtb, false, b, false, stream, &g->b);
    }
    if (st == GEMM_OK && g->need_a && g->need_b) {
        const glk::DeviceInfo* dev = glk::current_device(&st);
        if (dev) pair_gradients(*dev, g);
    }
    return st;
}

int launch_gradients(const Gradients& g, hipStream_t stream) {
    if (!g.pair) {
        int st = g.need_a ? launch(g.a, stream) : GEMM_OK;
        if (st == GEMM_OK && g.need_b) st = launch(g.b, stream);
        return st;
    }
    const OpArgs &a = g.a.a, &b = g.b.a;
    if (glk::launch_op_pair(g.a.p.bm, tile_args(glk::kOpAbt, a, g.a.p, 0, a.M, 0, a.N, g.a.w),
                            tile_args(glk::kOpAtb, b, g.b.p, 0, b.M, 0, b.N, g.b.w), (int)(g.a.p.grid + g.b.p.grid),
                            stream) != hipSuccess)
        return GEMM_ERR_HIP;
    glk::set_last_plan(plan_of(g.b), plan_of(g.a));
    return GEMM_OK;
}

// checks of the operands of the gradients; W columns of D
int check_gradients(int64_t M, int64_t W, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb,
                    const void* dA, int64_t ldda, const void* dB, int64_t lddb) {
    if (dA && (ldb < W || ldda < K || (K > 0 && W > 0 && !B))) return GEMM_ERR_INVALID_ARG;
    if (dB && (lda < K || lddb < W || (M > 0 && K > 0 && !A))) return GEMM_ERR_INVALID_ARG;
    if ((dA && (misaligned(dA, 2) || misaligned(B, 2))) || (dB && (misaligned(dB, 2) || misaligned(A, 2))))
        return GEMM_ERR_INVALID_ARG;
    return GEMM_OK;
}

}  // namespace

extern "C" {

int gemm_i8_quantize(int64_t R, int64_t K, const void* X, int64_t ldx, void* Q, int64_t ldq, float* S,
                     gemm_stream_t stream) {
    return guarded([&] { return quantize(R, K, X, ldx, Q, ldq, S, hip_stream(stream)); });
}

int gemm_i8(int64_t M, int64_t N, int64_t K, const void* Aq, int64_t ldaq, const float* Sa, const void* Wq,
            int64_t ldwq, const float* Sw, void* C, int64_t ldc, gemm_stream_t stream) {
    return guarded([&] { return i8_product(M, N, K, Aq, ldaq, Sa, Wq, ldwq, Sw, C, ldc, false, hip_stream(stream)); });
}

int gemm_i8_swiglu(int64_t M, int64_t N, int64_t K, const void* Aq, int64_t ldaq, const float* Sa, const void* Wq,
                   int64_t ldwq, const float* Sw, void* C, int64_t ldc, gemm_stream_t stream) {
    return guarded([&] { return i8_product(M, N, K, Aq, ldaq, Sa, Wq, ldwq, Sw, C, ldc, true, hip_stream(stream)); });
}

int gemm_i8_work_bytes(int64_t M, int64_t K, int64_t* bytes) {
    if (M < 0 || K < 0 || !bytes) return GEMM_ERR_INVALID_ARG;
    if (M > kMaxRows || K > kMaxCodesK) return GEMM_ERR_UNSUPPORTED;
    *bytes = work_bytes_of(M, K);
    return GEMM_OK;
}

int gemm_i8_bf16(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* Wq, int64_t ldwq,
                 const float* Sw, void* C, int64_t ldc, void* work, int64_t work_bytes, gemm_stream_t stream) {
    return guarded([&] {
        return i8_product_bf16(M, N, K, A, lda, Wq, ldwq, Sw, C, ldc, work, work_bytes, false, hip_stream(stream));
    });
}

int gemm_i8_swiglu_bf16(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* Wq, int64_t ldwq,
                        const float* Sw, void* C, int64_t ldc, void* work, int64_t work_bytes,
                        gemm_stream_t stream) {
    return guarded([&] {
        return i8_product_bf16(M, N, K, A, lda, Wq, ldwq, Sw, C, ldc, work, work_bytes, true, hip_stream(stream));
    });
}

int gemm_bf16_bwd(int64_t M, int64_t N, int64_t K, const void* dC, int64_t lddc, const void* A, int64_t lda,
                  const void* B, int64_t ldb, void* dA, int64_t ldda, void* dB, int64_t lddb,
                  gemm_stream_t stream) {
    return guarded([&]() -> int {
        if (M < 0 || N < 0 || K < 0 || lddc < N || misaligned(dC, 2)) return GEMM_ERR_INVALID_ARG;
        if ((dA || dB) && M > 0 && N > 0 && K > 0 && !dC) return GEMM_ERR_INVALID_ARG;
        int st = check_gradients(M, N, K, A, lda, B, ldb, dA, ldda, dB, lddb);
        if (st != GEMM_OK) return st;
        Gradients g;
        st = prepare_gradients(M, N, K, dC, lddc, A, lda, B, ldb, dA, ldda, dB, lddb, hip_stream(stream), &g);
        return st == GEMM_OK ? launch_gradients(g, hip_stream(stream)) : st;
    });
}

int gemm_bf16_swiglu_train(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb,
                           void* GU, int64_t ldgu, void* C, int64_t ldc, gemm_stream_t stream) {
    return guarded([&]() -> int {
        if (M < 0 || N < 0 || K < 0 || N > INT64_MAX / 2) return GEMM_ERR_INVALID_ARG;
        if (lda < K || ldb < 2 * N || ldgu < 2 * N || ldc < N) return GEMM_ERR_INVALID_ARG;
        if ((M > 0 && K > 0 && !A) || (K > 0 && N > 0 && !B) || (M > 0 && N > 0 && (!GU || !C)))
            return GEMM_ERR_INVALID_ARG;
        if (misaligned(A, 2) || misaligned(B, 2) || misaligned(GU, 2) || misaligned(C, 2)) return GEMM_ERR_INVALID_ARG;
        if (M == 0 || N == 0) return GEMM_OK;
        const OpArgs a{A, B, static_cast<uint16_t*>(C), static_cast<uint16_t*>(GU), nullptr, nullptr,
                       M, N, K, lda, ldb, ldc, ldgu};
        Ready r;
        const int st = prepare(glk::kOpTrain, true, a, false, hip_stream(stream), &r);
        return st == GEMM_OK ? launch(r, hip_stream(stream)) : st;
    });
}

int gemm_bf16_swiglu_bwd(int64_t M, int64_t N, int64_t K, const void* dC, int64_t lddc, const void* GU,
                         int64_t ldgu, const void* A, int64_t lda, const void* B, int64_t ldb, void* dGU,
                         int64_t lddgu, void* dA, int64_t ldda, void* dB, int64_t lddb, gemm_stream_t stream) {
    return guarded([&]() -> int {
        if (M < 0 || N < 0 || K < 0 || N > INT64_MAX / 2) return GEMM_ERR_INVALID_ARG;
        if (lddc < N || ldgu < 2 * N || lddgu < 2 * N) return GEMM_ERR_INVALID_ARG;
        if (M > 0 && N > 0 && (!dC || !GU || !dGU)) return GEMM_ERR_INVALID_ARG;
        if (misaligned(dC, 2) || misaligned(GU, 2) || misaligned(dGU, 2)) return GEMM_ERR_INVALID_ARG;
        int st = check_gradients(M, 2 * N, K, A, lda, B, ldb, dA, ldda, dB, lddb);
        if (st != GEMM_OK) return st;
        Gradients g;
        st = prepare_gradients(M, 2 * N, K, dGU, lddgu, A, lda, B, ldb, dA, ldda, dB, lddb, hip_stream(stream), &g);
        if (st != GEMM_OK) return st;
        if (M > 0 && N > 0) {
            if (!glk::current_device(&st)) return st;
            if (glk::launch_swiglu_grad(static_cast<const uint16_t*>(dC), lddc, static_cast<const uint16_t*>(GU), ldgu,
                                        static_cast<uint16_t*>(dGU), lddgu, M, N, hip_stream(stream)) != hipSuccess)
                return GEMM_ERR_HIP;
        }
        return launch_gradients(g, hip_stream(stream));
    });
}

}  // extern "C"
