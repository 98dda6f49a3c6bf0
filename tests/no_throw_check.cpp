// A host without memory: the C entries that build a plan's text return a status, and throw nothing. operator new
// is replaced here, for the library too.
#include <cstdio>
#include <cstdlib>
#include <new>

#include "abi.h"
#include "gemm_bf16.h"

static bool g_fail = false;
void* operator new(std::size_t n) {
    void* p = g_fail ? nullptr : std::malloc(n ? n : 1);
    if (!p) throw std::bad_alloc();
    return p;
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, std::size_t) noexcept { std::free(p); }

template <class F>
static int call(const char* name, F f) {
    int st = -1;
    try {
        g_fail = true;
        st = f();
        g_fail = false;
    } catch (...) {
        g_fail = false;
        std::printf("%s threw\n", name);
        return 1;
    }
    if (st == GEMM_OK) std::printf("%s did not allocate\n", name);
    return st == GEMM_OK;
}

int main() {
    char buf[4096];
    int bad = 0;
    for (int flags : {0, GEMM_PLAN_SWIGLU, GEMM_PLAN_MX, GEMM_PLAN_PACKED})
        bad += call("gemm_plan_describe", [&] { return gemm_plan_describe(64, 4096, 4096, 256, flags, buf, sizeof buf); });
    // what the newest 8-bit or training call leaves
    glk::OpPlan o;
    o.op = "i8";
    o.plan.kernel = 3;
    glk::set_last_plan(o, o);
    if (gemm_last_plan(buf, sizeof buf) != GEMM_OK) return 1;
    bad += call("gemm_last_plan", [&] { return gemm_last_plan(buf, sizeof buf); });
    if (gemm_last_plan(buf, sizeof buf) != GEMM_OK) return 1;  // its lock is free again
    std::puts(bad ? "failed" : "ok");
    return bad;
}
