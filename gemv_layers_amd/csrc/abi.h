// What the entry points share across files (internal header): the current device's state, a
// stream's workspace region, and the plan that gemm_last_plan reports.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_bf16.h"
#include "plan.h"

namespace glk {

struct Workspace {
    float* ws = nullptr;
    uint32_t* counters = nullptr;
};

// the planner's view of the current device, or nullptr with the status that the call returns
const DeviceInfo* current_device(int* status);
// the workspace region of `stream` on the current device, made on its first use
int stream_workspace(hipStream_t stream, Workspace* out);
// a product's plan and sizes; `op` is a static string
struct OpPlan {
    const char* op = nullptr;
    Plan plan;
    int64_t M = 0, N = 0, K = 0;
};
// the plan of the call that just succeeded, and that of the other product of its launch
void set_last_plan(OpPlan plan, OpPlan with = {});

// No C++ exception leaves a C entry point: a plan's text or a lock that the host has no memory for.
template <class F>
int guarded(F f) {
    try {
        return f();
    } catch (...) {
        return GEMM_ERR_HIP;
    }
}

}  // namespace glk
