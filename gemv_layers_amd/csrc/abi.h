// What the entry points share across files (internal header): the current device's state, a
// stream's workspace region, and the plan that gemm_last_plan reports.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

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
// the plan of the call that just succeeded; `op` is a static string
void set_last_plan(const Plan& p, int64_t M, int64_t N, int64_t K, const char* op);

}  // namespace glk
