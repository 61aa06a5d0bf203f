// One kernel launch and its status.  (Host code only, without the device
// headers.)
#pragma once

#include <hip/hip_runtime_api.h>

#include "gemm_f32.h"

namespace gemmf32 {

// A failed HIP call's status, recorded for gemm_f32_last_hip_error.  In
// gemm_f32.hip.
int record_hip_error(hipError_t e);

// kernel(a) on stream s; a gemm_f32_status.  The status is that of this launch:
// hipGetLastError would also report what an earlier call, of anyone on this
// thread, has left there.  A launch holds less than 2^32 threads (HIP supports
// no more): a larger one is refused.
template <class Args>
int launch(void (*kernel)(Args), long long workgroups, int threads, size_t lds_bytes, hipStream_t s, Args a)
{
    if (workgroups > 0xffffffffll / threads) return GEMM_F32_ERR_INVALID_VALUE;
    void *args[] = {&a};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(kernel), dim3((unsigned)workgroups),
                                         dim3((unsigned)threads), args, lds_bytes, s);
    return e == hipSuccess ? GEMM_F32_SUCCESS : record_hip_error(e);
}

}  // namespace gemmf32
