// bounded_wait.cuh -- waits with a limit and the status word of the kernels that
// include this: after `timeout_ns` a wait records where it gave up, raises its CTA's
// abort flag and returns, so a protocol error ends a kernel instead of hanging the
// GPU.  (The GEMM's own are in gemm_kernel.cuh, with its kernels; each translation
// unit that includes this has a status word of its own.)
#pragma once

#include <stdint.h>

#include "../ptx.cuh"

namespace linear_ops {

static __device__ int g_group_status;               // GEMM_ERR_DEVICE_TIMEOUT of the first wait that ran out (0: none)
static __device__ unsigned long long g_group_info;  // its role, CTA and tile

enum : uint32_t { kWaitProducer = 1, kWaitMma = 2, kWaitEpilogue = 3 };

// The wait of a thread that found nothing yet (out of line: the roles' loops are short, and
// what bounds those of small tiles is a thread's instructions).
static __device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int *abort_flag, uint64_t timeout_ns,
                                            uint32_t role, uint32_t seq, bool honor_abort) {
    namespace ptx = gemm_f16::ptx;
    const uint64_t begun = ptx::globaltimer_ns();
    for (uint32_t turn = 1; !ptx::mbar_try_wait(bar, parity); ++turn) {
        if (turn % 16 != 0) continue;
        if (honor_abort && *abort_flag) return false;
        if (ptx::globaltimer_ns() - begun > timeout_ns) {
            *abort_flag = 1;
            if (atomicCAS(&g_group_status, 0, -7) == 0) {
                g_group_info = static_cast<unsigned long long>(role) << 56 |
                               static_cast<unsigned long long>(blockIdx.x & 0xFFFFFFu) << 32 | seq;
            }
            return false;
        }
    }
    return true;
}

// By one thread.  False if the wait ran out or, when `honor_abort`, as soon as another
// role of this CTA has given up.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int *abort_flag, uint64_t timeout_ns,
                                             uint32_t role, uint32_t seq, bool honor_abort = true) {
    namespace ptx = gemm_f16::ptx;
    if (ptx::mbar_try_wait(bar, parity)) return true;
    return wait_on(bar, parity, abort_flag, timeout_ns, role, seq, honor_abort);
}

}  // namespace linear_ops
