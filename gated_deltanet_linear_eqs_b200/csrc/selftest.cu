// selftest.cu -- a kernel whose bounded waits are made to run out.
//
// Every wait in the library's kernels is bounded: when it gives up, the kernel records
// GDN_ERR_TIMEOUT in the device status word, unwinds and returns, so that a lost arrival
// becomes an error the host can read instead of a hung GPU.  This kernel takes that path on
// purpose, safely, on mbarriers that nothing arrives on (flags that nothing sets):
//  - warp 0: one thread waits, with a short limit (mbar_wait);
//  - warp 1: all lanes wait together, with the same limit (wait_all), and leave their number behind;
//  - warps 2 and 3: the same with the full limit of two seconds.  The number ends them early; they go on as
//    the kernels' warps do, to further waits (which end at their first poll) and to a named barrier.
// The error is recorded only if every wait gave up and the number is warp 1's.  Nothing else is touched, so the
// context stays usable.
#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace gdn {

namespace {

using namespace sm100;

__global__ void __launch_bounds__(128) wait_timeout_kernel(int* status, unsigned long long limit_ns) {
    __shared__ uint64_t bars[2];
    __shared__ int flags[2];  // never set; the number of the wait that gave up
    __shared__ int gave_up;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(&bars[0], 1);  // each expects one arrival; none ever comes
        mbar_init(&bars[1], 1);
        flags[0] = flags[1] = gave_up = 0;
        fence_mbar_init();
    }
    __syncthreads();
    volatile int *never = &flags[0], *abort = &flags[1];
    if (warp == 0) {
        if (lane == 0 && !mbar_wait(&bars[0], 0, never, limit_ns)) atomicAdd(&gave_up, 1);
        __syncwarp();
    } else if (warp == 1) {
        if (!wait_all(&bars[1], 0, abort, 6, 2 * static_cast<long long>(limit_ns)) && lane == 0) atomicAdd(&gave_up, 1);
    } else {
        for (int i = 0; i < 100; ++i)
            if (!wait_all(&bars[1], 0, abort, 7) && lane == 0) atomicAdd(&gave_up, 1);
        named_sync(1, 64);
    }
    __syncthreads();
    if (threadIdx.x == 0 && gave_up == 2 + 2 * 100 && *abort == 6 + 1) record_status(status, GDN_ERR_TIMEOUT);
}

}  // namespace

cudaError_t launch_wait_timeout_selftest(int* status, unsigned long long limit_ns, cudaStream_t st) {
    wait_timeout_kernel<<<1, 128, 0, st>>>(status, limit_ns);
    return cudaGetLastError();
}

}  // namespace gdn
