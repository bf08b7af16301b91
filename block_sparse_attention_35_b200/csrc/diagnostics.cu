// diagnostics.cu - a kernel that exercises the library's bounded wait on a barrier that
// nothing completes, so the timeout path can be tested without hanging a GPU, and the wait of
// a whole warp on one that completes after the first of its lanes has given up.
#include "pbsa_device.cuh"
#include "pbsa_internal.cuh"

namespace pbsa {

namespace {

__global__ void wait_selftest_kernel(int32_t* status, unsigned long long limit_ns) {
    __shared__ uint64_t bar, late;
    __shared__ int abort_flag;
    const unsigned long long t0 = globaltimer_ns();
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        mbar_init(&late, 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (threadIdx.x >= 32) {
        // the late barrier completes when lane 0 of the other warp has given up (at a quarter of
        // the limit) and the rest of its lanes still wait
        if (threadIdx.x == 32) {
            while (globaltimer_ns() - t0 < limit_ns / 2) __nanosleep(1000);
            mbar_arrive(&late);
        }
    } else {
        const bool got = mbar_wait_warp(&late, 0, nullptr, nullptr, threadIdx.x == 0 ? limit_ns / 4 : limit_ns);
        if (got) set_status(status, PBSA_ERR_DEVICE_CHECK);   // some lane went on without the others
        // phase 0 never completes: the wait must give up and record PBSA_ERR_TIMEOUT
        if (threadIdx.x == 0) mbar_wait(&bar, 0, &abort_flag, status, limit_ns);
    }
    __syncthreads();
}

}  // namespace

cudaError_t launch_wait_selftest(int32_t* status, long long timeout_ns, cudaStream_t st) {
    wait_selftest_kernel<<<1, 64, 0, st>>>(status, static_cast<unsigned long long>(timeout_ns));
    return cudaGetLastError();
}

}  // namespace pbsa
