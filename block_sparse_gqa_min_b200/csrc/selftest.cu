// Self-test of the bounded waits every kernel of the library uses.
//
// One warp initialises an mbarrier that nothing ever arrives on and waits on its
// first phase with the library's own bounded wait (mbar_wait), limited to the
// caller's `limit_ns`: the wait runs out, reports SBA_DEV_TIMEOUT into the status
// word and the kernel returns, so the host sees the failure as data and the
// context stays usable.  No trap, no fault and no unbounded loop is involved.
//
// The second test is of mbar_wait_warp: the lanes of a warp wait with different limits, the phase completes
// in between, and all have to come back with the one verdict that the wait ran out.
#include "common.cuh"
#include "kv4.cuh"
#include "launch.cuh"

namespace sba {
namespace {

__global__ void wait_timeout_selftest_kernel(int32_t* status, uint64_t limit_ns) {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
    }
    __syncwarp();
    bool ok = true;
    if (threadIdx.x == 0) ok = mbar_wait(&bar, 0, status, limit_ns);  // nothing arrives: runs out
    ok = __shfl_sync(0xffffffffu, ok, 0);
    (void)ok;
}

__global__ void wait_vote_selftest_kernel(int32_t* status, int32_t* verdicts, uint64_t limit_ns) {
    __shared__ uint64_t bar;
    const int tid = threadIdx.x;
    if (tid == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
    }
    __syncthreads();
    if (tid >= 32) {
        if (tid == 32) {  // arrives after twice the limit; every lane of the other warp waits one or four
            const uint64_t t0 = globaltimer_ns();
            for (int i = 0; i < 1 << 26 && globaltimer_ns() - t0 < 2 * limit_ns; ++i) __nanosleep(1000);
            mbar_arrive(&bar);
        }
    } else {
        verdicts[tid] = mbar_wait_warp(&bar, 0, status, tid < 16 ? limit_ns : 4 * limit_ns);
    }
    __syncthreads();
}

}  // namespace

int launch_wait_vote_selftest(int32_t* status, int32_t* verdicts, uint64_t limit_ns, cudaStream_t stream) {
    wait_vote_selftest_kernel<<<1, 64, 0, stream>>>(status, verdicts, limit_ns);
    return cudaGetLastError() == cudaSuccess ? SBA_OK : SBA_ERR_CUDA;
}

int launch_wait_timeout_selftest(int32_t* status, uint64_t limit_ns, cudaStream_t stream) {
    wait_timeout_selftest_kernel<<<1, 32, 0, stream>>>(status, limit_ns);
    return cudaGetLastError() == cudaSuccess ? SBA_OK : SBA_ERR_CUDA;
}

}  // namespace sba
