// selftest.cu -- the bounded-wait paths of the kernels, run on their own: a
// kernel waits on an mbarrier phase that nothing completes, first as the decode
// and selection kernels do (mbar_wait_limit), then as the kernels over pages do
// (wait_for: with the limit, and with an abort flag that is set).  Each gives
// up, and KVD_ERR_TIMEOUT goes to the status word, as it does when data never
// arrive; a wait that did not give up records KVD_ERR_CUDA instead.  The test
// export of kvd_debug_wait_timeout; no fault, trap or endless loop is involved.
#include "common.cuh"
#include "internal.h"
#include "paged_attn_dev.cuh"

namespace kvd {
namespace {

__global__ void __launch_bounds__(32) wait_probe_kernel(int32_t *status, uint64_t limit_ns) {
    __shared__ uint64_t bar;
    __shared__ int never;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);  // one arrival expected; none comes
        never = 0;
        fence_barrier_init();
    }
    __syncthreads();
    bool ok = mbar_wait_limit(&bar, 0, &never, limit_ns);
    __syncwarp();
    ok |= wait_for(&bar, 0, &never, static_cast<uint32_t>(limit_ns));
    if (threadIdx.x == 0) never = 1;
    __syncwarp();
    ok |= wait_for(&bar, 0, &never);  // ends at once
    if (threadIdx.x == 0) report_status(status, ok ? KVD_ERR_CUDA : KVD_ERR_TIMEOUT);
}

}  // namespace

cudaError_t launch_wait_probe(int32_t *status, uint64_t limit_ns, cudaStream_t st) {
    wait_probe_kernel<<<1, 32, 0, st>>>(status, limit_ns);
    return cudaGetLastError();
}

}  // namespace kvd
