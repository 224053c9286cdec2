// kvp_selftest.cu -- exercises the bounded mbarrier waits that every pipeline wait of the
// library goes through (dev::mbar_wait_bounded, and mm::wait of the block-scaled
// products): barriers that nothing arrives on, a short limit, the shared abort flag that
// ends the other waits of the CTA, and the status word the host reads afterwards.  The GPU
// and the context stay usable; nothing faults or hangs.
#include "kvp_device.cuh"
#include "kvp_internal.h"
#include "kvp_matmul.cuh"

namespace kvp {
namespace {

constexpr int kWaits = 3;   // a warp each

__global__ void selftest_wait_kernel(int32_t* status, uint64_t limit_ns) {
  using namespace dev;
  // barriers with one arrival expected on each; none comes.  Warp 0 waits with the
  // caller's limit, warp 1 with the default 2 s; both poll one abort flag, so warp 1
  // gives up right after warp 0 does (within 16 tries), the way every role of a pipeline
  // stops once one of its waits has failed.  Warp 2 waits as the products do.
  __shared__ uint64_t bar[kWaits];
  __shared__ int abort_flag, gave_up;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWaits; ++i) mbar_init(smem_addr(&bar[i]), 1);
    abort_flag = 0;
    gave_up = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
    const uint32_t at = smem_addr(&bar[warp]);
    const bool ok = warp == 2 ? mm::wait(at, 0, limit_ns)
                              : mbar_wait_bounded(at, 0, warp == 0 ? limit_ns : kWaitTimeoutNs,
                                                  &abort_flag);
    if (!ok) atomicAdd(&gave_up, 1);
  }
  __syncthreads();
  if (threadIdx.x == 0 && gave_up == kWaits) set_status(status, kErrTimeout);
}

}  // namespace

cudaError_t launch_selftest_wait(int32_t* status, uint64_t limit_ns, cudaStream_t s) {
  selftest_wait_kernel<<<1, 32 * kWaits, 0, s>>>(status, limit_ns);
  return cudaGetLastError();
}

}  // namespace kvp
