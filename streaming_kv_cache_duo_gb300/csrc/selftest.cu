// Self-test of the kernels' failure detection: a bounded wait that runs out.
//
// One CTA initialises an mbarrier that nothing will ever complete and waits on
// it with the same bounded wait the attention kernels use, but with a caller
// chosen limit. The wait gives up, records kErrSelftest in this translation
// unit's error word and the kernel returns; the host then reads the word through
// duo_device_error(). No fault, trap or endless loop is involved.
//
// Then the form in which a whole warp waits: lane 0's time is over after a quarter of
// the limit, the other lanes' after the whole of it, and another warp completes the
// barrier halfway. The lanes have to come out with one answer (waiting each for itself,
// lane 0 would give up and the others would not); kErrSelftestSplit records if they do not.
#include "duo_device.cuh"

namespace duo {
namespace {

__device__ unsigned int g_selftest_err;

__global__ void bounded_wait_kernel(uint64_t limit_ns) {
  __shared__ __align__(8) uint64_t bar, warp_bar;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    fence_mbarrier_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 0;; ++it) {
      if (mbar_try_wait(&bar, 0)) break;  // never true: nothing arrives
      if ((it & 255u) == 255u && global_timer_ns() - t0 > limit_ns) {
        atomicOr(&g_selftest_err, kErrSelftest);
        break;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    mbar_init(&warp_bar, 1);
    fence_mbarrier_init();
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const bool ok = mbar_wait_warp_for(&warp_bar, 0, threadIdx.x == 0 ? limit_ns / 4 : limit_ns);
    __syncwarp();
    if (__any_sync(0xffffffffu, ok) != __all_sync(0xffffffffu, ok) && threadIdx.x == 0)
      atomicOr(&g_selftest_err, kErrSelftestSplit);
  } else if (threadIdx.x == 32) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < limit_ns / 2) {
    }
    mbar_arrive(&warp_bar);
  }
  __syncthreads();
}

}  // namespace

cudaError_t launch_selftest_wait(uint64_t limit_ns, cudaStream_t stream) {
  bounded_wait_kernel<<<1, 64, 0, stream>>>(limit_ns);
  return cudaGetLastError();
}

cudaError_t selftest_read_clear_error(uint32_t* code) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_selftest_err, sizeof(v));
  if (e != cudaSuccess) return e;
  *code = v;
  if (v) {
    v = 0;
    e = cudaMemcpyToSymbol(g_selftest_err, &v, sizeof(v));
  }
  return e;
}

}  // namespace duo
