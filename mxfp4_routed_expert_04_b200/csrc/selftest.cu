// moe_selftest_bounded_wait: a check of the bounded waits that the stage-ring
// kernels of this library use (mbar_wait for a producer draining its copies,
// wait_or_abort for a consumer waiting for a stage, wait_bounded for every role
// of the dense operators' kernels), made on a stage whose bytes never arrive.
//
// One CTA of five warps. Warp 0 plays the producer: it arms an mbarrier for a
// 512-byte stage (arrive.expect_tx) and, when `deliver` is set, issues the
// bulk copy that fills it; otherwise nothing ever delivers those bytes. It then
// waits for its own stage with mbar_wait (the drain every ring kernel runs
// before it exits after an abort). Warps 1, 2 and 3 play consumers that wait
// for the stage with wait_or_abort and with both forms of wait_bounded, each
// with an abort flag of its own, so that each runs into its own limit. Warp 4
// plays another role of warp 2's CTA: it waits with the kernels' own limit of
// seconds for something that does not come, and returns at once when warp 2
// raises their flag. Thread 0 finally ORs kStatusWaitTimeout into the status
// word when every wait gave up, the same last step as the ring kernels, and
// kDisagree when only some did. No copy is ever in flight when a wait gives up
// (the stage that times out was never requested), so the CTA exits cleanly and
// the context stays usable.
#include <cuda_runtime.h>

#include "../../include/moe_mxfp4.h"
#include "common.cuh"
#include "dense.cuh"
#include "kernels.h"
#include "tc05.cuh"

namespace moe {
namespace {

constexpr uint32_t kStageBytes = 512;
constexpr int kWaiters = 5;
constexpr int32_t kDisagree = 1 << 16;

__global__ void __launch_bounds__(32 * kWaiters) k_selftest_wait(int32_t* status, const uint8_t* src,
                                                                 int deliver, uint32_t limit) {
  __shared__ __align__(128) uint8_t stage[kStageBytes];
  __shared__ __align__(8) uint64_t full, never;
  __shared__ int abort_flag[kWaiters], gave_up[kWaiters];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWaiters; ++i) abort_flag[i] = 0;
    mbar_init(&full, 1);
    mbar_init(&never, 1);
    fence_mbar_init();
  }
  __syncthreads();
  volatile int* abort = &abort_flag[warp];
  bool ok;
  if (warp == 0) {
    if (lane == 0) {
      mbar_expect_tx(&full, kStageBytes);
      if (deliver) bulk_g2s(stage, src, kStageBytes, &full);
    }
    __syncwarp();
    ok = mbar_wait(&full, 0, limit);    // the drain before exit
  } else if (warp == 1) {
    ok = tc::wait_or_abort(&full, 0, abort, limit);
  } else if (warp == 2) {
    ok = tc::wait_bounded(&full, 0, abort, 1000ull * limit);
  } else if (warp == 3) {
    ok = tc::wait_bounded<true>(&full, 0, abort, 1000ull * limit);
  } else {
    ok = tc::wait_bounded(deliver ? &full : &never, 0, &abort_flag[2]);
  }
  const bool all = __all_sync(0xFFFFFFFFu, ok), none = __all_sync(0xFFFFFFFFu, !ok);
  // a wait with a flag raises it when it gives up, and only then
  const bool flagged = warp == 0 || warp == 4 || (*abort != 0) == none;
  if (lane == 0) gave_up[warp] = !flagged || (!all && !none) ? -1 : none;
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = 0;
    bool odd = false;
    for (int i = 0; i < kWaiters; ++i) {
      n += gave_up[i];
      odd |= gave_up[i] < 0;
    }
    if (odd || (n != 0 && n != kWaiters)) atomicOr(status, kDisagree);
    else if (n) atomicOr(status, kStatusWaitTimeout);
  }
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_selftest_bounded_wait(int32_t* status, const void* src, int deliver,
                                                uint32_t limit, void* stream) {
  if (!status) return moe::record_error(MOE_ERR_INVALID_ARG, "status is NULL");
  if (deliver && (!src || (reinterpret_cast<uintptr_t>(src) & 15u)))
    return moe::record_error(MOE_ERR_ALIGNMENT, "src must be a 16-byte aligned device pointer");
  if (limit < 1 || limit > 4096)
    return moe::record_error(MOE_ERR_INVALID_ARG, "limit must be in [1, 4096] tries");
  moe::k_selftest_wait<<<1, 32 * moe::kWaiters, 0, (cudaStream_t)stream>>>(
      status, static_cast<const uint8_t*>(src), deliver ? 1 : 0, limit);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return moe::record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return MOE_OK;
}
