// Self-test of the device-side failure detection that every pipeline of the
// library relies on: a bounded mbarrier wait that gives up, raises the CTA's
// abort flag and records a timeout in the error word, and a second role of
// the CTA that leaves its own wait as soon as it sees the flag; and four warps
// that share a named barrier, of which one gives up a wait between two rounds:
// all four have to leave at the same round. Nothing here faults or hangs: the
// waits end, by the limit or by the flag, and every warp comes to each round.
#include <cuda_runtime.h>

#include "rag_prefill.h"
#include "leave.cuh"
#include "params.cuh"

namespace rag {

__global__ void __launch_bounds__(192, 1) wait_selftest_kernel(int32_t* err, uint64_t limit_ns) {
  __shared__ uint64_t never[3];   // barriers no thread ever arrives on
  __shared__ int abort_flag, left[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&never[0], 1);
    mbar_init(&never[1], 1);
    mbar_init(&never[2], 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  volatile int* abort = &abort_flag;
  if (warp >= 2) {
    // four times to the barrier; warp 4 gives up before the third
    constexpr int kTimes = 4, kLast = 2;
    int none = 0, done = 0;
    Run run = Run::kOn;
    for (; done < kTimes; ++done) {
      if (warp == 4 && done == kLast && !mbar_wait_for(&never[2], 0, &none, limit_ns)) run = Run::kGaveUp;
      if (run == Run::kOn && named_bar_leave(1, 128, false)) run = Run::kTold;
      if (run != Run::kOn) break;
    }
    if (run != Run::kTold) named_bar_leave(1, 128, run == Run::kGaveUp);
    if (lane == 0) left[warp - 2] = done;
  } else if (lane == 0) {
    if (warp == 0) {
      // the short wait runs out: report it and tell the other role
      if (!mbar_wait_for(&never[0], 0, abort, limit_ns)) {
        atomicOr(err, kDevErrTimeout);
        *abort = 1;
      }
    } else {
      // the full-length wait ends on the abort flag, long before its limit
      mbar_wait(&never[1], 0, abort);
    }
  }
  __syncthreads();
  if (threadIdx.x < 4 && left[threadIdx.x] != 2) atomicOr(err, kDevErrGeometry);
}

}  // namespace rag

extern "C" RAG_API rag_status rag_selftest_wait_timeout(int32_t* device_err, int64_t limit_ns, void* stream) {
  if (!device_err || limit_ns <= 0 || limit_ns > int64_t(rag::kWaitLimitNs)) return RAG_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = rag::launch_plain(rag::wait_selftest_kernel, dim3(1), dim3(192), 0, s, device_err,
                                          uint64_t(limit_ns));
  rag::note_cuda_error(e);
  return e == cudaSuccess ? RAG_OK : RAG_ERR_CUDA;
}
