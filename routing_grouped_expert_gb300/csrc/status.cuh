// The status word of a launch that clears it itself (a memset ahead of it costs 2
// us on the host and as much on the device): block 0 clears the word and then
// publishes the launch's own number beside it; a block that has something to
// report, which is rare, first waits for that number.  Block 0 is among the first
// to start and waits for nobody; the wait is bounded all the same.
#pragma once

#include "moe_common.cuh"
#include "ptx.cuh"

namespace moe {

__device__ __forceinline__ void status_begin(int* status, uint64_t launch) {
  if (launch != 0 && blockIdx.x == 0 && threadIdx.x == 0) {
    status[0] = 0;
    status[1] = 0;
    __threadfence();
    *reinterpret_cast<volatile uint64_t*>(status + 2) = launch;
  }
}
static __device__ __noinline__ void status_report(int* status, uint64_t launch, int code) {
  if (launch != 0) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (*reinterpret_cast<volatile uint64_t*>(status + 2) != launch &&
           ptx::globaltimer_ns() - t0 < 1000000000ull) {
    }
    __threadfence();
  }
  set_status(status, code);
}

// The launch's number, or 0 after a memset of the status.
inline cudaError_t begin_status(int* status, cudaStream_t s, uint64_t* launch) {
  const cudaError_t err = launch_number(s, launch);
  if (err != cudaSuccess) return err;
  return *launch == 0 ? cudaMemsetAsync(status, 0, 2 * sizeof(int), s) : cudaSuccess;
}

}  // namespace moe
