// expired_waits.cuh -- put in front of one of the library's kernel files (nvcc
// -include): some of its waits then report that they expired, though what they
// waited for has come.  So the handling of an expired wait runs on the GPU in
// microseconds, with every copy and product in its place.
//
// Waits on a ring of rows (norm.cu, which has no flag word): those of thread 7 of
// block 0, none of whose tries succeeds.  Waits of a warp on a product (ortho.cu, ortho_chip.cu): the one of warp
// 2 of block 0 whose number over the call's launches stands in the second word of
// the workspace's flags; the third counts them.
#pragma once

#include "common.cuh"
#include "tc_common.cuh"

namespace moe {

__device__ __forceinline__ bool expired_mbar_wait(uint32_t bar, uint32_t parity,
                                                  volatile int* abort_flag, int* err) {
  const bool ok = mbar_wait(bar, parity, abort_flag, err);  // the data's, before the report
  if (err == nullptr && blockIdx.x == 0 && threadIdx.x == 7) {
    *abort_flag = 1;
    return false;
  }
  return ok;
}

__device__ __forceinline__ bool expired_try_wait(uint32_t bar, uint32_t parity) {
  return !(blockIdx.x == 0 && threadIdx.x == 7) && mbar_try_wait(bar, parity);
}

namespace tc {

__device__ __forceinline__ bool expired_warp_wait(uint32_t bar, uint32_t parity,
                                                  volatile int* abort_flag, int* err) {
  const bool ok = mbar_wait_warp(bar, parity, abort_flag, err);
  if (blockIdx.x == 0 && threadIdx.x >> 5 == 2) {
    int stop = 0;
    if ((threadIdx.x & 31) == 0 && atomicAdd(err + 2, 1) == static_cast<volatile int*>(err)[1]) {
      *abort_flag = 1;
      flag_error(err, kErrTimeout);
      stop = 1;
    }
    if (__shfl_sync(0xffffffffu, stop, 0)) return false;
  }
  return ok;
}

}  // namespace tc
}  // namespace moe

#define mbar_wait expired_mbar_wait
#define mbar_try_wait expired_try_wait
#define mbar_wait_warp expired_warp_wait
