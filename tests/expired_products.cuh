// expired_products.cuh -- put in front of fp8_gemm.cu (nvcc -include): one of the waits in
// the 8-bit products then reports that it expired, though what it waited for has come.  So
// the products' winding down runs on the GPU in milliseconds, with every copy in its place.
//
// Which one: the workspace's flags hold the status, the number of the wait, a count and the
// warp.  Block 0's waits of that warp are counted over the call's launches.
#pragma once

#include "common.cuh"
#include "tc_common.cuh"

namespace moe {

// Whether the wait that this thread (of block 0, one a warp) has done is the one.
__device__ __forceinline__ bool product_wait_is_picked(volatile int* abort_flag, int* err) {
  const volatile int* pick = err;
  if ((int)(threadIdx.x >> 5) != pick[3] || atomicAdd(err + 2, 1) != pick[1]) return false;
  *abort_flag = 1;
  flag_error(err, kErrTimeout);
  return true;
}

__device__ __forceinline__ bool expired_product_wait(uint32_t bar, uint32_t parity,
                                                     volatile int* abort_flag, int* err) {
  const bool ok = mbar_wait(bar, parity, abort_flag, err);
  return blockIdx.x == 0 && product_wait_is_picked(abort_flag, err) ? false : ok;
}

namespace tc {

__device__ __forceinline__ bool expired_product_warp_wait(uint32_t bar, uint32_t parity,
                                                          volatile int* abort_flag, int* err) {
  const bool ok = mbar_wait_warp(bar, parity, abort_flag, err);
  if (blockIdx.x != 0) return ok;
  const bool picked = (threadIdx.x & 31) == 0 && product_wait_is_picked(abort_flag, err);
  return __any_sync(0xffffffffu, picked) ? false : ok;
}

}  // namespace tc
}  // namespace moe

#define mbar_wait expired_product_wait
#define mbar_wait_warp expired_product_warp_wait
