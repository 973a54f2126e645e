// fake_launches.cuh -- put in front of fp8_gemm.cu (nvcc -include): its launcher on the host
// alone, without a GPU.  The runtime reports `fake_regs` registers a thread for every kernel,
// launches are counted and go nowhere.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

static int fake_regs = 0, fake_launches = 0;

static cudaError_t fake_device(int* dev) {
  *dev = 0;
  return cudaSuccess;
}
static cudaError_t fake_attributes(cudaFuncAttributes* a) {
  *a = cudaFuncAttributes{};
  a->numRegs = fake_regs;
  a->maxThreadsPerBlock = 384;
  return cudaSuccess;
}
static cudaError_t fake_launch() {
  ++fake_launches;
  return cudaSuccess;
}

#define cudaGetDevice(dev) fake_device(dev)
#define cudaGetLastError() cudaSuccess
#define cudaFuncSetAttribute(...) cudaSuccess
#define cudaFuncGetAttributes(a, kernel) fake_attributes(a)
#define cudaLaunchKernelEx(...) fake_launch()

#include "internal.h"
#include "tc_common.cuh"

namespace moe {

int num_sms() { return 152; }
int tc_row_capacity(int P) { return (P + 31) / 32 * 32 + 256; }
void count_launch() {}
ProfScope::ProfScope(const char* n, cudaStream_t s, uint64_t) : name(n), stream(s), slot(-1) {}
ProfScope::~ProfScope() {}
bool make_tmap_2d(CUtensorMap*, const void*, CUtensorMapDataType, int, uint64_t, uint64_t,
                  uint32_t, uint32_t, CUtensorMapSwizzle) {
  return true;
}

}  // namespace moe

// The products of 100 rows where a thread has `regs` registers at launch: the launcher's
// status, and how many kernels it launched.
extern "C" int fake_products(int regs, int* launches) {
  fake_regs = regs, fake_launches = 0;
  const moe::Fp8Weight w{nullptr, nullptr};
  const cudaError_t e = moe::launch_ffn_fp8(nullptr, nullptr, nullptr, 4, 100, 256, 256, w, w, w,
                                            nullptr, nullptr, nullptr, nullptr, nullptr, nullptr);
  *launches = fake_launches;
  return (int)e;
}
