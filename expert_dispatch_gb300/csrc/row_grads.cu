// row_grads.cu -- gradients of the row movement around the expert FFN.
//
// The dispatch copies each token's row to its slots, x_perm[slot_row[t, j]] =
// x[t], so its gradient adds the slots' rows up again; the combine is
//   y[t] = sum_{j<k} w[t, j] y_perm[slot_row[t, j]] + sum_s y_perm[slot_row[t, k+s]],
// so its gradients are
//   dy_perm[slot_row[t, j]] = w[t, j] dy[t]   (w = 1 for a shared slot),
//   dw[t, j]                = <dy[t], y_perm[slot_row[t, j]]>.
// Sums and products are fp32 in slot order; rows are rounded to the layer's
// dtype once, when they are written.  Every output row has one writer, so
// there are no atomics and the results do not depend on any order of blocks.
#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kMaxSlots = 36;  // k <= 32, S <= 4

// 8 consecutive elements.
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, size_t at, float (&v)[8]) {
  if (BF16) {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* base, size_t at, const float (&v)[8]) {
  if (BF16) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at) =
        make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Most slots whose loads are in flight, and threads a block: 85 us at 4096 tokens
// x 7168 x 9 slots bf16 (6.9 TB/s); 3 or 9 slots and 256 threads take 87 to 89,
// a block for each 1024 columns of a token 93.
constexpr int kSlotsAtOnce = 5;
constexpr int kDispatchBwdThreads = 128;
constexpr int kDispatchBwdBlocks = 1216;  // blocks that keep the GPU busy

// Block (token t, slice of 1024-column steps): a slice is the whole row where
// there are tokens enough; each thread owns 8 consecutive columns of a step.
template <bool BF16>
__global__ void __launch_bounds__(kDispatchBwdThreads)
    dispatch_rows_backward_kernel(const void* __restrict__ dx_perm,
                                  const int32_t* __restrict__ slot_row, int d, int ks, int P,
                                  void* __restrict__ dx) {
  pdl_wait();
  pdl_trigger();
  __shared__ int rows_s[kMaxSlots];
  const int t = blockIdx.x;
  if (threadIdx.x < ks) {
    const int r = slot_row[(size_t)t * ks + threadIdx.x];
    rows_s[threadIdx.x] = (r < 0 || r >= P) ? -1 : r;
  }
  __syncthreads();
  // rounds of about equal size: a last one of a single slot would wait for HBM alone
  const int rounds = (ks + kSlotsAtOnce - 1) / kSlotsAtOnce, per = (ks + rounds - 1) / rounds;
  for (int c = (blockIdx.y * kDispatchBwdThreads + threadIdx.x) * 8; c < d;
       c += gridDim.y * kDispatchBwdThreads * 8) {
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < ks; j0 += per) {
      float v[kSlotsAtOnce][8];
#pragma unroll
      for (int u = 0; u < kSlotsAtOnce; ++u) {
        const int r = u < per && j0 + u < ks ? rows_s[j0 + u] : -1;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
        if (r >= 0) load8<BF16>(dx_perm, (size_t)r * d + c, v[u]);
      }
#pragma unroll
      for (int u = 0; u < kSlotsAtOnce; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += v[u][i];
    }
    store8<BF16>(dx, (size_t)t * d + c, acc);
  }
}

// Block (token, share of its slots): all slots where there are tokens enough
// (dy[t] then crosses HBM once), else one, as a chain of slots costs an HBM latency
// each.  Up to 256 threads, fewer for short rows.  Slot by slot, a thread writes
// its columns of the row's gradient and adds its part of the dot product with
// dy[t]; the warps' sums of all slots meet in shared memory once, at the end.
// Measured at 16384 tokens x 4096 x 8 slots bf16: 353 us, 6.8 TB/s; with 128
// threads 384, with 512 417, with dy[t] in registers (it stays in L1 as it is) 423.
// The rows from *total_rows to P that dropped slots leave over are set to zero,
// each token's first block taking every gridDim.x-th of them.
constexpr int kCombineBwdThreads = 256;
constexpr int kCombineBwdWarps = kCombineBwdThreads / 32;
constexpr int kCombineBwdTokens = 608;  // tokens that keep the GPU busy with a block each

template <bool BF16, bool WITH_DW, bool ALL>
__global__ void __launch_bounds__(kCombineBwdThreads)
    combine_backward_kernel(const float* __restrict__ dy, const void* __restrict__ y_perm,
                            const int32_t* __restrict__ total_rows,
                            const int32_t* __restrict__ slot_row,
                            const float* __restrict__ topk_w, int d, int k, int ks, int P,
                            void* __restrict__ dy_perm, float* __restrict__ dtopk_w) {
  pdl_wait();
  pdl_trigger();
  __shared__ int rows_s[kMaxSlots];
  __shared__ float w_s[kMaxSlots];
  __shared__ float red[kMaxSlots][kCombineBwdWarps];
  const int t = blockIdx.x, tid = threadIdx.x;
  const int threads = ALL ? kCombineBwdThreads : blockDim.x;
  const int first = ALL ? 0 : blockIdx.y, step = ALL ? 1 : gridDim.y;
  const int total = min(max(*total_rows, 0), P);
  auto slot = [&](int j) {
    const int r = slot_row[(size_t)t * ks + j];
    rows_s[j] = (r < 0 || r >= total) ? -1 : r;
    w_s[j] = (j < k && topk_w) ? topk_w[(size_t)t * k + j] : 1.f;
  };
  if constexpr (ALL) {
    if (tid < ks) slot(tid);
  } else {
    for (int j = tid; j < ks; j += threads) slot(j);
  }
  __syncthreads();
  for (int j = first; j < ks; j += step) {
    const int r = rows_s[j];
    float dot = 0.f;
    if (r >= 0) {
      const float w = w_s[j];
      for (int c = tid * 8; c < d; c += threads * 8) {
        float g[8], o[8];
        load8<false>(dy, (size_t)t * d + c, g);
        if (WITH_DW && j < k) {
          float v[8];
          load8<BF16>(y_perm, (size_t)r * d + c, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot = fmaf(g[i], v[i], dot);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = w * g[i];
        store8<BF16>(dy_perm, (size_t)r * d + c, o);
      }
    }
    if (WITH_DW && j < k) {
#pragma unroll
      for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if ((tid & 31) == 0) red[j][tid >> 5] = dot;
    }
  }
  if (WITH_DW) {
    __syncthreads();
    if constexpr (ALL) {
      if (tid < k) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kCombineBwdWarps; ++i) s += red[tid][i];
        dtopk_w[(size_t)t * k + tid] = s;
      }
    } else {
      for (int j = first + step * tid; j < k; j += step * threads) {
        float s = 0.f;
        for (int i = 0; i < threads / 32; ++i) s += red[j][i];
        dtopk_w[(size_t)t * k + j] = s;
      }
    }
  }
  if (first) return;
  const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (long long r = (long long)total + t; r < P; r += gridDim.x)
    for (int c = tid * 8; c < d; c += threads * 8)
      store8<BF16>(dy_perm, (size_t)r * d + c, zero);
}

}  // namespace

cudaError_t launch_dispatch_rows_backward(int dtype, const void* dx_perm,
                                          const int32_t* slot_row, int T, int d, int ks,
                                          void* dx, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  ProfScope pr("dispatch_rows_backward", s);
  const int steps = (d + kDispatchBwdThreads * 8 - 1) / (kDispatchBwdThreads * 8);
  const int want = (kDispatchBwdBlocks + T - 1) / T;
  const int slices = want < steps ? want : steps;
  (void)launch_kernel(dtype == MOE_BF16 ? dispatch_rows_backward_kernel<true>
                                        : dispatch_rows_backward_kernel<false>,
                      dim3(T, slices), kDispatchBwdThreads, 0, s, dx_perm, slot_row, d, ks, T * ks,
                      dx);
  return cudaGetLastError();
}

cudaError_t launch_combine_backward(int dtype, const float* dy, const void* y_perm,
                                    const int32_t* total_rows, const int32_t* slot_row,
                                    const float* topk_w, int T, int d, int k, int S,
                                    void* dy_perm, float* dtopk_w, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  ProfScope pr("combine_backward", s);
  const int ks = k + S, columns = (d / 8 + 31) / 32 * 32;
  const int threads = columns < kCombineBwdThreads ? columns : kCombineBwdThreads;
  const bool all = threads == kCombineBwdThreads && T >= kCombineBwdTokens;
  auto of = [&](auto bf16, auto dw) {
    constexpr bool B = decltype(bf16)::value, W = decltype(dw)::value;
    return all ? combine_backward_kernel<B, W, true> : combine_backward_kernel<B, W, false>;
  };
  using std::bool_constant;
  auto kern = dtype == MOE_BF16
                  ? (dtopk_w ? of(bool_constant<true>(), bool_constant<true>())
                             : of(bool_constant<true>(), bool_constant<false>()))
                  : (dtopk_w ? of(bool_constant<false>(), bool_constant<true>())
                             : of(bool_constant<false>(), bool_constant<false>()));
  (void)launch_kernel(kern, dim3(T, T < kCombineBwdTokens ? ks : 1), threads, 0, s, dy, y_perm,
                      total_rows, slot_row, topk_w, d, k, ks, T * ks, dy_perm, dtopk_w);
  return cudaGetLastError();
}

}  // namespace moe
