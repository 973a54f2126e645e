// norm.cu -- layer norm and RMS norm of token rows, forward and backward (the
// norm in front of the router: the layer's x is "already normed").
//
// Forward, per row:   mu = mean(x), var = mean((x - mu)^2), r = 1 / sqrt(var + eps),
//                     y = (x - mu) r gamma + beta;     RMS: mu = 0 and no beta.
// Backward, per row, with h = (x - mu) r and w = dy gamma:
//                     dx = r (w - mean(w) - h mean(w h));   RMS: without mean(w),
// and over the rows:  dgamma = sum dy h, dbeta = sum dy.
//
// Everything is computed and summed in fp32; the one rounding to bf16 is that
// of y or dx.  The variance is the mean of the squared deviations from the
// mean (two reductions over registers), not E[x^2] - mu^2, which cancels for
// rows whose mean is large against their spread.
//
// A row belongs to a group of whole warps that holds it in registers, so it
// crosses HBM once.  Rows whose bytes are a multiple of 16 move in 16-byte
// vectors, others element by element.
#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kMaxGroupWarps = 32;
constexpr int kBwdBlocks = 304;  // most blocks of the backward pass: two per SM

// VEC consecutive elements of a row as fp32: one 16-byte access, or one element.
template <typename T, int VEC>
__device__ __forceinline__ void load_pack(const T* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = load_as_f32(p, 0);
  } else if constexpr (sizeof(T) == 4) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    if constexpr (sizeof(T) == 4)
      *p = v[0];
    else
      *p = __float2bfloat16_rn(v[0]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// VEC elements of a parameter vector (fp32 or bf16, whatever the rows are);
// null stands for `otherwise`.
template <int VEC>
__device__ __forceinline__ void load_param(const void* p, bool bf16, int c, float otherwise,
                                           float (&v)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = otherwise;
  if (!p) return;
  if (bf16) {
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p) + c;
    if constexpr (VEC == 8) {
      load_pack<__nv_bfloat16, 8>(q, v);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = load_as_f32(q, i);
    }
  } else {
    const float* q = static_cast<const float*>(p) + c;
    if constexpr (VEC == 1) {
      v[0] = *q;
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        const float4 a = *reinterpret_cast<const float4*>(q + i);
        v[i] = a.x, v[i + 1] = a.y, v[i + 2] = a.z, v[i + 3] = a.w;
      }
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of N values over a group of `warps` warps, the same in every thread.
// `buf` holds the group's partial sums, [2][N][kMaxGroupWarps]; successive
// calls take its halves in turn, so one barrier a call is enough.  A group of
// several warps meets at named barrier 1 + group (at most 8 such groups).
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int warps, int warp_in_group, int group,
                                          float* buf, int& turn) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (warps == 1) return;
  float* b = buf + turn * N * kMaxGroupWarps;
  turn ^= 1;
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) b[i * kMaxGroupWarps + warp_in_group] = v[i];
  }
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(warps * 32) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < warps ? b[i * kMaxGroupWarps + lane] : 0.f);
}

// ---------------------------------------------------------------- forward
// blockDim.x = groups * warps * 32; the groups of a block take successive rows.
template <typename T, int VEC, int VPT, bool RMS>
__global__ void __launch_bounds__(512)
    norm_forward_kernel(const T* x, const void* gamma, const void* beta, bool w_bf16,
                                    int rows, int d, int warps, float eps, T* y, float* mean,
                                    float* rstd) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[8][2 * kMaxGroupWarps];
  const int gt = warps * 32;
  const int group = threadIdx.x / gt, tid = threadIdx.x - group * gt;
  const int row = blockIdx.x * (blockDim.x / gt) + group;
  if (row >= rows) return;  // a whole group
  const int nv = d / VEC;
  const T* xr = x + (size_t)row * d;
  float v[VPT][VEC];
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * gt;
    if (c < nv) {
      load_pack<T, VEC>(xr + (size_t)c * VEC, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[0] += RMS ? v[i][j] * v[i][j] : v[i][j];
  }
  int turn = 0;
  float* buf = red[warps == 1 ? 0 : group];
  group_sum<1>(s, warps, tid >> 5, group, buf, turn);
  float mu = 0.f;
  if (!RMS) {
    mu = s[0] / d;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (tid + i * gt < nv) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float c = v[i][j] - mu;
          s[0] = fmaf(c, c, s[0]);
        }
      }
    }
    group_sum<1>(s, warps, tid >> 5, group, buf, turn);
  }
  const float r = 1.f / sqrtf(s[0] / d + eps);
  if (tid == 0) {
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = r;
  }
  T* yr = y + (size_t)row * d;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = tid + i * gt;
    if (c >= nv) break;
    float g[VEC], b[VEC], o[VEC];
    load_param<VEC>(gamma, w_bf16, c * VEC, 1.f, g);
    load_param<VEC>(RMS ? nullptr : beta, w_bf16, c * VEC, 0.f, b);
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] = fmaf((v[i][j] - mu) * r, g[j], b[j]);
    store_pack<T, VEC>(yr + (size_t)c * VEC, o);
  }
}

// ---------------------------------------------------------------- backward
// Block b takes rows b * groups + group, + gridDim.x * groups, ...; a thread
// owns the same columns of every row and keeps their sums of dy h and dy in
// registers.  At the end the groups' sums are added in group order through
// shared memory and written to partial [2][gridDim.x][d].
template <typename T, int VEC, int VPT, bool RMS>
__global__ void __launch_bounds__(1024)
    norm_backward_kernel(const T* dy, const T* x, const void* gamma, bool w_bf16,
                         const float* mean, const float* rstd, int rows, int d, int warps, T* dx,
                         float* partial) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float sums[];  // [d] of one quantity, for the groups' sums
  __shared__ float red[8][4 * kMaxGroupWarps];
  const int gt = warps * 32, groups = blockDim.x / gt;
  const int group = threadIdx.x / gt, tid = threadIdx.x - group * gt;
  const int nv = d / VEC;
  float dg[VPT][VEC], db[VPT][VEC];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dg[i][j] = db[i][j] = 0.f;
  int turn = 0;
  float* buf = red[warps == 1 ? 0 : group];
  for (int row = blockIdx.x * groups + group; row < rows; row += gridDim.x * groups) {
    const float mu = RMS ? 0.f : mean[row], r = rstd[row];
    const size_t base = (size_t)row * d;
    float h[VPT][VEC], w[VPT][VEC];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = tid + i * gt;
      if (c < nv) {
        float g[VEC];
        load_pack<T, VEC>(x + base + (size_t)c * VEC, h[i]);
        load_pack<T, VEC>(dy + base + (size_t)c * VEC, w[i]);
        load_param<VEC>(gamma, w_bf16, c * VEC, 1.f, g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          h[i][j] = (h[i][j] - mu) * r;
          dg[i][j] = fmaf(w[i][j], h[i][j], dg[i][j]);
          if (!RMS) db[i][j] += w[i][j];
          w[i][j] *= g[j];
          s[0] = fmaf(w[i][j], h[i][j], s[0]);
          s[1] += w[i][j];
        }
      }
    }
    group_sum<2>(s, warps, tid >> 5, group, buf, turn);
    const float c1 = s[0] / d, c2 = RMS ? 0.f : s[1] / d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = tid + i * gt;
      if (c < nv) {
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = (w[i][j] - c2 - h[i][j] * c1) * r;
        store_pack<T, VEC>(dx + base + (size_t)c * VEC, o);
      }
    }
  }
  auto flush = [&](float (&acc)[VPT][VEC], float* out) {
    for (int g = 0; g < groups; ++g) {
      __syncthreads();
      if (group != g) continue;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * gt;
        if (c < nv) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float v = g ? sums[c * VEC + j] + acc[i][j] : acc[i][j];
            if (g == groups - 1)
              out[c * VEC + j] = v;
            else
              sums[c * VEC + j] = v;
          }
        }
      }
    }
  };
  if (partial) {
    flush(dg, partial + (size_t)blockIdx.x * d);
    if (!RMS) flush(db, partial + (size_t)(gridDim.x + blockIdx.x) * d);
  }
}

// out[c] = sum over the n blocks of partial[q][b][c], q = blockIdx.y: 32
// columns a block, 32 row lanes, added in a fixed order.
__global__ void __launch_bounds__(1024)
    norm_reduce_kernel(const float* partial, int n, int d, float* dgamma, float* dbeta) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float* out = blockIdx.y ? dbeta : dgamma;
  if (!out) return;
  float v = 0.f;
  if (c < d)
    for (int b = threadIdx.y; b < n; b += 32) v += partial[((size_t)blockIdx.y * n + b) * d + c];
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = warp_sum(s[threadIdx.x][threadIdx.y]);
  const int cc = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && cc < d) out[cc] = v;
}

struct Shape {
  int vec;    // elements an access
  int warps;  // warps a row
  int vpt;    // accesses a thread
  int groups; // rows a block works on at a time
};

int round_up_pow2(int v, int lo) {
  int p = lo;
  while (p < v) p *= 2;
  return p;
}

Shape forward_shape(int d, int es) {
  Shape s{};
  s.vec = d * es % 16 == 0 ? 16 / es : 1;
  const int nv = d / s.vec;
  const int least = s.vec == 1 ? 4 : 1;
  s.vpt = round_up_pow2((nv + 255) / 256, least);
  if (s.vpt > 8 * least) s.vpt = 8 * least;
  s.warps = (nv + 32 * s.vpt - 1) / (32 * s.vpt);
  s.groups = s.warps >= 5 ? 1 : 8 / s.warps;
  return s;
}

Shape backward_shape(int d, int es) {
  Shape s{};
  s.vec = d * es % 16 == 0 ? 16 / es : 1;
  const int nv = d / s.vec;
  const int most = 16 / s.vec;  // at most 16 columns a thread: their sums stay in registers
  s.vpt = s.vec == 1 ? 4 : 1;
  while (s.vpt < most && (nv + s.vpt - 1) / s.vpt > 512) s.vpt *= 2;
  s.warps = (nv + 32 * s.vpt - 1) / (32 * s.vpt);
  s.groups = s.warps >= 9 ? 1 : s.warps == 1 ? 8 : 16 / s.warps > 8 ? 8 : 16 / s.warps;
  return s;
}

template <typename T, bool RMS, typename F>
cudaError_t by_shape(const Shape& s, const F& f) {
  constexpr int V = 16 / (int)sizeof(T);
  using std::integral_constant;
  if (s.vec == 1) {
    switch (s.vpt) {
      case 4: return f(integral_constant<int, 1>(), integral_constant<int, 4>());
      case 8: return f(integral_constant<int, 1>(), integral_constant<int, 8>());
      case 16: return f(integral_constant<int, 1>(), integral_constant<int, 16>());
      case 32: return f(integral_constant<int, 1>(), integral_constant<int, 32>());
    }
    return cudaErrorInvalidValue;
  }
  switch (s.vpt) {
    case 1: return f(integral_constant<int, V>(), integral_constant<int, 1>());
    case 2: return f(integral_constant<int, V>(), integral_constant<int, 2>());
    case 4: return f(integral_constant<int, V>(), integral_constant<int, 4>());
    case 8: return f(integral_constant<int, V>(), integral_constant<int, 8>());
  }
  return cudaErrorInvalidValue;
}

template <typename T, bool RMS>
cudaError_t forward(const moe_norm_desc& D, const void* x, const void* gamma, const void* beta,
                    void* y, float* mean, float* rstd, cudaStream_t st) {
  const Shape s = forward_shape(D.d, (int)sizeof(T));
  return by_shape<T, RMS>(s, [&](auto vec, auto vpt) {
    (void)launch_kernel(norm_forward_kernel<T, decltype(vec)::value, decltype(vpt)::value, RMS>,
                        (D.T + s.groups - 1) / s.groups, s.groups * s.warps * 32, 0, st,
                        static_cast<const T*>(x), gamma, beta, D.wdtype == MOE_BF16, D.T, D.d,
                        s.warps, D.eps, static_cast<T*>(y), mean, rstd);
    return cudaGetLastError();
  });
}

template <typename T, bool RMS>
cudaError_t backward(const moe_norm_desc& D, const void* dy, const void* x, const void* gamma,
                     const float* mean, const float* rstd, void* dx, float* partial, int blocks,
                     cudaStream_t st) {
  const Shape s = backward_shape(D.d, (int)sizeof(T));
  return by_shape<T, RMS>(s, [&](auto vec, auto vpt) -> cudaError_t {
    if constexpr (decltype(vec)::value * decltype(vpt)::value > 16) {
      return cudaErrorInvalidValue;
    } else {
      const size_t smem = partial && s.groups > 1 ? (size_t)D.d * 4 : 0;
      (void)launch_kernel(
          norm_backward_kernel<T, decltype(vec)::value, decltype(vpt)::value, RMS>, blocks,
          s.groups * s.warps * 32, smem, st, static_cast<const T*>(dy), static_cast<const T*>(x),
          gamma, D.wdtype == MOE_BF16, mean, rstd, D.T, D.d, s.warps, static_cast<T*>(dx),
          partial);
      return cudaGetLastError();
    }
  });
}

}  // namespace

int norm_backward_blocks(const moe_norm_desc& D) {
  const Shape s = backward_shape(D.d, (int)dtype_size(D.dtype));
  const int need = (D.T + s.groups - 1) / s.groups;
  return need < kBwdBlocks ? need : kBwdBlocks;
}

cudaError_t launch_norm_forward(const moe_norm_desc& D, const void* x, const void* gamma,
                                const void* beta, void* y, float* mean, float* rstd,
                                cudaStream_t s) {
  ProfScope pr("norm_forward", s);
  const bool rms = D.kind == MOE_NORM_RMS;
  if (D.dtype == MOE_BF16)
    return rms ? forward<__nv_bfloat16, true>(D, x, gamma, beta, y, mean, rstd, s)
               : forward<__nv_bfloat16, false>(D, x, gamma, beta, y, mean, rstd, s);
  return rms ? forward<float, true>(D, x, gamma, beta, y, mean, rstd, s)
             : forward<float, false>(D, x, gamma, beta, y, mean, rstd, s);
}

cudaError_t launch_norm_backward(const moe_norm_desc& D, const void* dy, const void* x,
                                 const void* gamma, const float* mean, const float* rstd,
                                 void* dx, float* dgamma, float* dbeta, float* partial,
                                 cudaStream_t s) {
  const bool rms = D.kind == MOE_NORM_RMS;
  const int blocks = norm_backward_blocks(D);
  if (!dgamma && !dbeta) partial = nullptr;
  cudaError_t e;
  {
    ProfScope pr("norm_backward", s);
    if (D.dtype == MOE_BF16)
      e = rms ? backward<__nv_bfloat16, true>(D, dy, x, gamma, mean, rstd, dx, partial, blocks, s)
              : backward<__nv_bfloat16, false>(D, dy, x, gamma, mean, rstd, dx, partial, blocks,
                                               s);
    else
      e = rms ? backward<float, true>(D, dy, x, gamma, mean, rstd, dx, partial, blocks, s)
              : backward<float, false>(D, dy, x, gamma, mean, rstd, dx, partial, blocks, s);
  }
  if (e != cudaSuccess || !partial) return e;
  ProfScope pr("norm_reduce", s);
  (void)launch_kernel(norm_reduce_kernel, dim3((D.d + 31) / 32, dbeta ? 2 : 1), dim3(32, 32), 0, s,
                      partial, blocks, D.d, dgamma, dbeta);
  return cudaGetLastError();
}

}  // namespace moe
