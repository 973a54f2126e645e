// swiglu.cu -- the activation between the experts' products, for training, with
// its inputs kept in 8 bits (fp8.cuh) for the backward pass.
//
//   forward   h = silu(g) * u;  optionally the codes and scales of g and u
//   backward  sigma = 1 / (1 + exp(-g)),  dg = dh * u * sigma * (1 + g (1 - sigma)),
//             du = dh * g * sigma,  h again if wanted
// element by element, in fp32, each result rounded once.  Both passes are bound
// by memory: bf16 rows move 8.06 bytes an element forward with packing (4 read,
// 2 of h and 2.06 of codes and scales written), 8.06 backward (10.06 with h).
// 16 threads have a block of 128 columns in hand, so that its largest is four
// shuffles.  131072 x 1536 forward 254 us (6.4 TB/s), 36864 x 2048 backward with h
// 113 us (6.7 TB/s).  The number of thread blocks decides (8, 32, 64 an SM: 290, 257,
// 254 us forward); two blocks of columns at once a thread: 276 us, a division a block
// of columns instead of the walk: 285 us.
#include <cuda_bf16.h>

#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kSegs = kThreads / 16;  // blocks of 128 columns that a thread block has in hand

// Eight values of a block of 128 columns by one of its 16 threads: eight columns
// in a row (VEC), or every sixteenth.
template <bool VEC>
__device__ __forceinline__ int col(int lane, int j) {
  return VEC ? lane * 8 + j : lane + 16 * j;
}

template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* __restrict__ p, int lane, int n, float (&v)[8]) {
  if (VEC) {
    const int c = lane * 8;
    if (c >= n) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
      return;
    }
    if (sizeof(T) == 2) {
      const uint4 w = __ldcs(reinterpret_cast<const uint4*>(p + c));
      const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(a[j] << 16);
        v[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
      }
    } else {
      const float4 a = __ldcs(reinterpret_cast<const float4*>(p + c));
      const float4 b = __ldcs(reinterpret_cast<const float4*>(p + c + 4));
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = col<VEC>(lane, j) < n ? load_as_f32(p, col<VEC>(lane, j)) : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void load_codes8(const uint8_t* __restrict__ q, float scale, int lane,
                                            int n, float (&v)[8]) {
  if (VEC) {
    const int c = lane * 8;
    const uint2 k =
        c < n ? __ldcs(reinterpret_cast<const uint2*>(q + c)) : make_uint2(0u, 0u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = fp8::values2(((j < 2 ? k.x : k.y) >> (16 * (j & 1))) & 0xffffu);
      v[2 * j] = f.x * scale;
      v[2 * j + 1] = f.y * scale;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = col<VEC>(lane, j) < n ? fp8::values2(q[col<VEC>(lane, j)]).x * scale : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store_codes8(uint8_t* __restrict__ q, int lane, int n,
                                             const float (&v)[8], float inv) {
  if (VEC) {
    if (lane * 8 < n)
      __stcs(reinterpret_cast<uint2*>(q + lane * 8),
             make_uint2(fp8::codes4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                        fp8::codes4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv)));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col<VEC>(lane, j) < n) q[col<VEC>(lane, j)] = (uint8_t)fp8::codes2(v[j] * inv, 0.f);
  }
}

template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* __restrict__ p, int lane, int n, const float (&v)[8]) {
  if (VEC) {
    const int c = lane * 8;
    if (c >= n) return;
    if (sizeof(T) == 2) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        o[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      __stcs(reinterpret_cast<uint4*>(p + c), make_uint4(o[0], o[1], o[2], o[3]));
    } else {
      __stcs(reinterpret_cast<float4*>(p + c), make_float4(v[0], v[1], v[2], v[3]));
      __stcs(reinterpret_cast<float4*>(p + c + 4), make_float4(v[4], v[5], v[6], v[7]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col<VEC>(lane, j) < n) p[col<VEC>(lane, j)] = (T)v[j];
  }
}

// 1 / (1 + exp(-z)): the fast exponential and division where the result is rounded
// to bf16.  Their documented errors, 2 + 1.173 |z| and 2 steps of 2^-23, make at most
// 107 steps at |z| = 88, 1.3e-5: a three-hundredth of bf16's 2^-8.  Below z = -87.3 the
// divisor exceeds 2^126 and the result is 0: the sigmoid left out is below 2^-126.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
  return sizeof(T) == 2 ? __fdividef(1.0f, 1.0f + __expf(-z)) : 1.0f / (1.0f + expf(-z));
}

__device__ __forceinline__ uint32_t amax16(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, fp8::abs_bits(v[j]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// A walk over the blocks of 128 columns of all rows, `step` blocks at a time.
struct Walk {
  long long r;  // row
  int b;        // block of the row
  long long dr;
  int db, nb, I;
  __device__ __forceinline__ Walk(long long first, long long step, int I)
      : nb(fp8::blocks_of(I)), I(I) {
    r = first / nb, b = (int)(first - r * nb);
    dr = step / nb, db = (int)(step - dr * nb);
  }
  __device__ __forceinline__ size_t at() const {  // its first element
    return (size_t)r * I + (size_t)b * fp8::kBlock;
  }
  __device__ __forceinline__ int n() const { return min(fp8::kBlock, I - b * fp8::kBlock); }
  __device__ __forceinline__ void next() {
    r += dr;
    if ((b += db) >= nb) b -= nb, ++r;
  }
};

template <bool VEC, bool PACK, typename T>
__global__ void __launch_bounds__(kThreads)
    swiglu_forward_kernel(const T* __restrict__ gate, const T* __restrict__ up, long long segs,
                          int I, T* __restrict__ h, uint8_t* __restrict__ gate8,
                          float* __restrict__ gate_scale, uint8_t* __restrict__ up8,
                          float* __restrict__ up_scale) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 15;
  const long long step = (long long)gridDim.x * kSegs;
  long long i = (long long)blockIdx.x * kSegs + threadIdx.x / 16;
  Walk walk(i, step, I);
  // every thread runs every round: a block's maximum is a shuffle of whole warps
  for (long long base = (long long)blockIdx.x * kSegs; base < segs; base += step) {
    const bool there = i < segs;
    const size_t at = there ? walk.at() : 0;
    const int n = there ? walk.n() : 0;
    float g[8], u[8], y[8];
    load8<VEC>(gate + at, lane, n, g);
    load8<VEC>(up + at, lane, n, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = g[j] * sigmoid<T>(g[j]) * u[j];
    store8<VEC>(h + at, lane, n, y);
    if (PACK) {
      const fp8::Scale a = fp8::scale_of(amax16(g)), b = fp8::scale_of(amax16(u));
      store_codes8<VEC>(gate8 + at, lane, n, g, a.inv);
      store_codes8<VEC>(up8 + at, lane, n, u, b.inv);
      if (lane == 0 && there) {
        gate_scale[i] = a.scale;
        up_scale[i] = b.scale;
      }
    }
    walk.next();
    i += step;
  }
}

template <bool VEC, bool PACKED, typename T>
__global__ void __launch_bounds__(kThreads)
    swiglu_backward_kernel(const T* __restrict__ dh, const T* __restrict__ gate,
                           const T* __restrict__ up, const uint8_t* __restrict__ gate8,
                           const float* __restrict__ gate_scale, const uint8_t* __restrict__ up8,
                           const float* __restrict__ up_scale, long long segs, int I,
                           T* __restrict__ dgate, T* __restrict__ dup, T* __restrict__ h) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 15;
  const long long step = (long long)gridDim.x * kSegs;
  long long i = (long long)blockIdx.x * kSegs + threadIdx.x / 16;
  Walk walk(i, step, I);
  for (; i < segs; i += step, walk.next()) {
    const size_t at = walk.at();
    const int n = walk.n();
    float g[8], u[8], d[8];
    if (PACKED) {
      load_codes8<VEC>(gate8 + at, gate_scale[i], lane, n, g);
      load_codes8<VEC>(up8 + at, up_scale[i], lane, n, u);
    } else {
      load8<VEC>(gate + at, lane, n, g);
      load8<VEC>(up + at, lane, n, u);
    }
    load8<VEC>(dh + at, lane, n, d);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float sg = sigmoid<T>(g[j]);
      const float act = g[j] * sg;  // silu
      const float slope = sg * (1.0f + g[j] * (1.0f - sg));
      y[j] = act * u[j];
      g[j] = d[j] * u[j] * slope;
      u[j] = d[j] * act;
    }
    store8<VEC>(dgate + at, lane, n, g);
    store8<VEC>(dup + at, lane, n, u);
    if (h) store8<VEC>(h + at, lane, n, y);
  }
}

unsigned seg_grid(long long segs) {
  const long long most = (long long)num_sms() * 64, need = (segs + kSegs - 1) / kSegs;
  return (unsigned)(need < most ? need : most);
}

template <typename T>
void forward(const void* gate, const void* up, long long segs, int I, void* h, void* gate8,
             float* gate_scale, void* up8, float* up_scale, cudaStream_t s) {
  auto kern = I % 8 == 0 ? (gate8 ? swiglu_forward_kernel<true, true, T>
                                  : swiglu_forward_kernel<true, false, T>)
                         : (gate8 ? swiglu_forward_kernel<false, true, T>
                                  : swiglu_forward_kernel<false, false, T>);
  (void)launch_kernel(kern, seg_grid(segs), kThreads, 0, s, static_cast<const T*>(gate),
                      static_cast<const T*>(up), segs, I, static_cast<T*>(h),
                      static_cast<uint8_t*>(gate8), gate_scale, static_cast<uint8_t*>(up8),
                      up_scale);
}

template <typename T>
void backward(const void* dh, const void* gate, const void* up, const void* gate8,
              const float* gate_scale, const void* up8, const float* up_scale, long long segs,
              int I, void* dgate, void* dup, void* h, cudaStream_t s) {
  auto kern = I % 8 == 0 ? (gate8 ? swiglu_backward_kernel<true, true, T>
                                  : swiglu_backward_kernel<true, false, T>)
                         : (gate8 ? swiglu_backward_kernel<false, true, T>
                                  : swiglu_backward_kernel<false, false, T>);
  (void)launch_kernel(kern, seg_grid(segs), kThreads, 0, s, static_cast<const T*>(dh),
                      static_cast<const T*>(gate), static_cast<const T*>(up),
                      static_cast<const uint8_t*>(gate8), gate_scale,
                      static_cast<const uint8_t*>(up8), up_scale, segs, I,
                      static_cast<T*>(dgate), static_cast<T*>(dup), static_cast<T*>(h));
}

}  // namespace

cudaError_t launch_swiglu_forward(int dtype, const void* gate, const void* up, long long rows,
                                  int I, void* h, void* gate8, float* gate_scale, void* up8,
                                  float* up_scale, cudaStream_t s) {
  const long long segs = rows * fp8::blocks_of(I);
  if (segs == 0) return cudaSuccess;
  ProfScope pr("swiglu_forward", s);
  if (dtype == MOE_BF16)
    forward<__nv_bfloat16>(gate, up, segs, I, h, gate8, gate_scale, up8, up_scale, s);
  else
    forward<float>(gate, up, segs, I, h, gate8, gate_scale, up8, up_scale, s);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_backward(int dtype, const void* dh, const void* gate, const void* up,
                                   const void* gate8, const float* gate_scale, const void* up8,
                                   const float* up_scale, long long rows, int I, void* dgate,
                                   void* dup, void* h, cudaStream_t s) {
  const long long segs = rows * fp8::blocks_of(I);
  if (segs == 0) return cudaSuccess;
  ProfScope pr("swiglu_backward", s);
  if (dtype == MOE_BF16)
    backward<__nv_bfloat16>(dh, gate, up, gate8, gate_scale, up8, up_scale, segs, I, dgate, dup,
                            h, s);
  else
    backward<float>(dh, gate, up, gate8, gate_scale, up8, up_scale, segs, I, dgate, dup, h, s);
  return cudaGetLastError();
}

}  // namespace moe
