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
// vectors, of 4 in 4-byte ones, others (bf16, odd d) element by element.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kMaxGroupWarps = 32;
constexpr int kMaxStages = 8;
constexpr int kBwdBlocks = 304;  // most blocks of the backward pass: two an SM, or one of
                                 // more than 256 threads
constexpr size_t kBwdRingBytes = 104 * 1024;  // shared memory of the rings, two blocks an SM
constexpr size_t kFwdRingBytes = 204 * 1024;  // forward: the rings of all blocks of an SM
constexpr int kFwdRingRows = 608;             // forward: most blocks that take one row a group

// VEC consecutive elements of a row as they lie in memory (2, 4 or 16 bytes).
template <typename T, int VEC>
struct alignas(VEC * sizeof(T)) Raw {
  T e[VEC];
};
template <>
struct alignas(16) Raw<__nv_bfloat16, 8> {
  uint32_t w[4];
};
template <>
struct alignas(4) Raw<__nv_bfloat16, 2> {
  uint32_t w[1];
};

template <typename T, int VEC>
__device__ __forceinline__ void unpack(const Raw<T, VEC>& r, float* v) {
  if constexpr (sizeof(T) == 2 && VEC > 1) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      v[2 * i] = __uint_as_float(r.w[i] << 16);
      v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = load_as_f32(r.e, i);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> pack(const float* v) {
  Raw<T, VEC> r;
  if constexpr (sizeof(T) == 2 && VEC > 1) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      if constexpr (sizeof(T) == 2)
        r.e[i] = __float2bfloat16_rn(v[i]);
      else
        r.e[i] = v[i];
    }
  }
  return r;
}

template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T* p) {
  if constexpr (VEC * sizeof(T) == 16) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    Raw<T, VEC> r;
    *reinterpret_cast<uint4*>(&r) = a;
    return r;
  } else {
    return *reinterpret_cast<const Raw<T, VEC>*>(p);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_raw(T* p, const Raw<T, VEC>& r) {
  if constexpr (VEC * sizeof(T) == 16)
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&r);
  else
    *reinterpret_cast<Raw<T, VEC>*>(p) = r;
}

// VEC elements of a parameter vector (fp32 or bf16, whatever the rows are);
// null stands for `otherwise`.
template <int VEC>
__device__ __forceinline__ void load_param(const void* p, bool bf16, int c, float otherwise,
                                           float* v) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = otherwise;
  if (!p) return;
  if (bf16) {
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p) + c;
    if constexpr (VEC == 8 || VEC == 2) {
      unpack<__nv_bfloat16, VEC>(load_raw<__nv_bfloat16, VEC>(q), v);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = load_as_f32(q, i);
    }
  } else {
    const float* q = static_cast<const float*>(p) + c;
    if constexpr (VEC < 4) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = q[i];
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        const float4 a = *reinterpret_cast<const float4*>(q + i);
        v[i] = a.x, v[i + 1] = a.y, v[i + 2] = a.z, v[i + 3] = a.w;
      }
    }
  }
}

// Two fp32 values in a 64-bit register pair, for the packed fp32 instructions:
// the kernels below are bound by instruction issue before they are bound by
// HBM otherwise (the backward pass took 31 instructions an element and 116 us at
// 16384 x 4096 bf16 with one value an instruction).
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(F2 v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ float both(F2 v) {
  float a, b;
  split(v, a, b);
  return a + b;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The warp's sums of two values: in a lane of the lower half that of a, of the
// upper half that of b.  Five shuffles for both.
__device__ __forceinline__ float warp_sum2(float a, float b, int lane) {
  const bool up = lane & 16;
  float mine = up ? b : a;
  const float other = up ? a : b;
  mine += __shfl_xor_sync(0xffffffffu, other, 16);
#pragma unroll
  for (int o = 8; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  return mine;
}

// Sums of N (1 or 2) values over a group of `warps` warps, the same in every
// thread.  `buf` holds the warps' sums, [2][N][kMaxGroupWarps]; successive calls
// take its halves in turn, so one barrier a call is enough.  A group of several
// warps meets at named barrier 1 + group (at most 8 such groups).  Every thread
// adds the warps' sums in the same order.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int warps, int warp_in_group, int group,
                                          float* buf, int& turn) {
  const int lane = threadIdx.x & 31;
  float mine = N == 2 ? warp_sum2(v[0], v[N - 1], lane) : warp_sum(v[0]);
  if (warps > 1) {
    float* b = buf + turn * N * kMaxGroupWarps;
    turn ^= 1;
    if ((lane & (N == 2 ? 15 : 31)) == 0) b[(lane >> 4) * kMaxGroupWarps + warp_in_group] = mine;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(warps * 32) : "memory");
    if (warps <= 8) {  // each thread adds them up: no chain of shuffles
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float4 p = *reinterpret_cast<const float4*>(b + i * kMaxGroupWarps);
        const float4 q = *reinterpret_cast<const float4*>(b + i * kMaxGroupWarps + 4);
        const float s01 = p.x + p.y, s23 = (warps > 2 ? p.z : 0.f) + (warps > 3 ? p.w : 0.f);
        const float s45 = (warps > 4 ? q.x : 0.f) + (warps > 5 ? q.y : 0.f);
        const float s67 = (warps > 6 ? q.z : 0.f) + (warps > 7 ? q.w : 0.f);
        v[i] = (s01 + s23) + (s45 + s67);
      }
      return;
    }
    if constexpr (N == 2) {  // the lower half's lanes add up one value, the upper's the other
      const float* p = b + (lane >> 4) * kMaxGroupWarps;
      mine = ((lane & 15) < warps ? p[lane & 15] : 0.f) +
             ((lane & 15) + 16 < warps ? p[(lane & 15) + 16] : 0.f);
#pragma unroll
      for (int o = 8; o; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    } else {
      mine = warp_sum(lane < warps ? b[lane] : 0.f);
    }
  }
  if constexpr (N == 2) v[1] = __shfl_sync(0xffffffffu, mine, 16);
  v[0] = N == 2 ? __shfl_sync(0xffffffffu, mine, 0) : mine;
}

// `bytes` (a multiple of 16) from global into shared memory, asynchronously;
// completion is signalled on `bar` as transaction bytes.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// A group's ring of rows in shared memory, `streams` rows a stage, filled by
// bulk copies that one thread of the group requests `stages` rows ahead: HBM
// latency is hidden without registers, and a row's loads cost no instructions
// but its reads of shared memory.  Every wait for a copy is bounded.  The threads
// of a group wait each for itself, so some may give up on a row that the others
// still see arrive: one that has given up adds NaN to the sums of that row and of
// every row after it (backward: by its gamma), which makes NaN of these rows'
// results in all threads.  No more copies are requested then, and nobody waits for
// one that has not come.
struct Ring {
  uint8_t* base;
  uint32_t bar0, row_bytes;
  int streams, stages;
  int stage = 0;
  uint32_t parity = 0;
  int* gave_up;

  __device__ __forceinline__ Ring(uint8_t* dyn, uint64_t* bars, int* gave_up_, int group,
                                  int streams_, int stages_, uint32_t row_bytes_)
      : base(dyn + (size_t)group * stages_ * streams_ * row_bytes_),
        bar0(smem_u32(bars)),
        row_bytes(row_bytes_),
        streams(streams_),
        stages(stages_),
        gave_up(gave_up_) {}
  // by one thread of the group; a block barrier follows before any use
  __device__ __forceinline__ void init() const {
    for (int s = 0; s < stages; ++s) mbar_init(bar0 + 8u * s, 1);
    fence_barrier_init();
  }
  // by one thread of the group: the rows at a and b into stage s
  __device__ __forceinline__ void request(int s, const void* a, const void* b) const {
    const uint32_t dst = smem_u32(base) + (uint32_t)(s * streams) * row_bytes;
    mbar_arrive_expect_tx(bar0 + 8u * s, 2u * row_bytes);
    bulk_load(dst, a, row_bytes, bar0 + 8u * s);
    bulk_load(dst + row_bytes, b, row_bytes, bar0 + 8u * s);
  }
  // the same: n consecutive rows at a
  __device__ __forceinline__ void request_rows(int s, const void* a, int n) const {
    const uint32_t dst = smem_u32(base) + (uint32_t)(s * streams) * row_bytes;
    mbar_arrive_expect_tx(bar0 + 8u * s, (uint32_t)n * row_bytes);
    bulk_load(dst, a, (uint32_t)n * row_bytes, bar0 + 8u * s);
  }
  __device__ __forceinline__ bool wait() const {
    const uint32_t bar = bar0 + 8u * stage;
    return mbar_try_wait(bar, parity) || (open() && mbar_wait(bar, parity, gave_up, nullptr));
  }
  __device__ __forceinline__ bool open() const {
    return !*static_cast<volatile int*>(gave_up);
  }
  __device__ __forceinline__ const uint8_t* rows() const {
    return base + (size_t)stage * streams * row_bytes;
  }
  __device__ __forceinline__ void next() {
    if (++stage == stages) {
      stage = 0;
      parity ^= 1u;
    }
  }
  // leaves copies that are still on their way after giving up a bounded time to land
  __device__ __forceinline__ void close() const {
    if (open()) return;
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 100000ull) {
    }
  }
};

// ---------------------------------------------------------------- forward
// blockDim.x = groups * warps * 32; group g of block b takes R consecutive rows at
// a time, the (b * groups + g)-th R, + gridDim.x * groups, ...; the grid is at
// most what fits on the GPU at once.  With RING they come through a ring; rows of
// odd length, and few rows (a ring has nothing to run ahead of), are loaded where
// they are used.  A thread owns the same columns of every row and keeps their
// gamma and beta.
//
// Rows at a time.  A layer norm's bf16 rows are bound by the instructions that a
// row costs beside its elements (two sums with their barriers, the loop), so they
// are taken in twos: 16384 x 2048 31.5 -> 26.9 us, 8192 x 8192 65.5 -> 50.0.  An RMS
// norm has one sum and gains more from the blocks that the registers then allow:
// one row at a time against two, bf16 4096 x 7168 20.1 and 22.5 us (16384 x 4096, the
// other way round, 49.8 and 45.1), fp32 8192 x 4096 46.3 and 52.4.  For a layer norm of
// fp32 rows both take 48.7 there.
template <typename T, bool RMS, bool RING, int THREADS>
__host__ __device__ constexpr int forward_rows() {
  return RING && !RMS && sizeof(T) == 2 && THREADS == 512 ? 2 : 1;
}

template <typename T, int VEC, int VPT, bool RMS, bool RING, int THREADS>
__global__ void __launch_bounds__(THREADS, RMS && THREADS == 512 ? 2 : 1)
    norm_forward_kernel(const T* x, const void* gamma, const void* beta, bool w_bf16, int rows,
                        int d, int warps, int stages, float eps, T* y, float* mean,
                        float* rstd) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ alignas(16) float red[8][4 * kMaxGroupWarps];
  __shared__ __align__(8) uint64_t bars[8][kMaxStages];
  __shared__ int gave_up;
  constexpr int N = VPT * VEC, R = forward_rows<T, RMS, RING, THREADS>();
  const int gt = warps * 32, groups = blockDim.x / gt;
  const int group = threadIdx.x / gt, tid = threadIdx.x - group * gt;
  const int step = gridDim.x * groups * R;
  const int nv = d / VEC;
  int row = (blockIdx.x * groups + group) * R;
  Ring ring(dyn, bars[group], &gave_up, group, R, stages, (uint32_t)d * sizeof(T));
  if constexpr (RING) {
    if (threadIdx.x == 0) gave_up = 0;
    if (tid == 0) ring.init();
    __syncthreads();
    if (tid == 0)
      for (int s = 0; s < stages && row + s * step < rows; ++s)
        ring.request_rows(s, x + (size_t)(row + s * step) * d, min(R, rows - row - s * step));
  }
  F2 g[N / 2], b[RMS ? 1 : N / 2];
  auto params = [&](const void* p, float otherwise, F2* out) {
    float v[N];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i * VEC + j] = 0.f;
      if (tid + i * gt < nv)
        load_param<VEC>(p, w_bf16, (tid + i * gt) * VEC, otherwise, v + i * VEC);
    }
#pragma unroll
    for (int k = 0; k < N / 2; ++k) out[k] = f2(v[2 * k], v[2 * k + 1]);
  };
  params(gamma, 1.f, g);
  if constexpr (!RMS) params(beta, 0.f, b);
  const float inv_d = 1.f / (float)d;
  int turn = 0;
  float* buf = red[warps == 1 ? 0 : group];
  bool ok = true;  // this thread has not given up waiting
  for (; row < rows; row += step) {  // the same rows for a whole group
    const int have = min(R, rows - row);
    const T* xr = x + (size_t)row * d;
    if constexpr (RING) {
      ok = ok && ring.wait();
      xr = reinterpret_cast<const T*>(ring.rows());
    }
    F2 v[R][N / 2];  // zero beyond a row's end
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float f[N];
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        Raw<T, VEC> raw{};
        if (tid + i * gt < nv && q < have)
          raw = load_raw<T, VEC>(xr + (size_t)q * d + (size_t)(tid + i * gt) * VEC);
        unpack<T, VEC>(raw, f + i * VEC);
      }
#pragma unroll
      for (int k = 0; k < N / 2; ++k) v[q][k] = f2(f[2 * k], f[2 * k + 1]);
    }
    if constexpr (RING) {
      fence_proxy_async_shared();  // before the barrier that hands the stage back
      if (warps == 1) __syncwarp();
    }
    float s[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      F2 acc = f2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < N / 2; ++k) acc = RMS ? fma2(v[q][k], v[q][k], acc) : add2(v[q][k], acc);
      s[q] = ok ? both(acc) : quiet_nan();
    }
    group_sum<R>(s, warps, tid >> 5, group, buf, turn);
    if constexpr (RING) {
      if (tid == 0 && row + (long long)stages * step < rows && ring.open())
        ring.request_rows(ring.stage, x + (size_t)(row + stages * step) * d,
                          min(R, rows - row - stages * step));
      ring.next();
    }
    float mu[R];
#pragma unroll
    for (int q = 0; q < R; ++q) mu[q] = 0.f;
    if constexpr (!RMS) {
      const bool full = nv == gt * VPT;  // else the columns beyond the end would add mu^2 each
#pragma unroll
      for (int q = 0; q < R; ++q) {
        mu[q] = s[q] * inv_d;
        const F2 m = f2(-mu[q], -mu[q]);
        F2 acc = f2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
          v[q][k] = add2(v[q][k], m);
          if (!full) {
            float lo, hi;
            split(v[q][k], lo, hi);
            v[q][k] = f2(tid + (2 * k / VEC) * gt < nv ? lo : 0.f,
                         tid + ((2 * k + 1) / VEC) * gt < nv ? hi : 0.f);
          }
          acc = fma2(v[q][k], v[q][k], acc);
        }
        s[q] = both(acc);
      }
      group_sum<R>(s, warps, tid >> 5, group, buf, turn);
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (q >= have) break;
      const float r = 1.f / sqrtf(s[q] * inv_d + eps);
      if (tid == 0) {
        if (mean) mean[row + q] = mu[q];
        if (rstd) rstd[row + q] = r;
      }
      const F2 rr = f2(r, r);
      float o[N];
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        const F2 h = mul2(v[q][k], rr);
        if constexpr (RMS)
          split(mul2(h, g[k]), o[2 * k], o[2 * k + 1]);
        else
          split(fma2(h, g[k], b[k]), o[2 * k], o[2 * k + 1]);
      }
      T* yr = y + (size_t)(row + q) * d;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (tid + i * gt < nv)
          store_raw<T, VEC>(yr + (size_t)(tid + i * gt) * VEC, pack<T, VEC>(o + i * VEC));
    }
  }
  if constexpr (RING) ring.close();
}

// ---------------------------------------------------------------- backward
// Block b takes rows b * groups + group, + gridDim.x * groups, ...; a thread
// owns the same columns of every row and keeps their sums of dy h and dy in
// registers.  With RING (rows of 16-byte vectors) x and dy come through a ring;
// the barrier of the row's sums also says that every thread has read the
// stage.  Other rows are loaded where they are used.  At the end the groups'
// sums are added in group order through shared memory and written to
// partial [2][gridDim.x][d].
template <typename T, int VEC, int VPT, bool RMS, bool RING, int THREADS>
__global__ void __launch_bounds__(THREADS, 1)
    norm_backward_kernel(const T* dy, const T* x, const void* gamma, bool w_bf16,
                         const float* mean, const float* rstd, int rows, int d, int warps,
                         int stages, T* dx, float* partial) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(128) uint8_t dyn[];  // the rings, then the groups' sums [d]
  __shared__ alignas(16) float red[8][4 * kMaxGroupWarps];
  __shared__ __align__(8) uint64_t bars[8][kMaxStages];
  __shared__ int gave_up;
  constexpr int N = VPT * VEC;
  const int gt = warps * 32, groups = blockDim.x / gt;
  const int group = threadIdx.x / gt, tid = threadIdx.x - group * gt;
  const int nv = d / VEC;
  const int step = gridDim.x * groups;
  int row = blockIdx.x * groups + group;
  Ring ring(dyn, bars[group], &gave_up, group, 2, stages, (uint32_t)d * sizeof(T));
  if constexpr (RING) {
    if (threadIdx.x == 0) gave_up = 0;
    if (tid == 0) ring.init();
    __syncthreads();
    if (tid == 0)
      for (int s = 0; s < stages && row + s * step < rows; ++s)
        ring.request(s, x + (size_t)(row + s * step) * d, dy + (size_t)(row + s * step) * d);
  }

  // pairs of this thread's columns; columns beyond the row's end hold zeros in
  // dy, so they add nothing to the row's sums, and are never stored
  F2 g[N / 2], dg[N / 2], db[N / 2];
  {
    float gv[N];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) gv[i * VEC + j] = 0.f;
      if (tid + i * gt < nv)
        load_param<VEC>(gamma, w_bf16, (tid + i * gt) * VEC, 1.f, gv + i * VEC);
    }
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
      g[k] = f2(gv[2 * k], gv[2 * k + 1]);
      dg[k] = db[k] = f2(0.f, 0.f);
    }
  }
  const float inv_d = -1.f / (float)d;
  const T* xp = x + (size_t)row * d + (size_t)tid * VEC;
  const T* dp = dy + (size_t)row * d + (size_t)tid * VEC;
  T* op = dx + (size_t)row * d + (size_t)tid * VEC;
  const size_t jump = (size_t)step * d;
  int turn = 0;
  float* buf = red[warps == 1 ? 0 : group];
  float mu = 0.f, r = 0.f;
  if (row < rows) mu = RMS ? 0.f : mean[row], r = rstd[row];
  for (; row < rows; row += step, xp += jump, dp += jump, op += jump) {
    float mu2 = 0.f, r2 = 0.f;  // the next row's, loaded ahead
    if (row + step < rows) mu2 = RMS ? 0.f : mean[row + step], r2 = rstd[row + step];
    Raw<T, VEC> xr[VPT], dr[VPT];
    if constexpr (RING) {
      if (!ring.wait()) g[0] = f2(quiet_nan(), quiet_nan());
      const uint8_t* src = ring.rows() + (size_t)tid * sizeof(Raw<T, VEC>);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        xr[i] = dr[i] = Raw<T, VEC>{};
        if (tid + i * gt < nv) {
          const T* p = reinterpret_cast<const T*>(src + (size_t)i * gt * sizeof(Raw<T, VEC>));
          xr[i] = load_raw<T, VEC>(p);
          dr[i] = load_raw<T, VEC>(p + d);
        }
      }
      fence_proxy_async_shared();  // before the barrier that hands the stage back
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        xr[i] = dr[i] = Raw<T, VEC>{};
        if (tid + i * gt < nv) {
          xr[i] = load_raw<T, VEC>(xp + (size_t)i * gt * VEC);
          dr[i] = load_raw<T, VEC>(dp + (size_t)i * gt * VEC);
        }
      }
    }
    float xv[N], dv[N];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      unpack<T, VEC>(xr[i], xv + i * VEC);
      unpack<T, VEC>(dr[i], dv + i * VEC);
    }
    F2 h[N / 2], w[N / 2];
    F2 wh = f2(0.f, 0.f), ws = f2(0.f, 0.f);
    const F2 rr = f2(r, r), m = f2(-mu, -mu);
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
      const F2 x2 = f2(xv[2 * k], xv[2 * k + 1]), d2 = f2(dv[2 * k], dv[2 * k + 1]);
      h[k] = mul2(RMS ? x2 : add2(x2, m), rr);
      dg[k] = fma2(d2, h[k], dg[k]);
      w[k] = mul2(d2, g[k]);
      wh = fma2(w[k], h[k], wh);
      if (!RMS) {
        db[k] = add2(d2, db[k]);
        ws = add2(w[k], ws);
      }
    }
    float s[RMS ? 1 : 2];
    s[0] = both(wh);
    if constexpr (!RMS) s[1] = both(ws);
    if (RING && warps == 1) __syncwarp();
    group_sum<RMS ? 1 : 2>(s, warps, tid >> 5, group, buf, turn);
    if constexpr (RING) {
      if (tid == 0 && row + (long long)stages * step < rows && ring.open()) {
        const size_t at = (size_t)(row + stages * step) * d;
        ring.request(ring.stage, x + at, dy + at);
      }
      ring.next();
    }
    const float c1 = s[0] * inv_d;
    const F2 n1 = f2(c1, c1);
#pragma unroll
    for (int k = 0; k < N / 2; ++k) {
      F2 t = fma2(h[k], n1, w[k]);
      if constexpr (!RMS) t = add2(t, f2(s[1] * inv_d, s[1] * inv_d));
      split(mul2(t, rr), dv[2 * k], dv[2 * k + 1]);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (tid + i * gt < nv)
        store_raw<T, VEC>(op + (size_t)i * gt * VEC, pack<T, VEC>(dv + i * VEC));
    mu = mu2, r = r2;
  }
  if constexpr (RING) ring.close();
  if (!partial) return;
  bool lost = false;
  if constexpr (RING) {
    __syncthreads();
    lost = !ring.open();
  }
  float* sums = reinterpret_cast<float*>(dyn);  // every copy has landed and been read
  auto flush = [&](const F2 (&acc2)[N / 2], float* out) {
    float acc[N];
#pragma unroll
    for (int k = 0; k < N / 2; ++k) split(acc2[k], acc[2 * k], acc[2 * k + 1]);
    if (lost) {
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] = quiet_nan();
    }
    for (int k = 0; k < groups; ++k) {
      __syncthreads();
      if (group != k) continue;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * gt;
        if (c < nv) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float v = k ? sums[c * VEC + j] + acc[i * VEC + j] : acc[i * VEC + j];
            if (k < groups - 1)
              sums[c * VEC + j] = v;
            else
              acc[i * VEC + j] = v;
          }
          if (k == groups - 1) {
            if constexpr (VEC >= 4) {
#pragma unroll
              for (int j = 0; j < VEC; j += 4)
                *reinterpret_cast<float4*>(out + c * VEC + j) =
                    make_float4(acc[i * VEC + j], acc[i * VEC + j + 1], acc[i * VEC + j + 2],
                                acc[i * VEC + j + 3]);
            } else {
#pragma unroll
              for (int j = 0; j < VEC; ++j) out[c * VEC + j] = acc[i * VEC + j];
            }
          }
        }
      }
    }
  };
  flush(dg, partial + (size_t)blockIdx.x * d);
  if (!RMS) flush(db, partial + (size_t)(gridDim.x + blockIdx.x) * d);
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

int vector_of(int d, int es) {
  const int bytes = d * es;
  return bytes % 16 == 0 ? 16 / es : bytes % 4 == 0 ? 4 / es : 1;
}

// 16 columns a thread at most, so that what it keeps of them (parameters, sums)
// stays in registers.
Shape row_shape(int d, int es) {
  Shape s{};
  s.vec = vector_of(d, es);
  const int nv = d / s.vec;
  s.vpt = s.vec * es == 16 ? 1 : 4;
  while (s.vpt * s.vec < 16 && nv > 32 * s.vpt) s.vpt *= 2;
  s.warps = (nv + 32 * s.vpt - 1) / (32 * s.vpt);
  s.groups = s.warps >= 5 ? 1 : 8 / s.warps;
  return s;
}

// f(elements an access, accesses a thread) as constants.
template <typename T, typename F>
cudaError_t by_shape(const Shape& s, const F& f) {
  constexpr int V = 16 / (int)sizeof(T), V4 = 4 / (int)sizeof(T);
  using std::integral_constant;
  if (s.vec == V) {
    if (s.vpt == 1) return f(integral_constant<int, V>(), integral_constant<int, 1>());
    if (s.vpt == 2) return f(integral_constant<int, V>(), integral_constant<int, 2>());
    if constexpr (V == 4)
      if (s.vpt == 4) return f(integral_constant<int, V>(), integral_constant<int, 4>());
  } else if (s.vec == V4) {
    if (s.vpt == 4) return f(integral_constant<int, V4>(), integral_constant<int, 4>());
    if (s.vpt == 8) return f(integral_constant<int, V4>(), integral_constant<int, 8>());
    if constexpr (V4 == 1)
      if (s.vpt == 16) return f(integral_constant<int, V4>(), integral_constant<int, 16>());
  } else if constexpr (V4 > 1) {
    if (s.vpt == 4) return f(integral_constant<int, 1>(), integral_constant<int, 4>());
    if (s.vpt == 8) return f(integral_constant<int, 1>(), integral_constant<int, 8>());
    if (s.vpt == 16) return f(integral_constant<int, 1>(), integral_constant<int, 16>());
  }
  return cudaErrorInvalidValue;
}

// Stages of a ring in `room` bytes, at most kMaxStages.
int ring_stages(size_t room, size_t stage) {
  const size_t n = room / stage;
  return n < 1 ? 1 : n > kMaxStages ? kMaxStages : (int)n;
}

// Dynamic shared memory beyond the default limit, asked for once a device.
template <typename K>
cudaError_t allow_smem(K kern, size_t most, std::atomic<bool> (&configured)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (configured[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e == cudaSuccess) configured[dev] = true;
  return e;
}

template <typename T, int VEC, int VPT, bool RMS, bool RING, int THREADS>
cudaError_t launch_forward(const moe_norm_desc& D, const Shape& s, const void* x,
                           const void* gamma, const void* beta, void* y, float* mean, float* rstd,
                           cudaStream_t st) {
  auto kern = norm_forward_kernel<T, VEC, VPT, RMS, RING, THREADS>;
  const int threads = s.groups * s.warps * 32;
  constexpr int R = forward_rows<T, RMS, RING, THREADS>();
  const size_t stage = (size_t)s.groups * R * D.d * sizeof(T);
  int blocks = (D.T + s.groups * R - 1) / (s.groups * R), stages = 0;
  // what the registers allow at once: layer norm keeps beta too
  const int per_sm = threads <= 256 ? (RMS ? 4 : 2) : threads <= 512 && RMS ? 2 : 1;
  if (RING) {
    static std::atomic<bool> configured[64] = {};
    const cudaError_t e = allow_smem(kern, kFwdRingBytes, configured);
    if (e != cudaSuccess) return e;
    stages = ring_stages(kFwdRingBytes / per_sm, stage);
  }
  if (blocks > per_sm * num_sms()) blocks = per_sm * num_sms();
  (void)launch_kernel(kern, blocks, threads, stages * stage, st, static_cast<const T*>(x), gamma,
                      beta, D.wdtype == MOE_BF16, D.T, D.d, s.warps, stages, D.eps,
                      static_cast<T*>(y), mean, rstd);
  return cudaGetLastError();
}

// f(elements an access, accesses a thread, the block's largest size): more
// than 8192 columns take 1024 threads.
template <typename T, typename F>
cudaError_t by_threads(const Shape& s, const F& f) {
  return by_shape<T>(s, [&](auto vec, auto vpt) -> cudaError_t {
    if constexpr (decltype(vec)::value * decltype(vpt)::value == 16)
      if (s.warps > 16) return f(vec, vpt, std::integral_constant<int, 1024>());
    return f(vec, vpt, std::integral_constant<int, 512>());
  });
}

template <typename T, bool RMS>
cudaError_t forward(const moe_norm_desc& D, const void* x, const void* gamma, const void* beta,
                    void* y, float* mean, float* rstd, cudaStream_t st) {
  const Shape s = row_shape(D.d, (int)sizeof(T));
  return by_threads<T>(s, [&](auto vec, auto vpt, auto threads) -> cudaError_t {
    constexpr int VEC = decltype(vec)::value, VPT = decltype(vpt)::value;
    constexpr int THREADS = decltype(threads)::value;
    if constexpr (VEC * sizeof(T) == 16) {
      if (D.T > kFwdRingRows * s.groups)
        return launch_forward<T, VEC, VPT, RMS, true, THREADS>(D, s, x, gamma, beta, y, mean,
                                                               rstd, st);
    }
    return launch_forward<T, VEC, VPT, RMS, false, THREADS>(D, s, x, gamma, beta, y, mean, rstd,
                                                            st);
  });
}

template <typename T, int VEC, int VPT, bool RMS, int THREADS>
cudaError_t launch_backward(const moe_norm_desc& D, const Shape& s, const void* dy, const void* x,
                            const void* gamma, const float* mean, const float* rstd, void* dx,
                            float* partial, int blocks, cudaStream_t st) {
  constexpr bool RING = VEC * sizeof(T) == 16;
  auto kern = norm_backward_kernel<T, VEC, VPT, RMS, RING, THREADS>;
  const int threads = s.groups * s.warps * 32;
  const size_t stage = 2 * (size_t)s.groups * D.d * sizeof(T);
  int stages = 0;
  if (RING)  // a block's share of an SM's shared memory; all of it for one of > 256 threads
    stages = ring_stages(threads > 256 ? 2 * kBwdRingBytes : kBwdRingBytes, stage);
  const size_t sums = s.groups > 1 ? (size_t)D.d * 4 : 0;
  const size_t smem = stages * stage > sums ? stages * stage : sums;
  if (RING) {
    static std::atomic<bool> configured[64] = {};
    const cudaError_t e = allow_smem(kern, 2 * kBwdRingBytes, configured);
    if (e != cudaSuccess) return e;
  }
  (void)launch_kernel(kern, blocks, threads, smem, st, static_cast<const T*>(dy),
                      static_cast<const T*>(x), gamma, D.wdtype == MOE_BF16, mean, rstd, D.T,
                      D.d, s.warps, stages, static_cast<T*>(dx), partial);
  return cudaGetLastError();
}

template <typename T, bool RMS>
cudaError_t backward(const moe_norm_desc& D, const void* dy, const void* x, const void* gamma,
                     const float* mean, const float* rstd, void* dx, float* partial, int blocks,
                     cudaStream_t st) {
  const Shape s = row_shape(D.d, (int)sizeof(T));
  return by_threads<T>(s, [&](auto vec, auto vpt, auto threads) {
    return launch_backward<T, decltype(vec)::value, decltype(vpt)::value, RMS,
                           decltype(threads)::value>(D, s, dy, x, gamma, mean, rstd, dx, partial,
                                                     blocks, st);
  });
}

}  // namespace

int norm_backward_blocks(const moe_norm_desc& D) {
  const Shape s = row_shape(D.d, (int)dtype_size(D.dtype));
  const int need = (D.T + s.groups - 1) / s.groups;
  const int most = s.groups * s.warps > 8 ? kBwdBlocks / 2 : kBwdBlocks;
  return need < most ? need : most;
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
