// fp8_rows.cu -- rows and weights into 8 bits and back (the format: fp8.cuh).
#include <cuda_bf16.h>

#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kSegs = kThreads / 16;  // blocks of 128 columns that a thread block has in hand
constexpr long long kCopyElements = 1ll << 23;

// Eight values of a block of 128 columns by one of its 16 threads.  VEC: eight
// columns in a row, by 16-byte loads; else every sixteenth column, so that rows
// may begin anywhere.  Columns from n on are zero.
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
      const uint4 w = *reinterpret_cast<const uint4*>(p + c);
      const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(a[j] << 16);
        v[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
      }
    } else {
      const float4 a = *reinterpret_cast<const float4*>(p + c);
      const float4 b = *reinterpret_cast<const float4*>(p + c + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = lane + 16 * j < n ? load_as_f32(p, lane + 16 * j) : 0.f;
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(uint8_t* __restrict__ q, int lane, int n,
                                       const float (&v)[8], float inv) {
  if (VEC) {
    if (lane * 8 < n)
      *reinterpret_cast<uint2*>(q + lane * 8) =
          make_uint2(fp8::codes4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                     fp8::codes4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (lane + 16 * j < n) q[lane + 16 * j] = (uint8_t)fp8::codes2(v[j] * inv, 0.f);
  }
}

__device__ __forceinline__ uint32_t amax16(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, fp8::abs_bits(v[j]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// q, scale of x [rows, n]: 16 threads a block of 128 columns.
template <bool VEC, typename T>
__global__ void __launch_bounds__(kThreads) pack_rows_kernel(const T* __restrict__ x,
                                                             long long segs, int n,
                                                             uint8_t* __restrict__ q,
                                                             float* __restrict__ scale) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 15;
  const int nb = fp8::blocks_of(n);
  // every thread runs every round: the block's maximum is a shuffle of whole warps
  for (long long base = (long long)blockIdx.x * kSegs; base < segs;
       base += (long long)gridDim.x * kSegs) {
    const long long s = base + threadIdx.x / 16;
    const bool there = s < segs;
    const long long r = there ? s / nb : 0;
    const int b = there ? (int)(s - r * nb) : 0;
    const size_t at = (size_t)r * n + (size_t)b * fp8::kBlock;
    const int w = there ? min(fp8::kBlock, n - b * fp8::kBlock) : 0;
    float v[8];
    load8<VEC>(x + at, lane, w, v);
    const fp8::Scale sc = fp8::scale_of(amax16(v));
    store8<VEC>(q + at, lane, w, v, sc.inv);
    if (there && lane == 0) scale[s] = sc.scale;
  }
}

// The values again, rounded once to T.
template <bool VEC, typename T>
__global__ void __launch_bounds__(kThreads) unpack_rows_kernel(const uint8_t* __restrict__ q,
                                                               const float* __restrict__ scale,
                                                               long long segs, int n,
                                                               T* __restrict__ x) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 15;
  const int nb = fp8::blocks_of(n);
  for (long long s = (long long)blockIdx.x * kSegs + threadIdx.x / 16; s < segs;
       s += (long long)gridDim.x * kSegs) {
    const long long r = s / nb;
    const int b = (int)(s - r * nb);
    const size_t at = (size_t)r * n + (size_t)b * fp8::kBlock;
    const int w = min(fp8::kBlock, n - b * fp8::kBlock);
    const float sc = scale[s];
    if (VEC) {
      const int c = lane * 8;
      if (c >= w) continue;
      const uint2 k = *reinterpret_cast<const uint2*>(q + at + c);
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = fp8::values2(((j < 2 ? k.x : k.y) >> (16 * (j & 1))) & 0xffffu);
        v[2 * j] = f.x * sc;
        v[2 * j + 1] = f.y * sc;
      }
      if (sizeof(T) == 2) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
          o[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(x + at + c) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
        *reinterpret_cast<float4*>(x + at + c) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(x + at + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = lane + 16 * j;
        if (c < w) x[at + c] = (T)(fp8::values2(q[at + c]).x * sc);
      }
    }
  }
}

// One tile of 128 x 128 weights a thread block: 16 threads a row of the tile,
// 16 rows at once, the values held in registers until the tile's largest is known.
template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_fp8_kernel(const T* __restrict__ w, int rows,
                                                                int K, uint8_t* __restrict__ q,
                                                                float* __restrict__ scale) {
  pdl_wait();
  pdl_trigger();
  __shared__ uint32_t top[kThreads / 32];
  const int lane = threadIdx.x & 15, sub = threadIdx.x / 16;
  const int kb = fp8::blocks_of(K), rb = fp8::blocks_of(rows);
  const long long tile = blockIdx.x;
  const int c = (int)(tile % kb);
  const long long mr = tile / kb;  // matrix * rb + row block
  const long long m = mr / rb;
  const int r0 = (int)(mr - m * rb) * fp8::kBlock;
  const int n = min(fp8::kBlock, K - c * fp8::kBlock);
  float v[8][8];
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + sub + 16 * i;
    const size_t at = ((size_t)m * rows + r) * K + (size_t)c * fp8::kBlock;
    load8<false>(w + at, lane, r < rows ? n : 0, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) a = max(a, fp8::abs_bits(v[i][j]));
  }
  a = __reduce_max_sync(0xffffffffu, a);
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) a = max(a, top[i]);
  const fp8::Scale s = fp8::scale_of(a);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + sub + 16 * i;
    const size_t at = ((size_t)m * rows + r) * K + (size_t)c * fp8::kBlock;
    store8<false>(q + at, lane, r < rows ? n : 0, v[i], s.inv);
  }
  if (threadIdx.x == 0) scale[tile] = s.scale;
}

// The rows of every batch in 8 bits: q[r], scale[r] of x[tok[r]], scales
// fp8_scale_pitch(d) apart.  A thread block a row.  Rows from *total_rows on are
// skipped; a token index outside [0, T) is flagged and its row is zero.  Without tok:
// of x[r], T rows.
__global__ void __launch_bounds__(kThreads) gather_rows_fp8_kernel(
    const __nv_bfloat16* __restrict__ x, const int32_t* __restrict__ tok,
    const int32_t* __restrict__ total_rows, int P, int T, int d, uint8_t* __restrict__ q,
    float* __restrict__ scale, int* flags) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x;
  if (tok && (r >= P || r >= *total_rows)) return;
  const int t = tok ? tok[r] : r;
  const bool good = t >= 0 && t < T;
  if (!good && threadIdx.x == 0) flag_error(flags, kErrDeviceInput);
  const __nv_bfloat16* src = x + (size_t)(good ? t : 0) * d;
  const int lane = threadIdx.x & 15;
  const int nb = fp8::blocks_of(d);
  for (int b0 = 0; b0 < nb; b0 += kSegs) {
    const int b = b0 + threadIdx.x / 16;
    const int width = b < nb ? min(fp8::kBlock, d - b * fp8::kBlock) : 0;
    float v[8];
    load8<true>(src + (size_t)b * fp8::kBlock, lane, good ? width : 0, v);
    const fp8::Scale sc = fp8::scale_of(amax16(v));
    if (b < nb) {
      store8<true>(q + (size_t)r * d + (size_t)b * fp8::kBlock, lane, width, v, sc.inv);
      if (lane == 0) scale[(size_t)r * fp8_scale_pitch(d) + b] = sc.scale;
    }
  }
}

// The same from token rows that are in 8 bits already: q[r], scale[r] = q1, scale1 of
// tok[r], 16 bytes at once.  Two rows a thread block.  A token index outside [0, T) takes
// neither codes nor scales of any token: its row is that of a zero token here too.
__global__ void __launch_bounds__(kThreads) copy_rows_fp8_kernel(
    const uint4* __restrict__ q1, const float4* __restrict__ scale1,
    const int32_t* __restrict__ tok, const int32_t* __restrict__ total_rows, int P, int T,
    int vecs, int scale_vecs, uint4* __restrict__ q, float4* __restrict__ scale, int* flags) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & (kThreads / 2 - 1);
  const int r = blockIdx.x * 2 + threadIdx.x / (kThreads / 2);
  if (r >= P || r >= *total_rows) return;
  const int t = tok[r];
  const bool good = t >= 0 && t < T;
  if (!good && lane == 0) flag_error(flags, kErrDeviceInput);
  const uint4* src = q1 + (size_t)(good ? t : 0) * vecs;
  uint4* dst = q + (size_t)r * vecs;
#pragma unroll 4
  for (int i = lane; i < vecs; i += kThreads / 2) dst[i] = good ? src[i] : make_uint4(0, 0, 0, 0);
  const float zero = fp8::scale_of(0).scale;  // a zero token's
  for (int i = lane; i < scale_vecs; i += kThreads / 2)
    scale[(size_t)r * scale_vecs + i] = good ? scale1[(size_t)t * scale_vecs + i]
                                             : make_float4(zero, zero, zero, zero);
}

unsigned seg_grid(long long segs) {
  const long long most = (long long)num_sms() * 32, need = (segs + kSegs - 1) / kSegs;
  return (unsigned)(need < most ? need : most);
}

}  // namespace

cudaError_t launch_pack_rows(int dtype, const void* x, long long rows, int n, void* q,
                             float* scale, cudaStream_t s) {
  const long long segs = rows * fp8::blocks_of(n);
  if (segs == 0) return cudaSuccess;
  ProfScope pr("pack_rows", s);
  uint8_t* out = static_cast<uint8_t*>(q);
  if (dtype == MOE_BF16)
    (void)launch_kernel(n % 8 == 0 ? pack_rows_kernel<true, __nv_bfloat16>
                                   : pack_rows_kernel<false, __nv_bfloat16>,
                        seg_grid(segs), kThreads, 0, s, static_cast<const __nv_bfloat16*>(x), segs,
                        n, out, scale);
  else
    (void)launch_kernel(
        n % 8 == 0 ? pack_rows_kernel<true, float> : pack_rows_kernel<false, float>,
        seg_grid(segs), kThreads, 0, s, static_cast<const float*>(x), segs, n, out, scale);
  return cudaGetLastError();
}

cudaError_t launch_unpack_rows(int dtype, const void* q, const float* scale, long long rows, int n,
                               void* x, cudaStream_t s) {
  const long long segs = rows * fp8::blocks_of(n);
  if (segs == 0) return cudaSuccess;
  ProfScope pr("unpack_rows", s);
  const uint8_t* in = static_cast<const uint8_t*>(q);
  if (dtype == MOE_BF16)
    (void)launch_kernel(n % 8 == 0 ? unpack_rows_kernel<true, __nv_bfloat16>
                                   : unpack_rows_kernel<false, __nv_bfloat16>,
                        seg_grid(segs), kThreads, 0, s, in, scale, segs, n,
                        static_cast<__nv_bfloat16*>(x));
  else
    (void)launch_kernel(
        n % 8 == 0 ? unpack_rows_kernel<true, float> : unpack_rows_kernel<false, float>,
        seg_grid(segs), kThreads, 0, s, in, scale, segs, n, static_cast<float*>(x));
  return cudaGetLastError();
}

cudaError_t launch_quantize_fp8(int dtype, const void* w, int n_mats, int rows, int K, void* q,
                                float* scale, cudaStream_t s) {
  const long long tiles = (long long)n_mats * fp8::blocks_of(rows) * fp8::blocks_of(K);
  if (tiles == 0) return cudaSuccess;
  if (tiles > 0x7fffffffll) return cudaErrorInvalidValue;
  ProfScope pr("quantize_fp8", s);
  if (dtype == MOE_BF16)
    (void)launch_kernel(quantize_fp8_kernel<__nv_bfloat16>, (unsigned)tiles, kThreads, 0, s,
                        static_cast<const __nv_bfloat16*>(w), rows, K, static_cast<uint8_t*>(q),
                        scale);
  else
    (void)launch_kernel(quantize_fp8_kernel<float>, (unsigned)tiles, kThreads, 0, s,
                        static_cast<const float*>(w), rows, K, static_cast<uint8_t*>(q), scale);
  return cudaGetLastError();
}

cudaError_t launch_gather_rows_fp8(const void* x, const int32_t* tok_idx,
                                   const int32_t* total_rows, int P, int T, int d, void* q,
                                   float* scale, void* q1, float* scale1, int* flags,
                                   cudaStream_t s) {
  if (P == 0) return cudaSuccess;
  const __nv_bfloat16* in = static_cast<const __nv_bfloat16*>(x);
  // Every batch row from its token's bf16 row, or each token once and the codes copied:
  // two launches, worth it where the rows are many (8192 tokens x 8 slots x 4096: 143 us
  // against 89, 512 x 9 x 7168 20.6 against 17.3, 128 x 9 x 7168 10.4 against 11.5).
  if (P < 2 * T || (long long)P * d < kCopyElements) {
    ProfScope pr("gather_rows_fp8", s);
    (void)launch_kernel(gather_rows_fp8_kernel, P, kThreads, 0, s, in, tok_idx, total_rows, P, T,
                        d, static_cast<uint8_t*>(q), scale, flags);
    return cudaGetLastError();
  }
  ProfScope pr("gather_rows_fp8", s);
  (void)launch_kernel(gather_rows_fp8_kernel, T, kThreads, 0, s, in, (const int32_t*)nullptr,
                      total_rows, P, T, d, static_cast<uint8_t*>(q1), scale1, flags);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  (void)launch_kernel(copy_rows_fp8_kernel, (P + 1) / 2, kThreads, 0, s,
                      static_cast<const uint4*>(q1), reinterpret_cast<const float4*>(scale1),
                      tok_idx, total_rows, P, T, d / 16, fp8_scale_pitch(d) / 4,
                      static_cast<uint4*>(q), reinterpret_cast<float4*>(scale), flags);
  return cudaGetLastError();
}

}  // namespace moe
