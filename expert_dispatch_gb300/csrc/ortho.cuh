// ortho.cuh -- pieces shared by the kernels of the Newton-Schulz
// orthogonalisation (ortho.cu, ortho_chip.cu): the polynomial, the fp16 scales
// (see ortho.cu), the norm's sums and operand helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {
namespace ortho {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScaleX = 1024.f, kScaleA = 16384.f, kScaleB = 4096.f;
// Two steps at once: of B0 A (up to 1.1) and B1 B0 (up to 3.45^2).
constexpr float kScaleM = 8192.f, kScaleQ = 1024.f;

struct Scale {
  float f1, f2;  // X = g * f1 * f2, powers of two (one factor could leave fp32's range)
  float rho;     // what is left of 1 / (|G| + eps), in (1/2, 1]
  int shift;     // X is held 2^shift larger than its 2^10 says: where eps outweighs |G|
};

// X is small as long as eps outweighs |G|, and a step makes it 3.4445 times larger
// at most.  So after `steps` steps it is held 2^(shift - 2 steps) larger than
// otherwise, and its values stay in fp16's range: without it a matrix of 1e-8 eps
// came out 38 % off, one of 1e-9 eps as zeros.
__device__ __forceinline__ int shift_after(const Scale& s, int steps) {
  return max(s.shift - 2 * steps, 0);
}
// The factor of X X^T, and of B X, `ahead` steps further on; f includes rho where
// X is the first one.
__device__ __forceinline__ float gram_factor(const Scale& s, float f, int steps) {
  return s.shift ? scalbnf(f, -2 * shift_after(s, steps)) : f;
}
__device__ __forceinline__ float apply_factor(const Scale& s, float f, int steps, int ahead) {
  return s.shift ? scalbnf(f, shift_after(s, steps + ahead) - shift_after(s, steps)) : f;
}
// The same where the result is no longer held larger.
__device__ __forceinline__ float last_factor(const Scale& s, float f, int steps) {
  return s.shift ? scalbnf(f, -shift_after(s, steps)) : f;
}

// V consecutive elements as fp32: 16 aligned bytes.
template <typename T, int V>
__device__ __forceinline__ void load_elems(const T* p, float (&v)[V]) {
  if constexpr (sizeof(T) == 4) {
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

// Sums of squares.  A plain sum of squares in fp32 is good while it lies between
// 2^-80 and 2^100: no square was near overflow, and what underflowed lies 46
// powers of two below the sum (NaN, infinity and 0 are outside, too).  Otherwise
// three sums are kept in which no square over- or underflows: of values above
// 2^45 times 2^-84, of values below 2^-45 times 2^84, and of the rest.
constexpr float kBig = 0x1p45f, kSmall = 0x1p-45f, kUp = 0x1p84f, kDown = 0x1p-84f;

__device__ __forceinline__ bool plain_sum(float s) { return s >= 0x1p-80f && s <= 0x1p100f; }

__device__ __forceinline__ void add_square(float x, float (&s)[3]) {
  const float ax = fabsf(x);
  if (ax > kBig)
    s[0] = fmaf(x * kDown, x * kDown, s[0]);
  else if (ax < kSmall)
    s[2] = fmaf(x * kUp, x * kUp, s[2]);
  else
    s[1] = fmaf(x, x, s[1]);
}

// The scale of one matrix from its partial sums, added by one warp in a fixed
// order.
__device__ __forceinline__ Scale matrix_scale(const float* partial, int n, float eps) {
  float s[3] = {0.f, 0.f, 0.f};
  for (int i = threadIdx.x & 31; i < n; i += 32)
#pragma unroll
    for (int q = 0; q < 3; ++q) s[q] += partial[i * 3 + q];
#pragma unroll
  for (int q = 0; q < 3; ++q)
#pragma unroll
    for (int o = 16; o; o >>= 1) s[q] += __shfl_xor_sync(0xffffffffu, s[q], o);
  // |G| = norm * 2^off, |G| + eps = v * 2^off_v
  float norm, v;
  int off = 0, off_v = 0;
  if (s[0] > 0.f || s[0] != s[0]) {
    norm = sqrtf(s[0] + s[1] * kDown * kDown), off = 84;
    v = norm + eps * kDown, off_v = 84;
  } else if (s[1] > 0.f || s[1] != s[1]) {
    norm = sqrtf(s[1] + s[2] * kDown * kDown);
    v = norm + eps;
  } else {
    norm = sqrtf(s[2]), off = -84;
    if (eps > 0.f)
      v = norm * kDown + eps;
    else
      v = norm, off_v = -84;
  }
  Scale r{0.f, 0.f, 0.f, 0};
  if (v == 0.f) return r;  // a zero matrix, eps = 0: X = 0
  if (isinf(v) || v != v) {
    r.f1 = r.f2 = r.rho = __int_as_float(0x7fffffff);
    return r;
  }
  const int e = ilogbf(v);
  // |G| 2^shift stays below 2^(e + off_v), as large as |G| + eps at most
  if (norm > 0.f) r.shift = max(e + off_v - (ilogbf(norm) + off) - 1, 0);
  const int k = 10 - e - off_v + r.shift;  // X = g * 2^k
  r.f1 = scalbnf(1.f, k / 2);
  r.f2 = scalbnf(1.f, k - k / 2);
  r.rho = 1.f / scalbnf(v, -e);
  return r;
}

// Shared-memory descriptor of an MN-major operand written by TMA in boxes of 64
// columns (128 bytes, 128-byte swizzle): groups of 8 reduction rows are 1024
// bytes apart, the next 64 columns `next` bytes.
__device__ __forceinline__ uint64_t smem_desc_mn128(uint32_t saddr, uint32_t next) {
  uint64_t desc = 0;
  desc |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);  // start address
  desc |= static_cast<uint64_t>(next >> 4) << 16;          // leading byte offset: 64 columns
  desc |= static_cast<uint64_t>(1024 >> 4) << 32;          // stride byte offset: 8 rows
  desc |= static_cast<uint64_t>(1) << 46;                  // descriptor version
  desc |= static_cast<uint64_t>(2) << 61;                  // 128-byte swizzle
  return desc;
}
constexpr uint32_t kTransposeB = 1u << 16;  // instruction descriptor: B is MN-major

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float ld_shared_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

constexpr int kRowWords = 9;  // a lane's 16 bf16 values in shared memory, and a pad

// A warp stores 16 columns of 32 rows of one matrix's result: lane l has row
// row0 + l, columns c0 .. c0 + 15, in v.  base is [m, n], or [n, m] if tall.
// Rows of a multiple of 16 bytes take two 16-byte stores a lane, columns (tall)
// lie across the lanes; other rows go through `scratch` (32 kRowWords words of
// the warp's own), so that 16 lanes store 32 consecutive bytes of a row where
// each lane's own values would touch 32 rows at once.
__device__ __forceinline__ void store_result(__nv_bfloat16* base, int m, int n, bool tall,
                                             int row0, int c0, const float (&v)[16],
                                             uint32_t* scratch) {
  const int lane = threadIdx.x & 31, row = row0 + lane;
  if (tall) {
    if (row < m) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (c0 + j < n) base[(size_t)(c0 + j) * m + row] = __float2bfloat16_rn(v[j]);
    }
    return;
  }
  uint32_t w[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * t], v[2 * t + 1]);
    w[t] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (n % 8 == 0) {
    if (row < m) {
      uint4* dst = reinterpret_cast<uint4*>(base + (size_t)row * n + c0);
      if (c0 < n) dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      if (c0 + 8 < n) dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
    return;
  }
#pragma unroll
  for (int t = 0; t < 8; ++t) scratch[lane * kRowWords + t] = w[t];
  __syncwarp();
  const int c = lane & 15;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = 2 * i + (lane >> 4);
    const uint32_t word = scratch[r * kRowWords + (c >> 1)];
    if (row0 + r < m && c0 + c < n)
      reinterpret_cast<uint16_t*>(base)[(size_t)(row0 + r) * n + c0 + c] =
          (uint16_t)(c & 1 ? word >> 16 : word & 0xffffu);
  }
  __syncwarp();
}

}  // namespace ortho
}  // namespace moe
