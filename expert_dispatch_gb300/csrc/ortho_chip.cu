// ortho_chip.cu -- the Newton-Schulz orthogonalisation (ortho.cu) of matrices
// with at most 128 rows (columns, if tall), wholly on chip: one launch, one
// cluster of CTAs a matrix.
//
// The steps need X twice, as X X^T and as B X, and both products of a column of
// X need only that column: a CTA keeps a slice of X's columns in shared memory
// (fp16, 128 rows, blocks of 64 columns in the 128-byte swizzle) for all steps.
// The same bytes serve the tensor cores as K-major operand of X X^T and as
// MN-major operand of B X.  Only A = X X^T couples the slices: each CTA computes
// its slice's part (128 x 128, fp32) and stores it into the shared memory of the
// CTAs that add it up, each its share of A's columns, in rank order; these round
// their sums and store them into every CTA's copy of A.  (Stores into a partner's
// shared memory wait for nothing; loading the parts from the partners took 12000
// cycles a step with 8 CTAs.)  B is computed by every CTA for itself.
//
// What bounds it is latency: the chain of 3 products, 3 epilogues and 2 cluster
// barriers a step.  In launches of single products the same chain costs 17
// launches, about 64 us of host time and 2 to 5 us a launch on the GPU.
//
// Every wait is bounded; one that expires raises the CTA's abort flag and the
// workspace's error flag, and the warp goes on through the same barriers, so that
// no partner is left behind.  It waits for no product again and writes NaN in the
// place of everything that it takes from the accumulators from then on; the next
// products carry that through the matrix.
#include <cuda.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "ortho.cuh"
#include "tc_common.cuh"

namespace moe {
namespace {

using namespace ortho;

constexpr int kThreads = 512;       // 16 warps: four a TMEM lane quarter
constexpr int kWarps = kThreads / 32;
constexpr int kParts = kWarps / 4;  // warps a quarter
constexpr int kMaxCluster = 8;
constexpr int kBlockBytes = 128 * 128;  // 128 rows of 64 fp16 columns
constexpr int kPartBytes = 128 * 128 * 4;
constexpr int kMaxBlocksAlone = 8;  // 64-column blocks of X: 512 TMEM columns for B X
constexpr int kMaxBlocks = 6;       // beside a CTA's part of A: shared memory
// Enough shared memory, whatever the blocks need, that no other cluster's CTA of
// this library that uses tensor memory (the smallest takes 98 KB) shares the
// SM: a CTA takes all of the SM's tensor memory, and two clusters that each
// held it on one SM and waited for it on another would not end.
constexpr int kLeastSmem = 136 * 1024;
constexpr int kBlocksWanted = 4;    // blocks a CTA of a cluster, where eight CTAs are enough

struct ChipArgs {
  int rows, cols, m, n;
  int cluster, blocks;  // CTAs a matrix; 64-column blocks of X a CTA
  int steps;
  float eps;
  __nv_bfloat16* out;
  int* err;
};

__host__ __device__ constexpr int chip_smem(int cluster, int blocks) {
  const int need = 1024 + (blocks + 4) * kBlockBytes + (cluster > 1 ? kPartBytes : 0);
  return need > kLeastSmem ? need : kLeastSmem;
}

__device__ __forceinline__ void st_shared_cluster(uint32_t addr, uint32_t a, uint32_t b,
                                                  uint32_t c, uint32_t d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

// Byte offset of the 16-byte chunk that holds column c (a multiple of 8) of row
// r, in an operand of 64-column blocks.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return (uint32_t)((c >> 6) * kBlockBytes + r * 128 + ((((c & 63) >> 3) ^ (r & 7)) << 4));
}

// The 16 bytes from element `at` (a multiple of their number) of `total`; zeros
// behind the end.
template <typename T>
__device__ __forceinline__ uint4 load16(const T* __restrict__ g, int at, int total) {
  constexpr int V = 16 / (int)sizeof(T);
  if (at + V <= total) return *reinterpret_cast<const uint4*>(g + at);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (at + j >= total) continue;
    if constexpr (sizeof(T) == 4)
      w[j] = __float_as_uint(g[at + j]);
    else
      w[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(g)[at + j] << (16 * (j & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int V>
__device__ __forceinline__ void unpack16(uint4 q, float (&v)[V]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < V; ++j)
    v[j] = sizeof(T) == 4 ? __uint_as_float(w[j % 4])
           : j & 1        ? __uint_as_float(w[j / 2] & 0xffff0000u)
                          : __uint_as_float(w[j / 2] << 16);
}

// This CTA's columns c0 .. c0 + w - 1 of X = G or G^T, in the order in which its
// threads read them.  A line is a row of X, or a column (tall): what is
// consecutive in G.  It is read in aligned 16-byte vectors that may begin before
// it and end behind it; a vector's values are the line's positions start ..
// start + V - 1, of which 0 .. length - 1 count.  No vector reaches behind the
// stack's end.  A thread takes kSlots vectors at a time, all in flight at once; a
// slice of one such batch stays in registers, so G crosses into the SM once.
constexpr int kSlots = 16;

template <typename T>
struct Slice {
  static constexpr int V = 16 / (int)sizeof(T);
  const T* g;      // the vector in which the matrix begins; offsets below count from it
  int total;       // elements from g to the stack's end, or more than the matrix needs
  int first;       // the first line's offset
  int cols, lines, length, line0, vec0, line_step, vec_step, hshift, vec_batches, batches, used;

  __device__ __forceinline__ Slice(const T* stack, size_t stack_total, const ChipArgs& p, int mat,
                                   int c0, int w)
      : cols(p.cols) {
    const bool tall = p.rows > p.cols;
    const int wn = max(0, min(w, p.n - c0));  // columns that exist
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    lines = tall ? wn : (wn ? p.m : 0);
    length = tall ? p.m : wn;
    const size_t begin = (size_t)mat * p.rows * p.cols, aligned = begin / V * V;
    g = stack + aligned;
    total = (int)min(stack_total - aligned, (size_t)1 << 30);
    first = (int)(begin - aligned) + (tall ? c0 * cols : c0);
    // one vector more where lines begin inside one
    const int vectors = (length + V - 1) / V + (cols % V ? 1 : 0);
    // a warp takes one line by 32 vectors of a row; of a column 8 lines by 4
    // vectors, so that its stores into X share 16-byte chunks
    line0 = tall ? warp * 8 + (lane >> 2) : warp;
    vec0 = tall ? lane & 3 : lane;
    line_step = tall ? kWarps * 8 : kWarps;
    vec_step = tall ? 4 : 32;
    // slots: 2^hshift steps along a line by kSlots >> hshift lines
    const int along = (vectors + vec_step - 1) / vec_step;
    hshift = 0;
    while ((1 << hshift) < along && (1 << hshift) < kSlots) ++hshift;
    const int down = (lines + line_step - 1) / line_step, per = kSlots >> hshift;
    vec_batches = (along + (1 << hshift) - 1) >> hshift;
    batches = vec_batches * ((down + per - 1) / per);
    used = min(down, per) << hshift;  // slots that can hold something
  }
  // line and position of slot s of the batch from (line, vector) step (lb, vb) on;
  // false: none
  __device__ __forceinline__ bool place(int lb, int vb, int s, int& line, int& start,
                                        int& at) const {
    line = line0 + (lb + (s >> hshift)) * line_step;
    const int k = (vec0 + (vb + (s & ((1 << hshift) - 1))) * vec_step) * V;
    const int e = first + line * cols, shift = e & (V - 1);
    start = k - shift;
    at = e - shift + k;
    return line < lines && start < length;
  }
  template <typename F>
  __device__ __forceinline__ void slots(int b, F&& f) const {
    const int vb = b % vec_batches, lb = b / vec_batches;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      if (s >= used) break;  // the same for all threads
      int line, start, at;
      if (place(lb * (kSlots >> hshift), vb << hshift, s, line, start, at)) f(s, line, start, at);
    }
  }
  __device__ __forceinline__ void load(int b, uint4 (&raw)[kSlots]) const {
    slots(b, [&](int s, int, int, int at) { raw[s] = load16(g, at, total); });
  }
  // f(line, start, V values); values outside the line as they lie
  template <typename F>
  __device__ __forceinline__ void each(int b, const uint4 (&raw)[kSlots], F&& f) const {
    slots(b, [&](int s, int line, int start, int) {
      float v[V];
      unpack16<T, V>(raw[s], v);
      f(line, start, v);
    });
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    ortho_chip_kernel(const T* __restrict__ g, size_t total, const ChipArgs p) {
  constexpr int V = 16 / (int)sizeof(T);
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_s;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s;
  __shared__ float red[kWarps];
  __shared__ float sums[3], all_sums[kMaxCluster * 3];
  __shared__ Scale sc;
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* xs = smem;                              // X: blocks
  uint8_t* as = xs + p.blocks * kBlockBytes;       // A: 2 blocks
  uint8_t* bs = as + 2 * kBlockBytes;              // B: 2 blocks
  uint8_t* part = bs + 2 * kBlockBytes;  // parts of A: [CTA][8-column group][half][row][4] fp32
  const uint32_t xa = smem_u32(xs), aa = smem_u32(as), ba = smem_u32(bs);
  const uint32_t bar = smem_u32(&bar_s);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = p.cluster;
  const int mat = (int)blockIdx.x / C, rank = (int)blockIdx.x - mat * C;
  const int w = p.blocks * 64, c0 = rank * w;
  const bool tall = p.rows > p.cols;

  if (tid == 0) {
    mbar_init(bar, 1);
    abort_s = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  for (int i = tid; i < p.blocks * kBlockBytes / 16; i += kThreads)  // X: zeros
    reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && tid == 0) *p.err = 0;

  const Slice<T> slice(g, total, p, mat, c0, w);
  uint4 raw[kSlots];
  if (slice.batches == 1) slice.load(0, raw);
  // f over the slice: from the registers, or read again
  auto over_slice = [&](auto&& f) {
    if (slice.batches == 1) {
      slice.each(0, raw, f);
    } else {
      for (int b = 0; b < slice.batches; ++b) {
        slice.load(b, raw);
        slice.each(b, raw, f);
      }
    }
  };
  auto block_sum = [&](float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += red[i];
    return v;
  };

  // |G|, a CTA's slice in the place of a block's share (ortho_sumsq_kernel)
  {
    const int len = slice.length;
    float s[3] = {0.f, 0.f, 0.f};
    over_slice([&](int, int at, const float (&v)[V]) {
      if (at >= 0 && at + V <= len) {
#pragma unroll
        for (int j = 0; j < V; ++j) s[1] = fmaf(v[j], v[j], s[1]);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (at + j >= 0 && at + j < len) s[1] = fmaf(v[j], v[j], s[1]);
      }
    });
    s[1] = block_sum(s[1]);
    if (!plain_sum(s[1])) {
      s[1] = 0.f;
      over_slice([&](int, int at, const float (&v)[V]) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (at + j >= 0 && at + j < len) add_square(v[j], s);
      });
#pragma unroll
      for (int q = 0; q < 3; ++q) s[q] = block_sum(s[q]);
    }
    if (tid == 0) {
#pragma unroll
      for (int q = 0; q < 3; ++q) sums[q] = s[q];
    }
    __syncthreads();
    if (C > 1) cluster_sync();
    if (tid < 3 * C)
      all_sums[tid] = C > 1 ? ld_shared_cluster(mapa_shared(smem_u32(&sums[tid % 3]), tid / 3))
                            : sums[tid];
    __syncthreads();
    if (warp == 0) {
      const Scale own = matrix_scale(all_sums, C, p.eps);
      if (lane == 0) sc = own;
    }
    __syncthreads();
  }
  const Scale scale = sc;
  const float f1 = scale.f1, f2 = scale.f2;
  over_slice([&](int line, int at, const float (&v)[V]) {
    const int len = slice.length;
    if (!tall && V == 8 && (at & 7) == 0 && at + V <= len) {
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        u[j] = pack_half2(v[(2 * j) % V] * f1 * f2, v[(2 * j + 1) % V] * f1 * f2);
      *reinterpret_cast<uint4*>(xs + chunk_at(line, at)) = make_uint4(u[0], u[1], u[2], u[3]);
      return;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (at + j < 0 || at + j >= len) continue;
      const int r = tall ? at + j : line, c = tall ? line : at + j;
      *reinterpret_cast<__half*>(xs + chunk_at(r, c & ~7) + (c & 7) * 2) =
          __float2half_rn(v[j] * f1 * f2);
    }
  });

  uint32_t parity = 0;
  bool ok = true;  // this warp has not given up waiting
  volatile int* abort_flag = &abort_s;
  // Every thread's stores to the operands are in place and every read of the
  // accumulators is done: thread 0 issues the products, all run `meanwhile` and wait
  // for them.
  auto product = [&](auto&& issue, auto&& meanwhile) {
    fence_proxy_async_shared();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      issue();
      umma_commit(bar);
    }
    meanwhile();
    ok = ok && tc::mbar_wait_warp(bar, parity, abort_flag, p.err);
    parity ^= 1u;
    tc_fence_after();
  };
  const int q = warp & 3, sub = warp >> 2, row = q * 32 + lane;
  const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);

  for (int step = 0; step < p.steps; ++step) {
    const float rho = step == 0 ? scale.rho : 1.f;
    const bool last = step + 1 == p.steps;
    float alpha, beta;
    // ---- A = X X^T, this slice's part: TMEM columns 0 .. 127
    product([&] {
      constexpr uint32_t idesc = idesc_f16_f32(128, 128);
      for (int b = 0; b < p.blocks; ++b)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t d = smem_desc_sw128(xa + b * kBlockBytes + kk * 32);
          umma_bf16(tmem, d, d, idesc, b | kk ? 1u : 0u);
        }
    }, [&] {
      alpha = gram_factor(scale, rho * rho * (kScaleA / (kScaleX * kScaleX)), step);
      beta = last ? last_factor(scale, rho / (kScaleB * kScaleX), step)
                  : apply_factor(scale, rho / kScaleB, step, 1);
    });
    const float alpha1 = ok ? alpha : quiet_nan();
#pragma unroll 1
    for (int c = sub * 32; c < 128; c += 32 * kParts) {
      uint32_t a[2][16];
      tmem_ld16(lanes + c, a[0]);
      tmem_ld16(lanes + c + 16, a[1]);
      tmem_ld_wait();
      if (C == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 8 columns
          uint32_t u[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = 8 * i + 2 * j;
            u[j] = pack_half2(alpha1 * __uint_as_float(a[k >> 4][k & 15]),
                              alpha1 * __uint_as_float(a[k >> 4][(k & 15) + 1]));
          }
          *reinterpret_cast<uint4*>(as + chunk_at(row, c + 8 * i)) =
              make_uint4(u[0], u[1], u[2], u[3]);
        }
      } else {
        // one NaN in each of the warp's rows of A: products with A spread it over the matrix
        if (!ok) a[0][0] = __float_as_uint(quiet_nan());
        // 8-column group k of A is added up by CTA k % C: there, behind the
        // groups of the CTAs before this one, [row][4] fp32 of its two halves
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = c / 8 + i, owner = k & (C - 1), slot = k / C;
          const uint32_t to = mapa_shared(
              smem_u32(part) + (uint32_t)(((rank * (16 / C) + slot) * 256 + row) * 16), owner);
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 512 consecutive bytes a warp
            const uint32_t* u = &a[i >> 1][(i & 1) * 8 + 4 * h];
            st_shared_cluster(to + 2048u * h, u[0], u[1], u[2], u[3]);
          }
        }
      }
      __syncwarp();
    }
    if (C > 1) {
      __syncthreads();
      cluster_sync();  // every CTA's parts are in place; its copy of A is no longer read
      const int groups = 16 / C;
      for (int i = tid; i < groups * 128; i += kThreads) {
        const int slot = i >> 7, r = i & 127;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int src = 0; src < C; ++src) {
          const float4* f =
              reinterpret_cast<const float4*>(part) + (src * groups + slot) * 256 + r;
          const float4 lo = f[0], hi = f[128];
          v[0] += lo.x, v[1] += lo.y, v[2] += lo.z, v[3] += lo.w;
          v[4] += hi.x, v[5] += hi.y, v[6] += hi.z, v[7] += hi.w;
        }
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = pack_half2(alpha * v[2 * j], alpha * v[2 * j + 1]);
        // by way of B's place, group after group: a warp's stores are consecutive there
        const uint32_t to = ba + (uint32_t)(((slot * C + rank) * 128 + r) * 16);
        for (int k = 0; k < C; ++k)
          st_shared_cluster(mapa_shared(to, (rank + k) & (C - 1)), u[0], u[1], u[2], u[3]);
      }
      __syncthreads();
      cluster_sync();  // A's groups are in place
      for (int i = tid; i < 16 * 128; i += kThreads)
        *reinterpret_cast<uint4*>(as + chunk_at(i & 127, (i >> 7) * 8)) =
            reinterpret_cast<const uint4*>(bs)[i];
    }

    // ---- B = a I + b A + c A A: TMEM columns 128 .. 255
    product([&] {
      constexpr uint32_t idesc = idesc_f16_f32(128, 128);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint64_t d = smem_desc_sw128(aa + (k >> 2) * kBlockBytes + (k & 3) * 32);
        umma_bf16(tmem + 128, d, d, idesc, k ? 1u : 0u);
      }
    }, [] {});
    const float gamma1 = ok ? kC * (kScaleB / (kScaleA * kScaleA)) : quiet_nan();
#pragma unroll 1
    for (int c = sub * 32; c < 128; c += 32 * kParts) {
      uint32_t a[2][16];
      tmem_ld16(lanes + 128 + c, a[0]);
      tmem_ld16(lanes + 128 + c + 16, a[1]);
      uint4 gm[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        gm[i] = *reinterpret_cast<const uint4*>(as + chunk_at(row, c + 8 * i));
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // 8 columns
        const uint32_t gw[4] = {gm[i].x, gm[i].y, gm[i].z, gm[i].w};
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 ga = __half22float2(*reinterpret_cast<const __half2*>(&gw[j]));
          const int k = 8 * i + 2 * j;
          float v[2];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            v[t] = fmaf(kB * (kScaleB / kScaleA), t ? ga.y : ga.x,
                        gamma1 * __uint_as_float(a[k >> 4][(k & 15) + t]));
            if (row == c + k + t && row < p.m) v[t] += kA * kScaleB;
          }
          u[j] = pack_half2(v[0], v[1]);
        }
        *reinterpret_cast<uint4*>(bs + chunk_at(row, c + 8 * i)) =
            make_uint4(u[0], u[1], u[2], u[3]);
      }
      __syncwarp();
    }

    // ---- X = B X, the slice's columns: TMEM columns 0 .. w - 1
    product([&] {
      for (int b = 0; b < p.blocks; b += 4) {
        const int nb = min(4, p.blocks - b);
        const uint32_t idesc = idesc_f16_f32(128, 64 * nb) | kTransposeB;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_bf16(tmem + b * 64, smem_desc_sw128(ba + (k >> 2) * kBlockBytes + (k & 3) * 32),
                    smem_desc_mn128(xa + b * kBlockBytes + k * 2048, kBlockBytes), idesc,
                    k ? 1u : 0u);
      }
    }, [] {});
    const float beta1 = ok ? beta : quiet_nan();
#pragma unroll 1
    for (int c = sub * 32; c < w; c += 32 * kParts) {  // w is a multiple of 64
      uint32_t a[2][16];
      tmem_ld16(lanes + c, a[0]);
      tmem_ld16(lanes + c + 16, a[1]);
      tmem_ld_wait();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = beta1 * __uint_as_float(a[h][j]);
        const int cc = c + 16 * h;
        if (!last) {
          uint32_t u[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) u[j] = pack_half2(v[2 * j], v[2 * j + 1]);
          *reinterpret_cast<uint4*>(xs + chunk_at(row, cc)) = make_uint4(u[0], u[1], u[2], u[3]);
          *reinterpret_cast<uint4*>(xs + chunk_at(row, cc + 8)) =
              make_uint4(u[4], u[5], u[6], u[7]);
        } else if (tall) {  // a warp's lanes hold consecutive elements of the result
          if (row < p.m) {
            __nv_bfloat16* to = p.out + (size_t)mat * p.m * p.n + row;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c0 + cc + j < p.n)
                to[(size_t)(c0 + cc + j) * p.m] = __float2bfloat16_rn(v[j]);
          }
        } else {  // in X's place, to be stored along its rows
          uint32_t u[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            u[j] = *reinterpret_cast<const uint32_t*>(&b);
          }
          *reinterpret_cast<uint4*>(xs + chunk_at(row, cc)) = make_uint4(u[0], u[1], u[2], u[3]);
          *reinterpret_cast<uint4*>(xs + chunk_at(row, cc + 8)) =
              make_uint4(u[4], u[5], u[6], u[7]);
        }
      }
      __syncwarp();
    }
  }
  if (!tall) {
    __syncthreads();
    const int wn = min(w, p.n - c0);
    for (int r = warp; r < p.m; r += kWarps) {
      __nv_bfloat16* to = p.out + ((size_t)mat * p.m + r) * p.n + c0;
      if (p.n % 8 == 0) {  // 16-byte aligned rows
        for (int c = lane * 8; c < wn; c += 256)
          *reinterpret_cast<uint4*>(to + c) =
              *reinterpret_cast<const uint4*>(xs + chunk_at(r, c));
      } else {
        for (int c = lane; c < wn; c += 32)
          to[c] = *reinterpret_cast<const __nv_bfloat16*>(xs + chunk_at(r, c & ~7) + (c & 7) * 2);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // the last accesses to a peer's shared memory lie before its last barrier
}

template <typename T>
cudaError_t launch(const T* g, const ChipArgs& p, int n_mats, cudaStream_t s) {
  auto kern = ortho_chip_kernel<T>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  static std::atomic<bool> configured[64] = {};
  if (!configured[dev]) {
    constexpr int a = chip_smem(1, kMaxBlocksAlone), b = chip_smem(2, kMaxBlocks);
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, a > b ? a : b);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(n_mats * p.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)chip_smem(p.cluster, p.blocks);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  ProfScope pr("ortho_chip", s);
  count_launch();
  (void)cudaLaunchKernelEx(&cfg, kern, g, (size_t)n_mats * p.rows * p.cols, p);
  return cudaGetLastError();
}

}  // namespace

bool ortho_fits_chip(const moe_ortho_desc& D) {
  const int m = D.rows < D.cols ? D.rows : D.cols, n = D.rows < D.cols ? D.cols : D.rows;
  return m <= 128 && n <= kMaxCluster * kMaxBlocks * 64;
}

cudaError_t launch_ortho_chip(const moe_ortho_desc& D, const void* g, void* out, int* flags,
                              cudaStream_t s) {
  ChipArgs p{};
  p.rows = D.rows, p.cols = D.cols;
  p.m = D.rows < D.cols ? D.rows : D.cols;
  p.n = D.rows < D.cols ? D.cols : D.rows;
  p.steps = D.steps;
  p.eps = D.eps;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.err = flags;
  // a CTA alone while X fits it (no exchange), else the least power of two of
  // CTAs that hold it
  const int blocks = (p.n + 63) / 64;
  p.cluster = 1;
  if (blocks > kMaxBlocksAlone)
    for (p.cluster = 2; (blocks + p.cluster - 1) / p.cluster > kBlocksWanted &&
                        p.cluster < kMaxCluster;)
      p.cluster *= 2;
  p.blocks = (blocks + p.cluster - 1) / p.cluster;
  return D.dtype == MOE_BF16 ? launch(static_cast<const __nv_bfloat16*>(g), p, D.n_mats, s)
                             : launch(static_cast<const float*>(g), p, D.n_mats, s);
}

}  // namespace moe
