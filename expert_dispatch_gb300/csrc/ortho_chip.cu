// ortho_chip.cu -- the Newton-Schulz orthogonalisation (ortho.cu) of matrices
// with at most 128 rows (columns, if tall), wholly on chip: one launch, one
// cluster of CTAs a matrix.
//
// The steps need X twice, as X X^T and as B X, and both products of a column of
// X need only that column: a CTA keeps a slice of X's columns in shared memory
// (fp16, 128 rows, blocks of 64 columns in the 128-byte swizzle) for all steps.
// The same bytes serve the tensor cores as K-major operand of X X^T and as
// MN-major operand of B X.  Only A = X X^T couples the slices: each CTA computes
// its slice's part (128 x 128, fp32), leaves it in shared memory, and after a
// cluster barrier adds up its share of A's columns over the cluster in rank
// order, rounds it and stores it into every CTA's copy of A.  B is computed by
// every CTA for itself.  HBM sees G (twice) and the result.
//
// What bounds it is latency: the chain of 3 products, 3 epilogues and 2 cluster
// barriers a step.  In launches of single products the same chain costs 17
// launches, about 64 us of host time and 2 to 5 us a launch on the GPU.
//
// Every wait is bounded; one that expires raises the CTA's abort flag and the
// workspace's error flag, and the CTA goes on through the same barriers (its
// later waits end early), so that no partner is left behind.
#include <cuda.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "ortho.cuh"
#include "tc_common.cuh"

namespace moe {
namespace {

using namespace ortho;

constexpr int kThreads = 256;       // 8 warps: two a TMEM lane quarter
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

// Byte offset of the 16-byte chunk that holds column c (a multiple of 8) of row
// r, in an operand of 64-column blocks.
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return (uint32_t)((c >> 6) * kBlockBytes + r * 128 + ((((c & 63) >> 3) ^ (r & 7)) << 4));
}

// f(row, column of the slice, V values) over this CTA's columns c0 .. c0 + w - 1
// of X = G or G^T, V elements that are consecutive in G at a time (V == 1: any
// alignment); the values follow each other along X's row, or its column (tall).
template <typename T, int V, typename F>
__device__ __forceinline__ void for_slice(const T* __restrict__ g, const ChipArgs& p, int c0,
                                          int w, F&& f) {
  const bool tall = p.rows > p.cols;
  const int wn = min(w, p.n - c0);  // columns that exist
  if (wn <= 0) return;
  if (!tall) {
    const int per_row = (wn + V - 1) / V, total = p.m * per_row;
#pragma unroll 4
    for (int i = threadIdx.x; i < total; i += kThreads) {
      const int r = i / per_row, c = (i - r * per_row) * V;
      float v[V];
      load_elems<T, V>(g + (size_t)r * p.cols + c0 + c, v);
      f(r, c, v);
    }
  } else {
    // a warp takes 8 columns by 4 vectors of rows: 64-byte reads, and stores
    // into X that share a chunk
    const int nr = (p.m + V - 1) / V, nr4 = (nr + 3) / 4, total = ((wn + 7) / 8) * nr4 * 32;
#pragma unroll 4
    for (int i = threadIdx.x; i < total; i += kThreads) {
      const int t = i >> 5;
      const int r = ((t % nr4) * 4 + (i & 3)) * V, c = (t / nr4) * 8 + ((i >> 2) & 7);
      if (r < p.m && c < wn) {
        float v[V];
        load_elems<T, V>(g + (size_t)(c0 + c) * p.cols + r, v);
        f(r, c, v);
      }
    }
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 1)
    ortho_chip_kernel(const T* __restrict__ g_all, const ChipArgs p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bar_s;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s;
  __shared__ float red[3][kThreads / 32], top[kThreads / 32];
  __shared__ float sums[3], all_sums[kMaxCluster * 3];
  __shared__ Scale sc;
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* xs = smem;                              // X: blocks
  uint8_t* as = xs + p.blocks * kBlockBytes;       // A: 2 blocks
  uint8_t* bs = as + 2 * kBlockBytes;              // B: 2 blocks
  float* part = reinterpret_cast<float*>(bs + 2 * kBlockBytes);  // [128 columns][128 rows]
  const uint32_t xa = smem_u32(xs), aa = smem_u32(as), ba = smem_u32(bs);
  const uint32_t bar = smem_u32(&bar_s);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = p.cluster;
  const int mat = (int)blockIdx.x / C, rank = (int)blockIdx.x - mat * C;
  const int w = p.blocks * 64, c0 = rank * w;
  const bool tall = p.rows > p.cols;
  const T* g = g_all + (size_t)mat * p.rows * p.cols;

  if (tid == 0) {
    mbar_init(bar, 1);
    abort_s = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  for (int i = tid; i < (p.blocks + 4) * kBlockBytes / 16; i += kThreads)  // X, A and B: zeros
    reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && tid == 0) *p.err = 0;

  // |G|: sums of squares as in ortho_sumsq_kernel, a CTA's slice in the place of
  // a block's share
  {
    float s[3] = {0.f, 0.f, 0.f}, most = 0.f;
    for_slice<T, V>(g, p, c0, w, [&](int, int, const float (&v)[V]) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s[1] = fmaf(v[j], v[j], s[1]);
        most = fmaxf(most, fabsf(v[j]));
      }
    });
#pragma unroll
    for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (lane == 0) top[warp] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) most = fmaxf(most, top[i]);
    if (most != 0.f && (most > kBig || most < kSmall)) {
      s[1] = 0.f;
      for_slice<T, V>(g, p, c0, w, [&](int, int, const float (&v)[V]) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float ax = fabsf(v[j]);
          if (ax > kBig)
            s[0] = fmaf(v[j] * kDown, v[j] * kDown, s[0]);
          else if (ax < kSmall)
            s[2] = fmaf(v[j] * kUp, v[j] * kUp, s[2]);
          else
            s[1] = fmaf(v[j], v[j], s[1]);
        }
      });
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) {
#pragma unroll
      for (int o = 16; o; o >>= 1) s[q] += __shfl_xor_sync(0xffffffffu, s[q], o);
      if (lane == 0) red[q][warp] = s[q];
    }
    __syncthreads();
    if (tid < 3) {
      float v = 0.f;
      for (int i = 0; i < kThreads / 32; ++i) v += red[tid][i];
      sums[tid] = v;
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
  const float f1 = sc.f1, f2 = sc.f2, rho1 = sc.rho;
  for_slice<T, V>(g, p, c0, w, [&](int r, int c, const float (&v)[V]) {
    if (!tall && V == 8) {
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        u[j] = pack_half2(v[(2 * j) % V] * f1 * f2, v[(2 * j + 1) % V] * f1 * f2);
      *reinterpret_cast<uint4*>(xs + chunk_at(r, c)) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int rr = tall ? r + j : r, cc = tall ? c : c + j;
        *reinterpret_cast<__half*>(xs + chunk_at(rr, cc & ~7) + (cc & 7) * 2) =
            __float2half_rn(v[j] * f1 * f2);
      }
    }
  });

  uint32_t parity = 0;
  volatile int* abort_flag = &abort_s;
  // Every thread's stores to the operands are in place and every read of the
  // accumulators is done: thread 0 issues the products, all wait for them.
  auto product = [&](auto&& issue) {
    fence_proxy_async_shared();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      issue();
      umma_commit(bar);
    }
    (void)tc::mbar_wait_warp(bar, parity, abort_flag, p.err);
    parity ^= 1u;
    tc_fence_after();
  };
  const int q = warp & 3, half = warp >> 2, row = q * 32 + lane;
  const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);

  for (int step = 0; step < p.steps; ++step) {
    const float rho = step == 0 ? rho1 : 1.f;
    // ---- A = X X^T, this slice's part: TMEM columns 0 .. 127
    product([&] {
      constexpr uint32_t idesc = idesc_f16_f32(128, 128);
      for (int b = 0; b < p.blocks; ++b)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t d = smem_desc_sw128(xa + b * kBlockBytes + kk * 32);
          umma_bf16(tmem, d, d, idesc, b | kk ? 1u : 0u);
        }
    });
    const float alpha = rho * rho * (kScaleA / (kScaleX * kScaleX));
#pragma unroll 1
    for (int c = half * 64; c < half * 64 + 64; c += 16) {
      uint32_t a[16];
      tmem_ld16(lanes + c, a);
      tmem_ld_wait();
      if (C == 1) {
        uint32_t u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          u[j] = pack_half2(alpha * __uint_as_float(a[2 * j]),
                            alpha * __uint_as_float(a[2 * j + 1]));
        *reinterpret_cast<uint4*>(as + chunk_at(row, c)) = make_uint4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<uint4*>(as + chunk_at(row, c + 8)) = make_uint4(u[4], u[5], u[6], u[7]);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c + j) * 128 + row] = __uint_as_float(a[j]);
      }
      __syncwarp();
    }
    if (C > 1) {
      __syncthreads();
      cluster_sync();  // every CTA's part is in place; its copy of A is no longer read
      // 8 columns at a time, dealt out to the cluster and to the warps' halves
      for (int k = rank + half * C; k < 16; k += 2 * C) {
        const uint32_t at = smem_u32(part) + (uint32_t)(k * 8 * 128 + row) * 4u;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) {
          if (r < C) {
            const uint32_t peer = mapa_shared(at, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += ld_shared_cluster(peer + (uint32_t)j * 512u);
          }
        }
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = pack_half2(alpha * v[2 * j], alpha * v[2 * j + 1]);
        const uint32_t to = aa + chunk_at(row, k * 8);
        for (int r = 0; r < C; ++r)
          asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           mapa_shared(to, r)),
                       "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3])
                       : "memory");
      }
      // the stores reach the peers' tensor cores: ordered before this barrier
      // here and after it there (product's fence)
      asm volatile("fence.proxy.async;" ::: "memory");
      __syncthreads();
      cluster_sync();
    }

    // ---- B = a I + b A + c A A: TMEM columns 128 .. 255
    product([&] {
      constexpr uint32_t idesc = idesc_f16_f32(128, 128);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint64_t d = smem_desc_sw128(aa + (k >> 2) * kBlockBytes + (k & 3) * 32);
        umma_bf16(tmem + 128, d, d, idesc, k ? 1u : 0u);
      }
    });
#pragma unroll 1
    for (int c = half * 64; c < half * 64 + 64; c += 16) {
      uint32_t a[16];
      tmem_ld16(lanes + 128 + c, a);
      uint4 gm[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        gm[i] = *reinterpret_cast<const uint4*>(as + chunk_at(row, c + 8 * i));
      tmem_ld_wait();
      const uint32_t gw[8] = {gm[0].x, gm[0].y, gm[0].z, gm[0].w,
                              gm[1].x, gm[1].y, gm[1].z, gm[1].w};
      uint32_t u[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 ga = __half22float2(*reinterpret_cast<const __half2*>(&gw[j]));
        float v[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          v[t] = fmaf(kB * (kScaleB / kScaleA), t ? ga.y : ga.x,
                      kC * (kScaleB / (kScaleA * kScaleA)) * __uint_as_float(a[2 * j + t]));
          if (row == c + 2 * j + t && row < p.m) v[t] += kA * kScaleB;
        }
        u[j] = pack_half2(v[0], v[1]);
      }
      *reinterpret_cast<uint4*>(bs + chunk_at(row, c)) = make_uint4(u[0], u[1], u[2], u[3]);
      *reinterpret_cast<uint4*>(bs + chunk_at(row, c + 8)) = make_uint4(u[4], u[5], u[6], u[7]);
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
    });
    const bool last = step + 1 == p.steps;
    const float beta = last ? rho / (kScaleB * kScaleX) : rho / kScaleB;
#pragma unroll 1
    for (int c = half * 16; c < w; c += 32) {
      uint32_t a[16];
      tmem_ld16(lanes + c, a);
      tmem_ld_wait();
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = beta * __uint_as_float(a[j]);
      if (!last) {
        uint32_t u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = pack_half2(v[2 * j], v[2 * j + 1]);
        *reinterpret_cast<uint4*>(xs + chunk_at(row, c)) = make_uint4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<uint4*>(xs + chunk_at(row, c + 8)) =
            make_uint4(u[4], u[5], u[6], u[7]);
      } else if (row < p.m) {
        store_result<16>(p.out + (size_t)mat * p.m * p.n, p.m, p.n, tall, row, c0 + c, v);
      }
      __syncwarp();
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

template <typename T, int V>
cudaError_t launch(const T* g, const ChipArgs& p, int n_mats, cudaStream_t s) {
  auto kern = ortho_chip_kernel<T, V>;
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
  (void)cudaLaunchKernelEx(&cfg, kern, g, p);
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
  // four blocks a CTA; up to eight in a CTA alone where the stack fills the GPU
  const int blocks = (p.n + 63) / 64;
  p.cluster = (blocks + 3) / 4;
  if (p.cluster > kMaxCluster) p.cluster = kMaxCluster;
  if (blocks <= kMaxBlocksAlone && D.n_mats * p.cluster > num_sms()) p.cluster = 1;
  p.blocks = (blocks + p.cluster - 1) / p.cluster;
  p.cluster = (blocks + p.blocks - 1) / p.blocks;  // no CTA without columns
  if (D.dtype == MOE_BF16) {
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(g);
    return D.cols % 8 == 0 ? launch<__nv_bfloat16, 8>(x, p, D.n_mats, s)
                           : launch<__nv_bfloat16, 1>(x, p, D.n_mats, s);
  }
  const float* x = static_cast<const float*>(g);
  return D.cols % 4 == 0 ? launch<float, 4>(x, p, D.n_mats, s)
                         : launch<float, 1>(x, p, D.n_mats, s);
}

}  // namespace moe
