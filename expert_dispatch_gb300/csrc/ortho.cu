// ortho.cu -- orthogonalisation of a stack of matrices by Newton-Schulz products
// (the update of the Muon optimiser for the experts' and the router's matrices).
//
// For each matrix G [rows, cols], with m = min(rows, cols), n = max and G
// transposed first if it is tall:
//     X = G / (|G|_F + eps);   steps times:  A = X X^T,  B = a I + b A + c A A,  X = B X,
// a, b, c = 3.4445, -4.7750, 2.0315: an odd polynomial that drives every
// singular value of X (all in (0, 1] at the start) towards 1.
//
// Precision.  The products run on the tensor cores with fp16 operands and fp32
// accumulators.  fp16 keeps 11 bits where bf16 keeps 8: on the same inputs the
// result is off by about 1e-3 with fp16 operands and 1e-2 with bf16 ones (its
// own rounding to bf16 is 1.7e-3).  fp16's narrow range is met by powers of two:
// X is stored times 2^10 (entries up to about 1.2, of order 1/sqrt(m n) at the
// start), A times 2^14 (up to 1.5, and 1/m) and B times 2^12 (up to 3.5).
// Because |G|_F is rounded down to a power of two for the first X, a bf16 input
// is held without error; the remaining factor in (1/2, 1] is applied in fp32 to
// the first products.  B holds a I + b A + c A A as one matrix, so the update
// needs no second pass over X and no cancelling difference of rounded terms.
//
// Work.  A and B are symmetric: only the tiles of one triangle are computed and
// each is written twice, straight and mirrored.  X is kept in both layouts,
// X [m, n] for X X^T and X^T [n, m] for B X, so every operand is K-major.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "tc_common.cuh"

namespace moe {
namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kScaleX = 1024.f, kScaleA = 16384.f, kScaleB = 4096.f;
constexpr int kSumBlocks = 64;  // most blocks of the norm's sum, per matrix

struct Scale {
  float f1, f2;  // X = g * f1 * f2, powers of two (one factor could leave fp32's range)
  float rho;     // what is left of 1 / (|G| + eps), in (1/2, 1]
  float pad;
};

// ---------------------------------------------------------------- norm and first X
__device__ __forceinline__ float load_elem(const void* g, int bf16, size_t i) {
  return bf16 ? load_as_f32(static_cast<const __nv_bfloat16*>(g), i)
              : static_cast<const float*>(g)[i];
}

constexpr float kBig = 0x1p45f, kSmall = 0x1p-45f, kUp = 0x1p84f, kDown = 0x1p-84f;

// Sums of squares of one matrix, block blockIdx.x of gridDim.x; three sums so
// that no square over- or underflows: of values above 2^45 times 2^-84, of
// values below 2^-45 times 2^84, and of the rest.
__global__ void __launch_bounds__(512)
    ortho_sumsq_kernel(const void* g, int bf16, size_t per_mat, float* partial, int* flags) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[3][16];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) flags[0] = 0;
  const size_t base = (size_t)blockIdx.y * per_mat;
  float s[3] = {0.f, 0.f, 0.f};
  auto add = [&](float x) {
    const float ax = fabsf(x);
    if (ax > kBig) {
      s[0] = fmaf(x * kDown, x * kDown, s[0]);
    } else if (ax < kSmall) {
      s[2] = fmaf(x * kUp, x * kUp, s[2]);
    } else {
      s[1] = fmaf(x, x, s[1]);
    }
  };
  const size_t stride = (size_t)gridDim.x * blockDim.x;
  for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < per_mat; i += stride)
    add(load_elem(g, bf16, base + i));
#pragma unroll
  for (int q = 0; q < 3; ++q) {
#pragma unroll
    for (int o = 16; o; o >>= 1) s[q] += __shfl_xor_sync(0xffffffffu, s[q], o);
    if ((threadIdx.x & 31) == 0) red[q][threadIdx.x >> 5] = s[q];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    float v = 0.f;
    for (int w = 0; w < 16; ++w) v += red[threadIdx.x][w];
    partial[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * 3 + threadIdx.x] = v;
  }
}

// The scale of one matrix from its partial sums, added by one warp in a fixed
// order.
__device__ Scale matrix_scale(const float* partial, int n, float eps) {
  float s[3] = {0.f, 0.f, 0.f};
  for (int i = threadIdx.x & 31; i < n; i += 32)
#pragma unroll
    for (int q = 0; q < 3; ++q) s[q] += partial[i * 3 + q];
#pragma unroll
  for (int q = 0; q < 3; ++q)
#pragma unroll
    for (int o = 16; o; o >>= 1) s[q] += __shfl_xor_sync(0xffffffffu, s[q], o);
  // |G| + eps = v * 2^off
  float v;
  int off = 0;
  if (s[0] > 0.f || s[0] != s[0]) {
    v = sqrtf(s[0] + s[1] * kDown * kDown), off = 84;
  } else if (s[1] > 0.f || s[1] != s[1]) {
    v = sqrtf(s[1] + s[2] * kDown * kDown) + eps;
  } else if (eps > 0.f) {
    v = sqrtf(s[2]) * kDown + eps;
  } else {
    v = sqrtf(s[2]), off = -84;
  }
  Scale r{0.f, 0.f, 0.f, 0.f};
  if (v == 0.f) return r;  // a zero matrix, eps = 0: X = 0
  if (isinf(v) || v != v) {
    r.f1 = r.f2 = r.rho = __int_as_float(0x7fffffff);
    return r;
  }
  const int e = ilogbf(v);
  const int k = 10 - e - off;  // X = g * 2^k
  r.f1 = scalbnf(1.f, k / 2);
  r.f2 = scalbnf(1.f, k - k / 2);
  r.rho = 1.f / scalbnf(v, -e);
  return r;
}

// First X [mp, np] and X^T [np, mp] in fp16, padded with zeros: a 64 x 64 tile a
// block, through shared memory.
__global__ void __launch_bounds__(256)
    ortho_start_kernel(const void* g, int bf16, int rows, int cols, int m, int n, int mp, int np,
                       float eps, const float* partial, int n_partial, Scale* scales, __half* x,
                       __half* xt) {
  pdl_wait();
  pdl_trigger();
  __shared__ Scale sc;
  __shared__ __half tile[64][66];
  const int mat = blockIdx.z, r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;  // of [mp, np]
  if (threadIdx.x < 32) {
    const Scale own = matrix_scale(partial + (size_t)mat * n_partial * 3, n_partial, eps);
    if (threadIdx.x == 0) {
      sc = own;
      if (blockIdx.x == 0 && blockIdx.y == 0) scales[mat] = own;
    }
  }
  __syncthreads();
  const float f1 = sc.f1, f2 = sc.f2;
  const bool tall = rows > cols;
  const size_t base = (size_t)mat * rows * cols;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  // read along the input's rows; `tile` is indexed [row of X][column of X]
  for (int i = ty; i < 64; i += 4) {
    const int xr = tall ? r0 + tx : r0 + i, xc = tall ? c0 + i : c0 + tx;
    float v = 0.f;
    if (xr < m && xc < n)
      v = load_elem(g, bf16, base + (tall ? (size_t)xc * cols + xr : (size_t)xr * cols + xc));
    const __half h = __float2half_rn(v * f1 * f2);
    if (tall)
      tile[tx][i] = h;
    else
      tile[i][tx] = h;
  }
  __syncthreads();
  for (int i = ty; i < 64; i += 4) {
    x[((size_t)mat * mp + r0 + i) * np + c0 + tx] = tile[i][tx];
    xt[((size_t)mat * np + c0 + i) * mp + r0 + tx] = tile[tx][i];
  }
}

// ---------------------------------------------------------------- products
// Product P Q^T of the matrices' K-major operands, on pairs of SMs: a unit is
// (matrix, 256 rows of P, BN rows of Q, all of K).
//   kGram : A  = X X^T, from P = Q = X             -> out, both triangles
//   kPoly : B  = a I + b A + c A A, P = Q = A      -> out, both triangles
//   kApply: X' = B X, P = B, Q = X^T               -> out = X', out_t = X'^T
//   kLast : the same                               -> result in bf16
enum Op { kGram = 0, kPoly = 1, kApply = 2, kLast = 3 };

struct Product {
  int n_mats;
  int K;             // reduction length, a multiple of 64
  int rowsP, rowsQ;  // padded rows a matrix has in P and in Q: multiples of 64
  int m, n;          // the matrices' own size
  int first;         // X is the first one: apply rho
  const Scale* scales;
  __half* out;             // [n_mats * rowsP, rowsQ]
  __half* out_t;           // kApply: [n_mats * rowsQ, rowsP]
  const __half* gram;      // kPoly: A
  __nv_bfloat16* result;   // kLast: [n_mats, m, n], or [n_mats, n, m] if tall
  int tall;
  int* err;
};

constexpr int kThreads = 32 * (2 + tc::kEpiWarps);  // producer, MMA, epilogue

template <int BN, int STAGES>
struct Cfg {
  static constexpr int A_BYTES = 128 * 128;       // this CTA's 128 rows of P, 64 columns
  static constexpr int B_BYTES = (BN / 2) * 128;  // this CTA's half of Q's rows
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int TMEM_COLS = 2 * BN;  // two accumulator buffers
  static constexpr int NBARS = 2 * STAGES + 2 * 2 + 1;
  static constexpr int BAR_OFF = STAGES * STAGE_BYTES;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
  static constexpr int SMEM_TOTAL = MISC_OFF + 16 + 1024;
  static_assert(BN == 64 || BN == 128 || BN == 256, "tile");
  static_assert(SMEM_TOTAL <= 232448, "shared memory");
};

// Tiles of one matrix.  Symmetric products take the tiles that meet the lower
// triangle: row block i spans R column tiles and has (i + 1) R of them, less
// what the last one lacks.
template <int BN, bool SYM>
struct Tiles {
  static constexpr int R = 256 / BN;
  int mt, nt;
  __host__ __device__ Tiles(int rowsP, int rowsQ)
      : mt((rowsP + 255) / 256), nt((rowsQ + BN - 1) / BN) {}
  __host__ __device__ int count() const {
    if (!SYM) return mt * nt;
    return R * mt * (mt + 1) / 2 - (mt * R - nt);
  }
  __device__ void at(int u, int& i, int& j) const {
    if (!SYM) {  // the row blocks of a column tile back to back
      i = u % mt;
      j = u / mt;
      return;
    }
    i = 0;
    while (u >= (i + 1) * R) u -= ++i * R;
    j = u;
  }
};

__device__ __forceinline__ void store_row16(__half* p, const float (&v)[16]) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]),
               "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}

// 16 values of row `row` of the last product, columns c0 .. c0 + 15.
__device__ __forceinline__ void store_result16(const Product& p, int mat, int row, int c0,
                                               const float (&v)[16]) {
  __nv_bfloat16* base = p.result + (size_t)mat * p.m * p.n;
  if (p.tall) {  // [n, m]: a warp's lanes hold consecutive elements
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (c0 + j < p.n) base[(size_t)(c0 + j) * p.m + row] = __float2bfloat16_rn(v[j]);
    return;
  }
  __nv_bfloat16* dst = base + (size_t)row * p.n + c0;
  if (p.n % 8 == 0) {  // 16-byte aligned rows
#pragma unroll
    for (int j = 0; j < 16; j += 8) {
      if (c0 + j >= p.n) break;
      uint32_t w[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[j + 2 * t], v[j + 2 * t + 1]);
        w[t] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(dst + j) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (c0 + j < p.n) dst[j] = __float2bfloat16_rn(v[j]);
}

template <int OP, int BN, int STAGES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ortho_product_kernel(const __grid_constant__ CUtensorMap tmP,
                         const __grid_constant__ CUtensorMap tmQ, const Product p) {
  using C = Cfg<BN, STAGES>;
  constexpr bool SYM = OP == kGram || OP == kPoly;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::BAR_OFF;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  const uint32_t accf0 = bar0 + 8u * (2 * STAGES);
  const uint32_t acce0 = accf0 + 16u;
  const uint32_t drain_bar = acce0 + 16u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = (int)(blockIdx.x >> 1), n_pairs = (int)(gridDim.x >> 1);
  const Tiles<BN, SYM> tiles(p.rowsP, p.rowsQ);
  const int per_mat = tiles.count(), total = per_mat * p.n_mats;
  const int KB = p.K / 64;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf0 + 8u * b, 1);
      mbar_init(acce0 + 8u * b, 2 * tc::kEpiWarps);  // the epilogue warps of both CTAs
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before either signals the other
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();  // the operands, A and the scales are the predecessors' outputs
  pdl_trigger();

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (both CTAs)
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_parity = 0;
      bool ok = true;
      for (int u = pair; u < total && ok && !*abort_flag; u += n_pairs) {
        const int mat = u / per_mat;
        int i, j;
        tiles.at(u - mat * per_mat, i, j);
        const int prow = mat * p.rowsP + i * 256 + (int)rank * 128;
        const int qrow = mat * p.rowsQ + j * BN + (int)rank * (BN / 2);
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          if (rank == 0) {
            mbar_arrive_expect_tx(full_bar(stage), 2 * C::STAGE_BYTES);
            armed |= 1u << stage;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          }
          const uint32_t fb = mapa_shared(full_bar(stage), 0);
          const uint32_t s = sbase + stage * C::STAGE_BYTES;
          tma_load_2d_pair(s, &tmP, fb, kb * 64, prow);
          tma_load_2d_pair(s + C::A_BYTES, &tmQ, fb, kb * 64, qrow);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (rank == 0) {
        // wind down: every stage armed here has received both CTAs' copies
        for (int s = 0; s < STAGES; ++s)
          if (armed & (1u << s)) tc::mbar_wait_drain(full_bar(s), (armed_parity >> s) & 1u, p.err);
      } else if (*abort_flag) {
        // this CTA's copies complete on its partner's barriers: after giving
        // up, leave them a bounded time to land before the shared memory goes
        const unsigned long long t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 100000ull) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_f16_f32(256, BN);
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool issued = false;
      for (int u = pair; u < total && !*abort_flag; u += n_pairs, ++it) {
        const int buf = it & 1;
        if (!mbar_wait(acce0 + 8u * buf, ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag, p.err))
          break;
        tc_fence_after();
        const uint32_t d0 = tmem_base + (uint32_t)(buf * BN);
        bool ok = true;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(full_bar(stage), phase, abort_flag, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t s = sbase + stage * C::STAGE_BYTES;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_pair(d0, smem_desc_sw128(s + kk * 32),
                           smem_desc_sw128(s + C::A_BYTES + kk * 32), idesc, kb | kk ? 1u : 0u);
          issued = true;
          umma_commit_pair_mc(empty_bar(stage), 3);  // both CTAs' stage is free again
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair_mc(accf0 + 8u * buf, 3);  // both CTAs' accumulators are ready
      }
      // wind down: every MMA issued here has completed before the pair's TMEM is freed
      if (issued) {
        umma_commit_pair_mc(drain_bar, 1);
        tc::mbar_wait_drain(drain_bar, 0, p.err);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 2..9, both CTAs)
    // A warp reads its TMEM lane quarter (row = lane); the two warps of a
    // quarter take one half of the columns each, 16 at a time: one 32-byte
    // store along the row, and 16 stores of 64 bytes a warp for the mirrored
    // or transposed copy.
    const int q = warp & 3, half = (warp - 2) >> 2;
    int it = 0;
    for (int u = pair; u < total; u += n_pairs, ++it) {
      const int mat = u / per_mat;
      int ti, tj;
      tiles.at(u - mat * per_mat, ti, tj);
      const int buf = it & 1;
      if (!tc::mbar_wait_warp(accf0 + 8u * buf, (uint32_t)(it >> 1) & 1u, abort_flag, p.err)) break;
      tc_fence_after();
      const int row = ti * 256 + (int)rank * 128 + q * 32 + lane;
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * BN);
      const float rho = p.first ? p.scales[mat].rho : 1.f;
      const float alpha = OP == kGram    ? rho * rho * (kScaleA / (kScaleX * kScaleX))
                          : OP == kPoly  ? kC * (kScaleB / (kScaleA * kScaleA))
                          : OP == kApply ? rho / kScaleB
                                         : rho / (kScaleB * kScaleX);
      const bool mirror = SYM && (tj + 1) * BN <= ti * 256;
      const size_t out_row = ((size_t)mat * p.rowsP + row) * p.rowsQ;
#pragma unroll 1
      for (int cc = half * (BN / 2); cc < (half + 1) * (BN / 2); cc += 16) {
        const int c0 = tj * BN + cc;
        if (c0 >= p.rowsQ) break;  // warp-uniform
        uint32_t a[16];
        tmem_ld16(tb + cc, a);
        tmem_ld_wait();
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = alpha * __uint_as_float(a[j]);
        if (OP == kLast) {
          if (row < p.m) store_result16(p, mat, row, c0, v);
        } else if (row < p.rowsP) {
          if (OP == kPoly) {
            const uint4* src = reinterpret_cast<const uint4*>(p.gram + out_row + c0);
            const uint4 g0 = src[0], g1 = src[1];
            const uint32_t gw[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const __half2 h = *reinterpret_cast<const __half2*>(&gw[j / 2]);
              const float g = __half2float(j & 1 ? __high2half(h) : __low2half(h));
              v[j] = fmaf(kB * (kScaleB / kScaleA), g, v[j]);
              if (row == c0 + j && row < p.m) v[j] += kA * kScaleB;
            }
          }
          store_row16(p.out + out_row + c0, v);
          if (mirror || OP == kApply) {
            __half* t = OP == kApply ? p.out_t : p.out;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              t[((size_t)mat * p.rowsQ + c0 + j) * p.rowsP + row] = __float2half_rn(v[j]);
          }
        }
        __syncwarp();  // the next tcgen05.ld is the whole warp's
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(acce0 + 8u * buf, 0));
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the partner is done with this CTA's shared memory and TMEM
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
  }
}

template <int OP, int BN, int STAGES>
cudaError_t launch_product(const void* P, const void* Q, const Product& p, cudaStream_t s) {
  using C = Cfg<BN, STAGES>;
  auto kern = ortho_product_kernel<OP, BN, STAGES>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  // pairs that fit on the device at once; the grid never exceeds it
  static int max_clusters[64] = {};
  static std::mutex mu;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (max_clusters[dev] == 0) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_TOTAL);
      if (e != cudaSuccess) return e;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2 * (unsigned)(num_sms() / 2));
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = C::SMEM_TOTAL;
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
      if (e != cudaSuccess) return e;
      if (n <= 0) return cudaErrorInvalidConfiguration;
      max_clusters[dev] = n;
    }
  }
  CUtensorMap tp, tq;
  if (!make_tmap_2d(&tp, P, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, (uint64_t)p.K,
                    (uint64_t)p.n_mats * p.rowsP, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_2d(&tq, Q, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, (uint64_t)p.K,
                    (uint64_t)p.n_mats * p.rowsQ, 64, BN / 2, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const Tiles<BN, OP == kGram || OP == kPoly> tiles(p.rowsP, p.rowsQ);
  const long long units = (long long)tiles.count() * p.n_mats;
  const long long pairs = units < max_clusters[dev] ? units : max_clusters[dev];
  ProfScope pr(OP == kGram ? "ortho_gram" : OP == kPoly ? "ortho_poly" : "ortho_apply", s);
  (void)launch_kernel(kern, (unsigned)(2 * pairs), kThreads, C::SMEM_TOTAL, s, tp, tq, p);
  return cudaGetLastError();
}

template <int OP>
cudaError_t product(const void* P, const void* Q, const Product& p, cudaStream_t s) {
  return launch_product<OP, 256, 6>(P, Q, p, s);
}

int sum_blocks(size_t per_mat) {
  const size_t want = (per_mat + 16383) / 16384;  // 32 elements a thread
  return want < kSumBlocks ? (int)want : kSumBlocks;
}

}  // namespace

OrthoLayout ortho_layout(const moe_ortho_desc& D) {
  OrthoLayout L{};
  const size_t n = (size_t)D.n_mats;
  const int m = D.rows < D.cols ? D.rows : D.cols, c = D.rows < D.cols ? D.cols : D.rows;
  L.mp = (m + 63) / 64 * 64;
  L.np = (c + 63) / 64 * 64;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) & ~(size_t)255;
    return o;
  };
  L.partial = take(n * kSumBlocks * 3 * sizeof(float));
  L.scales = take(n * sizeof(Scale));
  L.x = take(n * L.mp * L.np * 2);
  for (size_t& o : L.xt) o = take(n * L.mp * L.np * 2);
  L.gram = take(n * L.mp * L.mp * 2);
  L.poly = take(n * L.mp * L.mp * 2);
  L.total = 512 + off;  // the flags' 16 bytes, then the regions at the next multiple of 256
  return L;
}

cudaError_t launch_orthogonalize(const moe_ortho_desc& D, const void* g, void* out, void* ws,
                                 cudaStream_t s) {
  const OrthoLayout L = ortho_layout(D);
  int* flags = static_cast<int*>(ws);
  uint8_t* b = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ws) + 16 + 255) &
                                          ~(uintptr_t)255);
  const int m = D.rows < D.cols ? D.rows : D.cols, n = D.rows < D.cols ? D.cols : D.rows;
  const int bf16 = D.dtype == MOE_BF16;
  const size_t per_mat = (size_t)D.rows * D.cols;
  float* partial = reinterpret_cast<float*>(b + L.partial);
  Scale* scales = reinterpret_cast<Scale*>(b + L.scales);
  __half* x = reinterpret_cast<__half*>(b + L.x);
  __half* xt[2] = {reinterpret_cast<__half*>(b + L.xt[0]), reinterpret_cast<__half*>(b + L.xt[1])};
  __half* gram = reinterpret_cast<__half*>(b + L.gram);
  __half* poly = reinterpret_cast<__half*>(b + L.poly);
  const int nb = sum_blocks(per_mat);
  {
    ProfScope pr("ortho_sumsq", s);
    (void)launch_kernel(ortho_sumsq_kernel, dim3(nb, D.n_mats), 512, 0, s, g, bf16, per_mat,
                        partial, flags);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  {
    ProfScope pr("ortho_start", s);
    (void)launch_kernel(ortho_start_kernel, dim3(L.np / 64, L.mp / 64, D.n_mats), 256, 0, s, g,
                        bf16, D.rows, D.cols, m, n, L.mp, L.np, D.eps, partial, nb, scales, x,
                        xt[0]);
  }
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  Product p{};
  p.n_mats = D.n_mats;
  p.m = m, p.n = n;
  p.scales = scales;
  p.err = flags;
  p.tall = D.rows > D.cols;
  p.result = static_cast<__nv_bfloat16*>(out);
  for (int i = 0; i < D.steps; ++i) {
    p.first = i == 0;
    p.K = L.np, p.rowsP = p.rowsQ = L.mp;
    p.out = gram;
    if ((e = product<kGram>(x, x, p, s)) != cudaSuccess) return e;
    p.K = L.mp;
    p.gram = gram, p.out = poly;
    if ((e = product<kPoly>(gram, gram, p, s)) != cudaSuccess) return e;
    p.rowsQ = L.np;
    p.out = x, p.out_t = xt[(i + 1) & 1];
    e = i + 1 < D.steps ? product<kApply>(poly, xt[i & 1], p, s)
                        : product<kLast>(poly, xt[i & 1], p, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace moe
