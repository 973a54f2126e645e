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
// accumulators, for fp32 matrices too: the output is bf16, whose rounding alone is
// 1.7e-3 of its norm, and operands split into two fp16 parts would take three products
// for each.  fp16 keeps 11 bits where bf16 keeps 8: on the same inputs the
// result is off by about 1e-3 with fp16 operands and 1e-2 with bf16 ones, where the
// singular values grow together.  Where a few directions hold almost all of the
// norm, the roundings of A and B (relative to those) weigh on the others until they
// have grown: 2e-2 for singular values falling as 1/k^2, up to 4e-2 where all but
// eight are 0.1 % of the largest; the tests hold the kernels to twice what these
// roundings alone give in 64 bits.  fp16's narrow range is met by powers of two:
// X is stored times 2^10 (entries up to about 1.2, of order 1/sqrt(m n) at the
// start; where eps outweighs |G|, more: Scale in ortho.cuh), A times 2^14 (up to 1.5,
// and 1/m) and B times 2^12 (up to 3.5).
// Because |G|_F is rounded down to a power of two for the first X, a bf16 input
// is held without error; the remaining factor in (1/2, 1] is applied in fp32 to
// the first products.  B holds a I + b A + c A A as one matrix, so the update
// needs no second pass over X and no cancelling difference of rounded terms.
//
// Work.  A and B are symmetric: only the tiles of one triangle are computed and
// each is written twice, straight and mirrored.  X [m, n] is the only copy of
// X: it is K-major in X X^T, and in B X the tensor cores read it MN-major
// (rows of 64 columns of X, the reduction running down the rows), so no
// transposed copy is written.
//
// Two steps at once.  With B0 the first step's B, A after it is B0 A B0, so that
// two steps are X = (B1 B0) X with B1 = a I + b A1 + c A1 A1, A1 = (B0 A) B0: five
// m x m products take the place of one product each of X X^T and of B X.  All
// of them commute, so they are symmetric and one triangle is enough.  That is
// fewer operations where n is well above m; measured, 4 x 7168 x 2048 bf16 1438
// -> 1182 us, 16 x 1536 x 4096 2060 -> 1794 us.  Five steps run as 2 + 1 + 2: X is
// formed and rounded again before errors of A (which sees the squares of the
// singular values) have grown; the error of the result is that of five single
// steps within a few percent, while all five on A alone lose what has small
// singular values (0.2 where the direct form has 3e-3, singular values falling as
// 1/k).
//
// Waits are bounded (common.cuh).  One that expires leaves a part of a product
// unwritten and raises the workspace's flag: the last product, which reads the flag
// once its predecessors are done, then makes every result NaN.  What a wait of the
// last product itself keeps from being computed is written as NaN.
//
// Matrices with m <= 128 and n up to a cluster's shared memory take one launch of
// the kernel in ortho_chip.cu; what follows here serves the others.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "ortho.cuh"
#include "tc_common.cuh"

namespace moe {
namespace {

using namespace ortho;

constexpr int kSumBlocks = 128;  // most blocks of the norm's sum, per matrix

// ---------------------------------------------------------------- norm and first X
// Sums of squares of one matrix, block blockIdx.x of gridDim.x: a plain sum, or
// where that is not good (ortho.cuh) three, over values read again.  A matrix that
// starts off a 16-byte boundary is read in vectors from the next one on.
template <typename T>
__global__ void __launch_bounds__(512)
    ortho_sumsq_kernel(const T* g, size_t per_mat, float* partial, int* flags) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[16];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) flags[0] = 0;
  constexpr int V = 16 / (int)sizeof(T);
  const T* p = g + (size_t)blockIdx.y * per_mat;
  const size_t tid = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  const size_t stride = (size_t)gridDim.x * blockDim.x;
  const size_t off = (reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T);
  const size_t head = off ? (V - off < per_mat ? V - off : per_mat) : 0;
  const size_t nv = (per_mat - head) / V, tail = head + nv * V;
  auto each = [&](auto&& add) {
    if (tid < head) add(load_as_f32(p, tid));
    if (tid < per_mat - tail) add(load_as_f32(p, tail + tid));
    constexpr int U = 4;  // vectors in flight
    for (size_t i = tid; i < nv; i += U * stride) {
      float v[U][V];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (i + k * stride < nv) {
          load_elems<T, V>(p + head + (i + k * stride) * V, v[k]);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) v[k][j] = 0.f;
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) add(v[k][j]);
    }
  };
  auto block_sum = [&](float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < 16; ++w) v += red[w];
    return v;
  };
  float s[3] = {0.f, 0.f, 0.f};
  each([&](float x) { s[1] = fmaf(x, x, s[1]); });
  s[1] = block_sum(s[1]);
  if (!plain_sum(s[1])) {
    s[1] = 0.f;
    each([&](float x) { add_square(x, s); });
#pragma unroll
    for (int q = 0; q < 3; ++q) s[q] = block_sum(s[q]);
  }
  if (threadIdx.x < 3)
    partial[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * 3 + threadIdx.x] =
        threadIdx.x == 0 ? s[0] : threadIdx.x == 1 ? s[1] : s[2];
}

// First X in fp16, padded with zeros: the input, [rows, cols] padded to
// [rp, cp], or its transpose [cp, rp] (TURN): a 64 x 64 tile a block.  A thread
// loads and stores 8 elements of a row at a time; a transposed tile goes
// through shared memory.
template <typename T, bool VEC, bool TURN>
__global__ void __launch_bounds__(256)
    ortho_start_kernel(const T* g, int rows, int cols, int rp, int cp, float eps,
                       const float* partial, int n_partial, Scale* scales, __half* x) {
  pdl_wait();
  pdl_trigger();
  __shared__ Scale sc;
  __shared__ uint32_t tile[64][33];  // two elements a word
  // the last matrices first: the sum before this kernel left them in L2
  const int mat = gridDim.z - 1 - blockIdx.z, r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  const T* src = g + (size_t)mat * rows * cols;
  const int tc = (threadIdx.x & 7) * 8, tr = threadIdx.x >> 3;  // 8 columns of rows tr, tr + 32
  float v[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + tr + 32 * h, c = c0 + tc;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[h][j] = 0.f;
    if (r < rows && c < cols) {
      const T* p = src + (size_t)r * cols + c;
      if constexpr (VEC && sizeof(T) == 2) {  // cols % 8 == 0
        load_elems<T, 8>(p, v[h]);
      } else if constexpr (VEC) {  // cols % 4 == 0
        float q[4];
        load_elems<T, 4>(p, q);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[h][j] = q[j];
        if (c + 4 < cols) {
          load_elems<T, 4>(p + 4, q);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[h][4 + j] = q[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < cols) v[h][j] = load_as_f32(p, j);
      }
    }
  }
  if (threadIdx.x < 32) {
    const Scale own = matrix_scale(partial + (size_t)mat * n_partial * 3, n_partial, eps);
    if (threadIdx.x == 0) {
      sc = own;
      if (blockIdx.x == 0 && blockIdx.y == 0) scales[mat] = own;
    }
  }
  __syncthreads();
  const float f1 = sc.f1, f2 = sc.f2;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 p = __floats2half2_rn(v[h][2 * j] * f1 * f2, v[h][2 * j + 1] * f1 * f2);
      u[j] = *reinterpret_cast<const uint32_t*>(&p);
      if (TURN) tile[tr + 32 * h][tc / 2 + j] = u[j];
    }
    if (!TURN)
      *reinterpret_cast<uint4*>(x + ((size_t)mat * rp + r0 + tr + 32 * h) * cp + c0 + tc) =
          make_uint4(u[0], u[1], u[2], u[3]);
  }
  if (!TURN) return;
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int c = tr + 32 * h;  // this thread writes rows r0 + tc .. + 7 of column c
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = tile[tc + 2 * j][c / 2], b = tile[tc + 2 * j + 1][c / 2];
      u[j] = c & 1 ? (a >> 16) | (b & 0xffff0000u) : (a & 0xffffu) | (b << 16);
    }
    *reinterpret_cast<uint4*>(x + ((size_t)mat * cp + c0 + c) * rp + r0 + tc) =
        make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// ---------------------------------------------------------------- products
// Products of the matrices' operands, on pairs of SMs: a unit is (matrix, 256
// rows of P, BN columns of the product, all of K).  The tiles that are left for
// the last round of the pairs are cut along their columns into as many parts as
// keep every pair to one unit.
//   kGram : alpha P Q^T, symmetric: A = X X^T, or a product of two of the
//           m x m matrices                         -> out, both triangles
//   kPoly : B  = a I + b A + c A A, P = Q = A      -> out, both triangles
//   kApply: X' = B X, P = B, Q = X (MN-major)      -> out
//   kLast : the same                               -> result in bf16
enum Op { kGram = 0, kPoly = 1, kApply = 2, kLast = 3 };

struct Product {
  int n_mats;
  int K;             // reduction length, a multiple of 64
  int rowsP, rowsQ;  // padded rows and columns of a product: multiples of 64
  int m, n;          // the matrices' own size
  int steps;         // steps behind the X that is read: 0, the first one, takes rho; -1: no X
  int ahead;         // kApply: steps that the product takes X forward
  float alpha;       // kGram, kApply, kLast: factor of the accumulators
  int whole, cut;    // SM pairs: units that are whole tiles; the rest are cut into `cut` parts
  const Scale* scales;
  __half* out;             // [n_mats * rowsP, rowsQ]
  const __half* gram;      // kPoly: A
  __nv_bfloat16* result;   // kLast: [n_mats, m, n], or [n_mats, n, m] if tall
  int tall;
  int* err;
};

constexpr int kThreads = 32 * (2 + tc::kEpiWarps);  // producer, MMA, epilogue

struct PairCfg {
  static constexpr int BN = 256, STAGES = 6;
  static constexpr int A_BYTES = 128 * 128;       // this CTA's 128 rows of P, 64 columns
  static constexpr int B_BYTES = (BN / 2) * 128;  // this CTA's half of Q's rows
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int TMEM_COLS = 2 * BN;  // two accumulator buffers
  static constexpr int NBARS = 2 * STAGES + 2 * 2 + 1;
  static constexpr int BAR_OFF = STAGES * STAGE_BYTES;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
  static constexpr int SMEM_TOTAL = MISC_OFF + 16 + 1024;
  static_assert(SMEM_TOTAL + tc::kEpiWarps * 32 * kRowWords * 4 <= 232448, "shared memory");
};

// Tiles of BM x BN of one matrix.  Symmetric products take the tiles that meet
// the lower triangle: row block i spans R column tiles and has (i + 1) R of
// them, less what the last one lacks.
template <int BM, int BN, bool SYM>
struct Tiles {
  static constexpr int R = BM / BN;
  int mt, nt;
  __host__ __device__ Tiles(int rowsP, int rowsQ)
      : mt((rowsP + BM - 1) / BM), nt((rowsQ + BN - 1) / BN) {}
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
  // whether a tile has a mirror image outside the row block's own square
  __device__ bool mirrored(int i, int j) const { return SYM && (j + 1) * BN <= i * BM; }
};

// kLast: whether a wait in one of the call's earlier products expired.
template <int OP>
__device__ __forceinline__ bool predecessors_failed(const Product& p) {
  return OP == kLast && (*static_cast<const volatile int*>(p.err) & kErrTimeout);
}

// The factor of a product's accumulators.
template <int OP>
__device__ __forceinline__ float product_scale(const Product& p, int mat) {
  if (OP == kPoly) return kC * (kScaleB / (kScaleA * kScaleA));
  if (p.steps < 0) return p.alpha;
  const Scale s = p.scales[mat];
  const float rho = p.steps == 0 ? s.rho : 1.f;
  return OP == kGram    ? gram_factor(s, rho * rho * p.alpha, p.steps)
         : OP == kApply ? apply_factor(s, rho * p.alpha, p.steps, p.ahead)
                        : last_factor(s, rho * p.alpha, p.steps);
}

// kPoly: 16 columns of A, to be loaded ahead of their use; other kinds have none.
template <int OP>
__device__ __forceinline__ void load_gram(const Product& p, int mat, int row, int c0,
                                          uint4 (&g)[2]) {
  if (OP != kPoly || row >= p.rowsP) return;
  const uint4* src =
      reinterpret_cast<const uint4*>(p.gram + ((size_t)mat * p.rowsP + row) * p.rowsQ + c0);
#pragma unroll
  for (int i = 0; i < 2; ++i) g[i] = src[i];
}

// Accumulators of W columns (8 or 16) of row `row` from column c0 on, already
// scaled, to the product's outputs: along the row in one 16- or 32-byte store,
// and column by column (64 bytes a warp) for the mirrored copy.
template <int OP, int W>
__device__ __forceinline__ void store_product(const Product& p, int mat, int row, int c0,
                                              bool mirror, const uint4* gram, float (&v)[W]) {
  if (row >= p.rowsP) return;
  const size_t at = ((size_t)mat * p.rowsP + row) * p.rowsQ + c0;
  if (OP == kPoly) {
#pragma unroll
    for (int i = 0; i < W / 8; ++i) {
      const uint32_t gw[4] = {gram[i].x, gram[i].y, gram[i].z, gram[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&gw[j]));
        v[8 * i + 2 * j] = fmaf(kB * (kScaleB / kScaleA), f.x, v[8 * i + 2 * j]);
        v[8 * i + 2 * j + 1] = fmaf(kB * (kScaleB / kScaleA), f.y, v[8 * i + 2 * j + 1]);
      }
    }
    if (row < p.m) {
#pragma unroll
      for (int j = 0; j < W; ++j)
        if (row == c0 + j) v[j] += kA * kScaleB;
    }
  }
  uint32_t u[W / 2];
#pragma unroll
  for (int j = 0; j < W / 2; ++j) u[j] = pack_half2(v[2 * j], v[2 * j + 1]);
  if constexpr (W == 16) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p.out + at),
                 "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]),
                 "r"(u[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(p.out + at) = make_uint4(u[0], u[1], u[2], u[3]);
  }
  if (mirror) {  // rowsP == rowsQ
    uint16_t* t = reinterpret_cast<uint16_t*>(p.out) +
                  ((size_t)mat * p.rowsP + c0) * p.rowsP + row;
#pragma unroll
    for (int j = 0; j < W; ++j)
      t[(size_t)j * p.rowsP] = (uint16_t)(j & 1 ? u[j / 2] >> 16 : u[j / 2] & 0xffffu);
  }
}

template <int OP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ortho_product_kernel(const __grid_constant__ CUtensorMap tmP,
                         const __grid_constant__ CUtensorMap tmQ, const Product p) {
  using C = PairCfg;
  constexpr int BN = C::BN, STAGES = C::STAGES;
  constexpr bool SYM = OP == kGram || OP == kPoly;  // else Q is MN-major
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t scratch[tc::kEpiWarps][OP == kLast ? 32 * kRowWords : 1];
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
  const Tiles<256, BN, SYM> tiles(p.rowsP, p.rowsQ);
  const int per_mat = tiles.count(), whole = p.whole;
  const int total = whole + (per_mat * p.n_mats - whole) * p.cut;
  const int KB = p.K / 64;
  // unit u -> matrix, row block, first column and width
  auto unit = [&](int u, int& mat, int& ti, int& col, int& width) {
    int tile = u, part = 0;
    width = BN;
    if (u >= whole) {
      part = (u - whole) % p.cut;
      tile = whole + (u - whole) / p.cut;
      width = BN / p.cut;
    }
    mat = tile / per_mat;
    int tj;
    tiles.at(tile - mat * per_mat, ti, tj);
    col = tj * BN + part * width;
  };

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
        int mat, ti, col, width;
        unit(u, mat, ti, col, width);
        const int prow = mat * p.rowsP + ti * 256 + (int)rank * 128;
        const int qcol = col + (int)rank * (width / 2);
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.err)) {
            ok = false;
            break;
          }
          if (rank == 0) {
            mbar_arrive_expect_tx(full_bar(stage), 2 * (C::A_BYTES + (width / 2) * 128));
            armed |= 1u << stage;
            armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
          }
          const uint32_t fb = mapa_shared(full_bar(stage), 0);
          const uint32_t s = sbase + stage * C::STAGE_BYTES;
          tma_load_2d_pair(s, &tmP, fb, kb * 64, prow);
          for (int c = 0; c < width / 2; c += 64) {  // boxes of 64 columns of the product
            if (SYM)
              tma_load_2d_pair(s + C::A_BYTES + c * 128, &tmQ, fb, kb * 64,
                               mat * p.rowsQ + qcol + c);
            else
              tma_load_2d_pair(s + C::A_BYTES + c * 128, &tmQ, fb, qcol + c, mat * p.K + kb * 64);
          }
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
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool issued = false;
      for (int u = pair; u < total && !*abort_flag; u += n_pairs, ++it) {
        const int buf = it & 1;
        if (!mbar_wait(acce0 + 8u * buf, ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag, p.err))
          break;
        tc_fence_after();
        const uint32_t d0 = tmem_base + (uint32_t)(buf * BN);
        const uint32_t idesc =
            idesc_f16_f32(256, u < whole ? BN : BN / p.cut) | (SYM ? 0u : kTransposeB);
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
                           SYM ? smem_desc_sw128(s + C::A_BYTES + kk * 32)
                               : smem_desc_mn128(s + C::A_BYTES + kk * 2048, 8192),
                           idesc, kb | kk ? 1u : 0u);
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
    // quarter take one half of the unit's columns each, 32 at a time.
    const int q = warp & 3, half = (warp - 2) >> 2;
    const bool failed = predecessors_failed<OP>(p);
    bool ok = true;  // once a wait has expired: NaN for this warp's share of all units left
    int it = 0;
    for (int u = pair; u < total; u += n_pairs, ++it) {
      int mat, ti, col, width;
      unit(u, mat, ti, col, width);
      const int buf = it & 1;
      const float scale = product_scale<OP>(p, mat);
      ok = ok && tc::mbar_wait_warp(accf0 + 8u * buf, (uint32_t)(it >> 1) & 1u, abort_flag, p.err);
      if (!ok && OP != kLast) break;
      tc_fence_after();
      const int row = ti * 256 + (int)rank * 128 + q * 32 + lane;
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * BN);
      const float alpha = ok && !failed ? scale : quiet_nan();
      const bool mirror = tiles.mirrored(ti, col / BN);
#pragma unroll 1
      for (int cc = half * (width / 2); cc < (half + 1) * (width / 2); cc += 32) {
        if (col + cc >= p.rowsQ) break;  // warp-uniform; rowsQ is a multiple of 64
        uint32_t a[2][16];
        uint4 gram[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          load_gram<OP>(p, mat, row, col + cc + 16 * i, gram[i]);
          tmem_ld16(tb + cc + 16 * i, a[i]);
        }
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c0 = col + cc + 16 * i;
          float v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = alpha * __uint_as_float(a[i][j]);
          if constexpr (OP == kLast)
            store_result(p.result + (size_t)mat * p.m * p.n, p.m, p.n, p.tall, row - lane, c0, v,
                         scratch[warp - 2]);
          else
            store_product<OP, 16>(p, mat, row, c0, mirror, gram[i], v);
        }
        __syncwarp();  // the next tcgen05.ld is the whole warp's
      }
      tc_fence_before();
      __syncwarp();
      // after giving up, no arrival that would count for a warp still reading
      if (ok && lane == 0) mbar_arrive_cluster(mapa_shared(acce0 + 8u * buf, 0));
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

// The same products where they have few tiles: one CTA a tile of 128 x 64, or, for
// X X^T (kGram) with its long reduction, a cluster of `split` CTAs that share the
// tile's reduction length.  There a CTA leaves its partial sums in its shared
// memory, and after a cluster barrier each adds up its share of the columns over
// the cluster in rank order.
constexpr int kSmallN = 64, kSmallStages = 4, kSmallWarps = 6;  // producer, MMA, 4 epilogue
constexpr int kSmallThreads = 32 * kSmallWarps;
constexpr int kMaxSplit = 8;

struct SmallCfg {
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = kSmallN * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int BAR_OFF = kSmallStages * STAGE_BYTES;
  static constexpr int MISC_OFF = BAR_OFF + (2 * kSmallStages + 2) * 8;
  static constexpr int SMEM_TOTAL = MISC_OFF + 16 + 1024;
  static_assert(kSmallN * 128 * 4 <= BAR_OFF, "partial sums reuse the stages");
};

// Two CTAs share an SM (their shared memory allows no third).  Told so, the compiler
// gives each the registers of half an SM and keeps the loads of an epilogue in
// flight: 1 x 2048 x 2048 205.0 -> 200.1 us, 1 x 1536 x 4096 222.2 -> 217.0.
template <int OP>
__global__ void __launch_bounds__(kSmallThreads, 2)
    ortho_small_kernel(const __grid_constant__ CUtensorMap tmP,
                       const __grid_constant__ CUtensorMap tmQ, const Product p, int split) {
  using C = SmallCfg;
  constexpr bool SYM = OP == kGram || OP == kPoly;
  if constexpr (OP != kGram) split = 1;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t scratch[4][OP == kLast ? 32 * kRowWords : 1];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::BAR_OFF;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kSmallStages + s); };
  const uint32_t accf = bar0 + 8u * (2 * kSmallStages), drain_bar = accf + 8u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = (int)blockIdx.x / split, rank = (int)blockIdx.x - unit * split;
  const Tiles<128, kSmallN, SYM> tiles(p.rowsP, p.rowsQ);
  const int per_mat = tiles.count(), mat = unit / per_mat;
  int ti, tj;
  tiles.at(unit - mat * per_mat, ti, tj);
  const int KB = p.K / 64, kb0 = KB * rank / split, kb1 = KB * (rank + 1) / split;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kSmallStages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(accf, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kSmallN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();  // the operands, A and the scales are the predecessors' outputs
  pdl_trigger();

  const int q = warp & 3;  // epilogue warps 2..5: the TMEM lane quarter
  const int row = ti * 128 + q * 32 + lane;
  const bool mirror = tiles.mirrored(ti, tj);
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_parity = 0;
      const int prow = mat * p.rowsP + ti * 128, qcol = tj * kSmallN;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.err)) break;
        mbar_arrive_expect_tx(full_bar(stage), C::STAGE_BYTES);
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        const uint32_t s = sbase + stage * C::STAGE_BYTES;
        tma_load_2d(s, &tmP, full_bar(stage), kb * 64, prow);
        if (SYM)
          tma_load_2d(s + C::A_BYTES, &tmQ, full_bar(stage), kb * 64, mat * p.rowsQ + qcol);
        else
          tma_load_2d(s + C::A_BYTES, &tmQ, full_bar(stage), qcol, mat * p.K + kb * 64);
        if (++stage == kSmallStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      for (int s = 0; s < kSmallStages; ++s)  // every stage armed has received its copies
        if (armed & (1u << s)) tc::mbar_wait_drain(full_bar(s), (armed_parity >> s) & 1u, p.err);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_f16_f32(128, kSmallN) | (SYM ? 0u : kTransposeB);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = mbar_wait(full_bar(stage), phase, abort_flag, p.err))) break;
        tc_fence_after();
        const uint32_t s = sbase + stage * C::STAGE_BYTES;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16(tmem_base, smem_desc_sw128(s + kk * 32),
                    SYM ? smem_desc_sw128(s + C::A_BYTES + kk * 32)
                        : smem_desc_mn128(s + C::A_BYTES + kk * 2048, 8192),
                    idesc, kb != kb0 || kk ? 1u : 0u);
        umma_commit(empty_bar(stage));
        if (++stage == kSmallStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok) umma_commit(accf);
      umma_commit(drain_bar);  // every MMA has completed before the TMEM is freed
      tc::mbar_wait_drain(drain_bar, 0, p.err);
    }
  } else {
    // the row's part of A while the products run
    uint4 gram[kSmallN / 8];
    if (OP == kPoly) {
#pragma unroll
      for (int i = 0; i < kSmallN / 16; ++i)
        load_gram<OP>(p, mat, row, tj * kSmallN + 16 * i,
                          *reinterpret_cast<uint4(*)[2]>(&gram[2 * i]));
    }
    const bool failed = predecessors_failed<OP>(p);
    const float scale = product_scale<OP>(p, mat);
    const bool ready = tc::mbar_wait_warp(accf, 0, abort_flag, p.err);
    tc_fence_after();
    const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16);
    const float alpha = ready && !failed ? scale : quiet_nan();
    float* part = reinterpret_cast<float*>(smem);  // [kSmallN][128]
#pragma unroll
    for (int cc = 0; cc < kSmallN; cc += 16) {  // rowsQ is a multiple of the tile's width
      if (!ready && OP != kLast) break;
      const int c0 = tj * kSmallN + cc;
      uint32_t a[16];
      tmem_ld16(tb + cc, a);
      tmem_ld_wait();
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = alpha * __uint_as_float(a[j]);
      if (OP == kLast) {
        store_result(p.result + (size_t)mat * p.m * p.n, p.m, p.n, p.tall, row - lane, c0, v,
                     scratch[warp - 2]);
      } else if (split == 1) {
        store_product<OP, 16>(p, mat, row, c0, mirror, &gram[cc / 8], v);
      } else {
        // the stages' last reader was the MMA that this warp waited for
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(cc + j) * 128 + q * 32 + lane] = v[j];
      }
      __syncwarp();  // the next tcgen05.ld is the whole warp's
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kSmallN);
  }
  if (split == 1) return;
  if constexpr (OP == kGram) {
    cluster_sync();  // every CTA's partial sums are in place
    if (warp >= 2) {
      const int cols = kSmallN / split;  // 8 at least
      for (int cc = rank * cols; cc < (rank + 1) * cols; cc += 8) {
        const uint32_t mine = sbase + (uint32_t)(cc * 128 + q * 32 + lane) * 4u;
        float part[kMaxSplit][8];  // all loads in flight before the first sum
#pragma unroll
        for (int r = 0; r < kMaxSplit; ++r) {
          if (r < split) {
            const uint32_t peer = mapa_shared(mine, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) part[r][j] = ld_shared_cluster(peer + (uint32_t)j * 512u);
          }
        }
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = part[0][j];
#pragma unroll
          for (int r = 1; r < kMaxSplit; ++r)
            if (r < split) v[j] += part[r][j];
        }
        store_product<OP, 8>(p, mat, row, tj * kSmallN + cc, mirror, nullptr, v);
      }
    }
    cluster_sync();  // a CTA's shared memory stays until its peers have read it
  }
}

// ---------------------------------------------------------------- host
// Tensor maps of one operand, boxes of 64 columns by 128 or 64 rows.
struct OperandMaps {
  CUtensorMap rows128, rows64;
};

bool make_maps(OperandMaps* o, const void* base, int K, long long rows) {
  return make_tmap_2d(&o->rows128, base, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, (uint64_t)K,
                      (uint64_t)rows, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) &&
         make_tmap_2d(&o->rows64, base, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, (uint64_t)K,
                      (uint64_t)rows, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B);
}

constexpr const char* kOpName[] = {"ortho_gram", "ortho_poly", "ortho_apply", "ortho_apply"};

template <int OP>
cudaError_t launch_pairs(const OperandMaps& P, const OperandMaps& Q, Product p,
                         long long tiles, cudaStream_t s) {
  using C = PairCfg;
  auto kern = ortho_product_kernel<OP>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  // pairs that fit on the device at once; the grid never exceeds it
  static int max_clusters[64] = {};
  static std::mutex mu;
  int most;
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
    most = max_clusters[dev];
  }
  const int rest = (int)(tiles % most);
  p.cut = 2 * rest <= most ? 2 : 1;
  p.whole = (int)tiles - (p.cut > 1 ? rest : 0);
  const long long units = p.whole + (tiles - p.whole) * p.cut;
  const long long pairs = units < most ? units : most;
  ProfScope pr(kOpName[OP], s);
  (void)launch_kernel(kern, (unsigned)(2 * pairs), kThreads, C::SMEM_TOTAL, s, P.rows128,
                      Q.rows64, p);
  return cudaGetLastError();
}

template <int OP>
cudaError_t launch_small(const OperandMaps& P, const OperandMaps& Q, const Product& p,
                         long long units, int split, cudaStream_t s) {
  using C = SmallCfg;
  auto kern = ortho_small_kernel<OP>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  static std::atomic<bool> configured[64] = {};
  if (!configured[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_TOTAL);
    if (e != cudaSuccess) return e;
    configured[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * split));
  cfg.blockDim = dim3(kSmallThreads);
  cfg.dynamicSmemBytes = C::SMEM_TOTAL;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  ProfScope pr(kOpName[OP], s);
  count_launch();
  (void)cudaLaunchKernelEx(&cfg, kern, P.rows128, Q.rows64, p, split);
  return cudaGetLastError();
}

// Whether a product runs in 256 x 256 tiles on SM pairs or in 128 x 64 tiles,
// and over how many CTAs a small tile's reduction is shared: whatever these
// times, fitted to graph replays of whole calls (bf16), say is least.  In 10 ns:
//   pairs: 27 a round of the pairs and 64-column block of the reduction
//          (512 cycles of the tensor cores), and 550 for a tile's first loads
//          and its epilogue;
//   small: 17 a block (24 KB from L2 into an SM) and 125 of prologue and
//          epilogue for each tile an SM has, and 125 once; a shared reduction
//          adds 400 for the cluster's launch, barriers and exchange.
// Measured, us a call: 4 x 512 x 512 98 pairs, 74 small; 2 x 1536 x 4096 340
// pairs, 516 small; 1 x 1024 x 1024 130 with 1024 over two CTAs, 100 unshared.
// With X X^T over 1, 2, 4 and 8 CTAs, what the rule takes in brackets:
// 1 x 512 x 2048 95.7, 87.6, 81.7, [82.7]; 1 x 256 x 4096 120.5, 94.7, 77.4, [70.5];
// 1 x 576 x 2112 103.3, 96.8, [87.4], 91.6; 1 x 960 x 3264 143.7, [135.8], 135.4,
// 157.5.
struct Choice {
  long long cost;         // 10 ns
  long long large, small; // tiles of each kind
  int split;              // small tiles: CTAs a tile; 0: SM pairs
};

template <int OP>
Choice choose(int n_mats, int K, int rowsP, int rowsQ) {
  constexpr bool SYM = OP == kGram || OP == kPoly;
  const long long n = n_mats, blocks = K / 64;
  const long long sms = num_sms() > 2 ? num_sms() : 2;  // 1 where no device answers
  Choice c{};
  c.large = n * Tiles<256, 256, SYM>(rowsP, rowsQ).count();
  c.small = n * Tiles<128, kSmallN, SYM>(rowsP, rowsQ).count();
  c.cost = (c.large + sms / 2 - 1) / (sms / 2) * blocks * 27 + 550;
  // only X X^T has a reduction long enough: over all sizes up to 65536 the rule
  // takes one CTA a tile for the other products
  const int most = OP == kGram ? kMaxSplit : 1;
  for (int k = 1; k <= most && k <= blocks; k *= 2) {
    const long long each = 125 + 17 * ((blocks + k - 1) / k);
    const long long tiles = c.small * k > sms ? c.small * k : sms;
    const long long cost = 125 + each * tiles / sms + (k > 1 ? 400 : 0);
    if (cost < c.cost) {
      c.cost = cost;
      c.split = k;
    }
  }
  return c;
}

template <int OP>
cudaError_t product(const OperandMaps& P, const OperandMaps& Q, const Product& p,
                    cudaStream_t s) {
  const Choice c = choose<OP>(p.n_mats, p.K, p.rowsP, p.rowsQ);
  return c.split ? launch_small<OP>(P, Q, p, c.small, c.split, s)
                 : launch_pairs<OP>(P, Q, p, c.large, s);
}

// Whether two steps at once take less time than one after the other, by a
// tenth at least (they are one launch more).
bool pair_steps(int n_mats, int mp, int np) {
  const long long gram = choose<kGram>(n_mats, np, mp, mp).cost;
  const long long square = choose<kPoly>(n_mats, mp, mp, mp).cost;
  const long long apply = choose<kApply>(n_mats, mp, mp, np).cost;
  return 11 * 5 * square < 10 * (gram + 2 * square + apply);
}

// Blocks of the norm's sum for each matrix: four an SM over the stack, 32 elements
// a thread at least.
int sum_blocks(size_t per_mat, int n_mats) {
  const size_t want = (per_mat + 16383) / 16384;
  const int share = (4 * num_sms() + n_mats - 1) / n_mats;
  const int most = share < kSumBlocks ? share : kSumBlocks;
  return want < (size_t)most ? (int)want : most;
}

// |G|, the scales and the first X.
template <typename T>
cudaError_t start(const moe_ortho_desc& D, const T* g, const OrthoLayout& L, float* partial,
                  Scale* scales, int* flags, __half* x, cudaStream_t s) {
  const size_t per_mat = (size_t)D.rows * D.cols;
  const int nb = sum_blocks(per_mat, D.n_mats);
  {
    ProfScope pr("ortho_sumsq", s);
    (void)launch_kernel(ortho_sumsq_kernel<T>, dim3(nb, D.n_mats), 512, 0, s, g, per_mat, partial,
                        flags);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const bool tall = D.rows > D.cols;
  const int rp = tall ? L.np : L.mp, cp = tall ? L.mp : L.np;
  ProfScope pr("ortho_start", s);
  const bool vec = D.cols % (16 / (int)sizeof(T)) == 0;
  auto kern = vec ? (tall ? ortho_start_kernel<T, true, true> : ortho_start_kernel<T, true, false>)
                  : (tall ? ortho_start_kernel<T, false, true>
                          : ortho_start_kernel<T, false, false>);
  (void)launch_kernel(kern, dim3(cp / 64, rp / 64, D.n_mats), 256, 0, s, g, D.rows, D.cols, rp,
                      cp, D.eps, partial, nb, scales, x);
  return cudaGetLastError();
}

}  // namespace

OrthoLayout ortho_layout(const moe_ortho_desc& D) {
  OrthoLayout L{};
  const size_t n = (size_t)D.n_mats;
  const int m = D.rows < D.cols ? D.rows : D.cols, c = D.rows < D.cols ? D.cols : D.rows;
  L.mp = (m + 63) / 64 * 64;
  L.np = (c + 63) / 64 * 64;
  if (ortho_fits_chip(D)) {
    L.total = 256;  // the flags
    return L;
  }
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) & ~(size_t)255;
    return o;
  };
  L.partial = take(n * kSumBlocks * 3 * sizeof(float));
  L.scales = take(n * sizeof(Scale));
  for (size_t& o : L.x) o = take(n * L.mp * L.np * 2);
  L.gram = take(n * L.mp * L.mp * 2);
  L.poly = take(n * L.mp * L.mp * 2);
  L.mul = take(n * L.mp * L.mp * 2);
  L.total = 512 + off;  // the flags' 16 bytes, then the regions at the next multiple of 256
  return L;
}

cudaError_t launch_orthogonalize(const moe_ortho_desc& D, const void* g, void* out, void* ws,
                                 cudaStream_t s) {
  const OrthoLayout L = ortho_layout(D);
  int* flags = static_cast<int*>(ws);
  if (ortho_fits_chip(D)) return launch_ortho_chip(D, g, out, flags, s);
  uint8_t* b = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ws) + 16 + 255) &
                                          ~(uintptr_t)255);
  const int m = D.rows < D.cols ? D.rows : D.cols, n = D.rows < D.cols ? D.cols : D.rows;
  float* partial = reinterpret_cast<float*>(b + L.partial);
  Scale* scales = reinterpret_cast<Scale*>(b + L.scales);
  __half* x[2] = {reinterpret_cast<__half*>(b + L.x[0]), reinterpret_cast<__half*>(b + L.x[1])};
  __half* gram = reinterpret_cast<__half*>(b + L.gram);
  __half* poly = reinterpret_cast<__half*>(b + L.poly);
  __half* mul = reinterpret_cast<__half*>(b + L.mul);
  cudaError_t e = D.dtype == MOE_BF16
                      ? start(D, static_cast<const __nv_bfloat16*>(g), L, partial, scales, flags,
                              x[0], s)
                      : start(D, static_cast<const float*>(g), L, partial, scales, flags, x[0],
                              s);
  if (e != cudaSuccess) return e;
  Product p{};
  p.n_mats = D.n_mats;
  p.m = m, p.n = n;
  p.scales = scales;
  p.err = flags;
  p.tall = D.rows > D.cols;
  p.result = static_cast<__nv_bfloat16*>(out);
  OperandMaps mx[2], mg, mb, mq;
  const long long rows = (long long)D.n_mats * L.mp;
  if (!make_maps(&mx[0], x[0], L.np, rows) || !make_maps(&mx[1], x[1], L.np, rows) ||
      !make_maps(&mg, gram, L.mp, rows) || !make_maps(&mb, poly, L.mp, rows) ||
      !make_maps(&mq, mul, L.mp, rows))
    return cudaErrorInvalidValue;
  // alpha P Q of m x m matrices
  auto square = [&](const OperandMaps& P, const OperandMaps& Q, __half* to, float alpha) {
    p.K = p.rowsP = p.rowsQ = L.mp;
    p.out = to, p.alpha = alpha;
    return product<kGram>(P, Q, p, s);
  };
  const bool pairs = pair_steps(D.n_mats, L.mp, L.np);
  int at = 0;  // which x holds X
  int done = 0;
  bool paired = false;
  for (int left = D.steps; left > 0;) {
    paired = pairs && !paired && left >= 2;
    p.ahead = paired ? 2 : 1;
    left -= p.ahead;
    p.steps = done;
    p.K = L.np, p.rowsP = p.rowsQ = L.mp;
    p.out = gram, p.alpha = kScaleA / (kScaleX * kScaleX);
    if ((e = product<kGram>(mx[at], mx[at], p, s)) != cudaSuccess) return e;
    p.steps = -1;
    p.K = L.mp;
    p.gram = gram, p.out = poly;
    if ((e = product<kPoly>(mg, mg, p, s)) != cudaSuccess) return e;
    if (paired) {
      if ((e = square(mb, mg, mul, kScaleM / (kScaleB * kScaleA))) != cudaSuccess ||  // B0 A
          (e = square(mq, mb, gram, kScaleA / (kScaleM * kScaleB))) != cudaSuccess)   // A1
        return e;
      p.out = mul;
      if ((e = product<kPoly>(mg, mg, p, s)) != cudaSuccess ||                        // B1
          (e = square(mq, mb, gram, kScaleQ / (kScaleB * kScaleB))) != cudaSuccess)   // B1 B0
        return e;
    }
    p.steps = done;
    p.K = p.rowsP = L.mp, p.rowsQ = L.np;
    p.out = x[at ^ 1];
    p.alpha = 1.f / (paired ? kScaleQ : kScaleB);
    const OperandMaps& by = paired ? mg : mb;
    if (left > 0) {
      e = product<kApply>(by, mx[at], p, s);
    } else {
      p.alpha /= kScaleX;
      e = product<kLast>(by, mx[at], p, s);
    }
    if (e != cudaSuccess) return e;
    at ^= 1;
    done += p.ahead;
  }
  return cudaSuccess;
}

}  // namespace moe
