// fp8_gemm.cu -- the expert FFN's grouped products with 8-bit operands (format:
// fp8.cuh) on the 5th-generation tensor cores ("Distributed MoE" (tenzro docs),
// expert-host-runtime and compute-seam paragraphs: SwiGLU experts, every
// projection Y = X * W^T with W stored [out, in]).
//
//   gate/up : h[r, n] = silu(g) u,  g = sum_b sx[r, b] sg[n / 128, b] <x8[r, b], Wg[n, b]>
//             (u likewise), then h's row into 8 bits, 128 columns a scale
//   down    : y[r, m] = slot_w[r] sum_b sh[r, b] sd[m / 128, b] <h8[r, b], Wd[m, b]>
// for every batch row r of expert e (rows offsets[e] .. offsets[e+1]); b runs over
// the blocks of 128 along the reduction: a block's products are summed over codes in
// fp32, then scaled and added in fp32.
//
// Design (sm_103a, one CTA an SM, persistent):
//   * A unit is (expert, 256 weight rows, up to 128 token rows): 128 rows of gate
//     and the same 128 of up, or 256 rows of down.  Token rows are the MMA's M
//     side (the lanes of TMEM), weight rows its N side.  A thread of the epilogue
//     then has one token row: that row's scale times the block's weight scale is
//     one factor for all its columns, a column block of h is one thread's (and its
//     partner's), and outputs are written along rows.
//   * A block of 128 along K is one 128-byte swizzled row per operand row: four
//     tcgen05.mma (kind::f8f6f4, K = 32, N = 256; 128 cycles each) into one of two
//     TMEM buffers of 256 columns.  The epilogue's warps add each block's products
//     into registers with their factors while the next block's MMAs fill the other
//     buffer.
//   * Warp 0 lane 0 issues TMA loads into a ring of stages, lane 0 of warps 1 and 2
//     the MMAs of even and odd blocks.  A block's products go to a buffer of their
//     own, so the two need no order, and one waits for its stage and buffer while
//     the other's MMAs run (one issuing thread left the tensor cores idle for 300 of
//     800 cycles a block).
//   * Warps 4-11 are the epilogue: two warps a TMEM lane quarter, each with half of
//     the columns (64 of gate and the same 64 of up, or 128 of down).  A thread holds
//     128 sums, so the registers are split unevenly (setmaxnreg).  Sixteen warps of
//     64 sums were slower (gate/up 217 -> 256 us), and so was waiting in a spin.
//   * Warp 3 turns scales into factors, row's times tile's, two for each of the 128
//     rows (gate's and up's, or those of down's two tiles), a block ahead: they lie in
//     shared memory before a block's products are announced, and cost the epilogue's
//     warps one load a block (formed there they took a tenth of the time).
//   * SM pairs (cta_group::2, 256 token rows, half of the weight rows to a CTA) were
//     built and dropped: the tensor cores do not wait for operands
//     (8192 tokens x 8, 4096 x 1536, 32 experts: 1.5 % faster; 600 rows an expert 14 %
//     slower, for its larger tiles).
//   * Every wait is bounded (tc_common.cuh); that for registers ends because the launcher
//     has checked that there are enough.
//
// What bounds it: with few rows an expert the weights' bytes (64 tokens, 65 experts of
// 7168 x 2048: 420 us for 2.86 GB, 6.8 TB/s; on another GB300 444 us).  With many rows a
// block takes 910 cycles in gate/up and 1310 in down, units' starts and ends included
// (tensor pipe 52 and 38 % active, 16384 rows).  Its MMAs take 512; reading its 128 x 256
// sums from TMEM takes 160 cycles, adding them 270 (350 without the packed instruction),
// both together 310 where nothing else runs, beside the next block's MMAs.  What fills
// the rest is not known; barriers, factors and a unit's end (SwiGLU: two special functions
// a value) are in it.
#include <cuda.h>
#include <cuda_bf16.h>

#include <mutex>

#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"
#include "tc_common.cuh"

namespace moe {
namespace {

using tc::MODE_DOWN;
using tc::MODE_GATEUP;
using tc::Unit;

constexpr int kEpiWarps = 8, kEpiWarp0 = 4;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
// Registers a thread: 384 threads are launched with 168 each; 4 warps give up what 8 take:
// 128 x 72 + 256 x 216 = 384 x 168.
constexpr int kRegsLaunch = 168, kRegsIssue = 72, kRegsEpi = 216;
static_assert(128 * kRegsIssue + 256 * kRegsEpi == kThreads * kRegsLaunch, "register split");
// Whether a launch with so many registers a thread (given out in steps of 8) covers the split.
// What the compiler took decides, and a warp that asks for more than the block has left
// waits without a limit: the launcher asks first.
constexpr bool covers_split(int regs) {
  const int given = (regs + 7) / 8 * 8;
  return given >= kRegsLaunch && given <= kRegsEpi;
}
static_assert(covers_split(kRegsLaunch) && !covers_split(kRegsLaunch - 8), "register split");
constexpr int kRows = 128;  // token rows of a unit
constexpr int kCols = 256;  // weight rows of a unit
constexpr int kBK = 128;    // bytes (= elements) along K of a stage

// Scales of a row lie pitch_of(n) apart, so that two blocks' are one 8-byte load.
__device__ __forceinline__ int pitch_of(int n) { return fp8_scale_pitch(n); }

struct F8Params {
  tc::Params b;       // offsets, groups, Mg, K, row_scale, err, max_rows
  const float* xs;    // [rows, pitch_of(K)] scales of the token rows
  const float* ws0;   // [groups, MB, KB] weight scales (gate, or down)
  const float* ws1;   // up
  uint8_t* hq;        // gate/up: h's codes [rows, Mg] and scales [rows, pitch_of(Mg)]
  float* hs;
  __nv_bfloat16* y;   // down: [rows, Mg]
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T, e4m3 inputs, fp32 accumulate, one CTA.
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// acc += {lo, hi} * f, two fp32 fused multiply-adds in one instruction (128 x 256 sums a
// block by 8 warps: 270 cycles, 350 one by one).  Volatile: the products of a load stay
// before the next load into the same registers, which would otherwise be copied.
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t f) {
  asm volatile(
      "{\n\t.reg .b64 v;\n\t"
      "mov.b64 v, {%1, %2};\n\t"
      "fma.rn.f32x2 %0, v, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(lo), "r"(hi), "l"(f));
}
__device__ __forceinline__ uint64_t pair_of(float f) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %1};" : "=l"(v) : "r"(__float_as_uint(f)));
  return v;
}
__device__ __forceinline__ float lo_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Instruction descriptor, kind::f8f6f4: e4m3 A and B (format 0, K-major), fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

template <int STAGES>
struct Cfg {
  static constexpr int A_BYTES = kRows * kBK;
  static constexpr int B_BYTES = kCols * kBK;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  // full, empty; TMEM buffers full, empty; four meetings of the warps of a quarter; wind-downs
  static constexpr int NBARS = 2 * STAGES + 4 + 4 + 2;
  static constexpr int BAR_OFF = STAGES * STAGE_BYTES;
  static constexpr int MISC_OFF = BAR_OFF + NBARS * 8;
  static constexpr int FAC_OFF = (MISC_OFF + 8 + 15) / 16 * 16;  // [2][128] pairs of factors
  static constexpr int TOP_OFF = FAC_OFF + 2 * kRows * 8;         // [2][2][128] row maxima
  static constexpr int PREFIX_OFF = TOP_OFF + 2 * 2 * kRows * 4;
  static constexpr int GSTART_OFF = PREFIX_OFF + 4 * (tc::kMaxGroups + 1);
  static constexpr int SMEM_TOTAL = GSTART_OFF + 4 * (tc::kMaxGroups + 1) + 1024;
  static_assert(SMEM_TOTAL <= 232448, "shared memory");
  // The issuers take alternate blocks.  With an even number of stages a stage is always the
  // same one's, which has seen every phase of its barrier; else one could find it two phases
  // behind and take the old parity for the one it waits for.
  static_assert(STAGES % 2 == 0, "a stage belongs to one MMA issuer");
};

template <int MODE, int STAGES>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_grouped_gemm(const __grid_constant__ CUtensorMap tmX,
                     const __grid_constant__ CUtensorMap tmXfull,
                     const __grid_constant__ CUtensorMap tmW0,
                     const __grid_constant__ CUtensorMap tmW1, const F8Params p) {
  using C = Cfg<STAGES>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::BAR_OFF;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  const uint32_t accf0 = bar0 + 8u * (2 * STAGES);
  const uint32_t acce0 = accf0 + 16;
  const uint32_t meet0 = acce0 + 16;
  const uint32_t drain_bar = meet0 + 32;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  float2* fac = reinterpret_cast<float2*>(smem + C::FAC_OFF);
  volatile uint32_t* top = reinterpret_cast<volatile uint32_t*>(smem + C::TOP_OFF);
  int* prefix = reinterpret_cast<int*>(smem + C::PREFIX_OFF);
  int* gstart = reinterpret_cast<int*>(smem + C::GSTART_OFF);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kUnitRows = MODE == MODE_GATEUP ? 128 : kCols;  // of one weight matrix
  const int m_tiles = (p.b.Mg + kUnitRows - 1) / kUnitRows;
  const int KB = (p.b.K + kBK - 1) / kBK;
  const int MB = fp8::blocks_of(p.b.Mg);
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf0 + 8u * b, 2);  // the products, the factors
      mbar_init(acce0 + 8u * b, kEpiWarps);
    }
    for (int q = 0; q < 4; ++q) mbar_init(meet0 + 8u * q, 2);
    for (int i = 0; i < 2; ++i) mbar_init(drain_bar + 8u * i, 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmXfull);
    tma_prefetch_desc(&tmW0);
    tma_prefetch_desc(&tmW1);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == 3) tc::build_schedule<MODE, kRows>(p.b, m_tiles, prefix, gstart);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = prefix[p.b.n_groups];
  auto unit = [&](int u) {
    return tc::decode_unit<MODE, kRows>(u, prefix, gstart, p.b.n_groups, m_tiles, KB, p.b);
  };

  if (warp < kEpiWarp0) {
    setmaxnreg_dec<kRegsIssue>();
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0, armed = 0, armed_parity = 0;
        // The unit's 256 weight rows: 128 of gate and of up, or of down twice.
        auto load_weights = [&](int s, const Unit& t, int kb) {
          const uint32_t sB = sbase + s * C::STAGE_BYTES + C::A_BYTES;
          const int row = t.g * p.b.Mg + t.mt * kUnitRows;
          tma_load_2d(sB, &tmW0, full_bar(s), kb * kBK, row);
          tma_load_2d(sB + C::B_BYTES / 2, &tmW1, full_bar(s), kb * kBK,
                      MODE == MODE_GATEUP ? row : row + 128);
        };
        auto arm = [&](int s, const Unit& t) {
          const int chunks = (t.nt + 31) / 32;
          mbar_arrive_expect_tx(full_bar(s), C::B_BYTES + chunks * 32 * kBK);
          armed |= 1u << s;
        };
        // The first unit's weight tiles are requested before waiting for the
        // predecessor grid: no kernel of the sequence writes weights, and the
        // schedule comes from a grid two launches back.
        int n_pre = 0;
        if ((int)blockIdx.x < total) {
          const Unit t = unit(blockIdx.x);
          n_pre = min(STAGES, KB);
          for (int i = 0; i < n_pre; ++i) {
            arm(i, t);
            load_weights(i, t, i);
          }
        }
        pdl_wait();
        bool first = true;
        for (int u = blockIdx.x; u < total && !*abort_flag; u += gridDim.x) {
          if (u + (int)gridDim.x >= total) pdl_trigger();  // this CTA's last unit
          const Unit t = unit(u);
          const int chunks = (t.nt + 31) / 32;
          bool ok = true;
          for (int kb = 0; kb < KB; ++kb) {
            if (!(first && kb < n_pre)) {
              if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.b.err)) {
                ok = false;
                break;
              }
              arm(stage, t);
              armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
              load_weights(stage, t, kb);
            }
            const uint32_t sA = sbase + stage * C::STAGE_BYTES;
            if (chunks == 4)
              tma_load_2d(sA, &tmXfull, full_bar(stage), kb * kBK, t.r0);
            else
              for (int c = 0; c < chunks; ++c)
                tma_load_2d(sA + c * 32 * kBK, &tmX, full_bar(stage), kb * kBK, t.r0 + c * 32);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          first = false;
          if (!ok) break;
        }
        if ((int)blockIdx.x >= total) pdl_trigger();
        // wind down: every copy this thread started has landed before exit
        for (int s = 0; s < STAGES; ++s)
          if (armed & (1u << s))
            tc::mbar_wait_drain(full_bar(s), (armed_parity >> s) & 1u, p.b.err);
      }
    } else if (warp <= 2) {
      // ---------------------------------------------------------- MMA issuers
      if (lane == 0) {
        constexpr uint32_t idesc = idesc_e4m3_f32(kRows, kCols);
        const uint32_t buf = warp - 1;  // even blocks of this CTA's sequence, or odd ones
        int stage = 0;
        uint32_t phase = 0, it = 0;
        bool issued = false, ok = true;
        for (int u = blockIdx.x; ok && u < total && !*abort_flag; u += gridDim.x) {
          for (int kb = 0; kb < KB; ++kb, ++it) {
            if ((it & 1u) == buf) {
              if (!mbar_wait(full_bar(stage), phase, abort_flag, p.b.err) ||
                  !mbar_wait(acce0 + 8u * buf, ((it >> 1) & 1u) ^ 1u, abort_flag, p.b.err)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t sA = sbase + stage * C::STAGE_BYTES;
              const uint32_t sB = sA + C::A_BYTES;
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const uint64_t a = smem_desc_sw128(sA + kk * 32);
                const uint64_t b = smem_desc_sw128(sB + kk * 32);
                umma_e4m3(tmem_base + buf * kCols, a, b, idesc, kk != 0);
              }
              issued = true;
              umma_commit(accf0 + 8u * buf);
              umma_commit(empty_bar(stage));
            }
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        // wind down: every MMA this thread issued has completed before TMEM is freed
        if (issued) {
          umma_commit(drain_bar + 8u * buf);
          tc::mbar_wait_drain(drain_bar + 8u * buf, 0, p.b.err);
        }
      }
    } else {
      // ---------------------------------------------------------- factors (warp 3)
      pdl_wait();  // the token rows' scales are the predecessor's
      const int pitch = pitch_of(p.b.K);
      uint32_t it = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
        const Unit t = unit(u);
        const int mine = t.nt;
        const size_t row0 = (size_t)t.r0 * pitch;
        // the tiles of gate and up, or of down's first and second 128 rows
        const size_t w0 = ((size_t)t.g * MB + (MODE == MODE_GATEUP ? t.mt : 2 * t.mt)) * KB;
        const size_t w1 =
            MODE == MODE_GATEUP ? w0 : ((size_t)t.g * MB + min(2 * t.mt + 1, MB - 1)) * KB;
        float2 x[4], nx[4];  // two blocks' scales of rows lane, lane + 32, ...; the next two's
        float s0 = 0.f, s1 = 0.f, n0 = 0.f, n1 = 0.f;  // 32 blocks' across the lanes; the next's
        auto ask_rows = [&](int kb) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (lane + 32 * i < mine)
              nx[i] = *reinterpret_cast<const float2*>(p.xs + row0 +
                                                       (size_t)(lane + 32 * i) * pitch + kb);
        };
        auto ask_tiles = [&](int kb) {
          if (kb + lane < KB) {
            n0 = p.ws0[w0 + kb + lane];
            n1 = p.ws1[w1 + kb + lane];
          }
        };
        ask_rows(0);
        ask_tiles(0);
        for (int kb = 0; kb < KB; ++kb, ++it) {
          const uint32_t buf = it & 1u;
          if ((kb & 1) == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = nx[i];
            if (kb + 2 < KB) ask_rows(kb + 2);
          }
          if ((kb & 31) == 0) {
            s0 = n0, s1 = n1;
            ask_tiles(kb + 32);
          }
          const float a = __shfl_sync(0xffffffffu, s0, kb & 31);
          const float b = __shfl_sync(0xffffffffu, s1, kb & 31);
          // free once the epilogue has let go of the block before the last
          if (!tc::mbar_wait_warp(acce0 + 8u * buf, ((it >> 1) & 1u) ^ 1u, abort_flag, p.b.err)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float s = (kb & 1) ? x[i].y : x[i].x;
            if (lane + 32 * i < mine) fac[buf * kRows + lane + 32 * i] = make_float2(s * a, s * b);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(accf0 + 8u * buf);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 4..11)
    setmaxnreg_inc<kRegsEpi>();
    pdl_wait();  // what is written here the predecessor may still read
    const int q = warp & 3;                    // TMEM lane quarter this warp may access
    const int half = (warp - kEpiWarp0) >> 2;  // its half of the columns
    const int lrow = q * 32 + lane;
    uint32_t it = 0, met = 0;
    bool ok = true;
    float slot_w = 1.0f;
    for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
      const Unit t = unit(u);
      const int mine = t.nt, tile = t.mt;
      const bool warp_live = q * 32 < mine, live = lrow < mine;
      const int out_row = t.r0 + (live ? lrow : 0);
      if (MODE == MODE_DOWN && p.b.row_scale && live) slot_w = p.b.row_scale[out_row];
      uint64_t sum[64];  // this thread's 128 columns, two a register pair
#pragma unroll
      for (int i = 0; i < 64; ++i) sum[i] = 0;
      auto release = [&](uint32_t buf) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acce0 + 8u * buf);
      };
      auto ready = [&]() {
        uint32_t r;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(r)
            : "r"(accf0 + 8u * (it & 1u)), "r"((it >> 1) & 1u)
            : "memory");
        return __all_sync(0xffffffffu, r);
      };
      auto wait = [&]() {
        const bool there = tc::mbar_wait_warp(accf0 + 8u * (it & 1u), (it >> 1) & 1u, abort_flag,
                                              p.b.err);
        if (there) tc_fence_after();
        return there;
      };
      if (!warp_live) {
        for (int kb = 0; kb < KB && (ok = wait()); ++kb, ++it) release(it & 1u);
      } else if ((ok = wait())) {
        // gate's 64 columns then up's, or down's 128: 32 at a time, the next 32 loaded
        // while these are added, also across blocks
        const uint32_t tq = tmem_base + ((uint32_t)(q * 32) << 16) +
                            (MODE == MODE_GATEUP ? half * 64 : half * 128);
        constexpr uint32_t kSecond = MODE == MODE_GATEUP ? 128 : 64;
        auto add = [&](int c, const uint32_t (&v)[32], float f) {
          const uint64_t ff = pair_of(f);
#pragma unroll
          for (int i = 0; i < 16; ++i) fma2(sum[c * 16 + i], v[2 * i], v[2 * i + 1], ff);
        };
        uint32_t va[32], vb[32];
        tmem_ld32(tq + (it & 1u) * kCols, va);
        float2 f = fac[(it & 1u) * kRows + lrow];
// 1, 2, 4 blocks a turn: gate/up 686, 672, 638 us (8192 x 8 rows, 4096 x 1536, 32
// experts), down 454, 429, 432; a short call (777 tokens) 70, 70, 75 us: more code to fetch
#pragma unroll 2
        for (int kb = 0; kb < KB; ++kb) {
          const uint32_t buf = it & 1u, tb = tq + buf * kCols;
          const float f0 = MODE == MODE_GATEUP || half == 0 ? f.x : f.y;
          const float f1 = MODE == MODE_GATEUP || half == 1 ? f.y : f.x;
          tmem_ld_wait();
          tmem_ld32(tb + 32, vb);
          add(0, va, f0);
          tmem_ld_wait();
          tmem_ld32(tb + kSecond, va);
          add(1, vb, f0);
          tmem_ld_wait();
          tmem_ld32(tb + kSecond + 32, vb);
          add(2, va, f1);
          tmem_ld_wait();
          release(buf);  // everything is in registers: the next MMAs may have the buffer
          ++it;
          if (kb + 1 < KB && !ready()) {  // nothing to load yet: add first
            add(3, vb, f1);
            if (!(ok = wait())) break;
            tmem_ld32(tq + (it & 1u) * kCols, va);
            f = fac[(it & 1u) * kRows + lrow];
          } else {
            if (kb + 1 < KB) {
              tc_fence_after();
              tmem_ld32(tq + (it & 1u) * kCols, va);
              f = fac[(it & 1u) * kRows + lrow];
            }
            add(3, vb, f1);
          }
        }
      }
      if (!ok) break;
      if constexpr (MODE == MODE_GATEUP) {
        // columns of h: tile * 128 + half * 64 .. + 63 (Mg is a multiple of 64)
        const int c0 = tile * 128 + half * 64;
        const bool cols = c0 < p.b.Mg;
        uint32_t m = 0;
        float acc[64];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          acc[2 * i] = silu_fast(lo_of(sum[i])) * lo_of(sum[32 + i]);
          acc[2 * i + 1] = silu_fast(hi_of(sum[i])) * hi_of(sum[32 + i]);
          m = max(m, max(fp8::abs_bits(acc[2 * i]), fp8::abs_bits(acc[2 * i + 1])));
        }
        if (!cols) m = 0;
        if (warp_live) {
          // the other half's largest, through shared memory.  Two sets of maxima in
          // turn: a set is written again only after a meeting that its reader came to.
          volatile uint32_t* mine = top + ((met & 1) * 2 + half) * kRows + lrow;
          *mine = m;
          __syncwarp();
          if (lane == 0) mbar_arrive(meet0 + 8u * q);
          if (!tc::mbar_wait_warp(meet0 + 8u * q, met & 1u, abort_flag, p.b.err)) break;
          m = max(m, top[((met & 1) * 2 + (half ^ 1)) * kRows + lrow]);
          ++met;
          const fp8::Scale sc = fp8::scale_of(m);
          if (live && cols) {
            uint4* dst = reinterpret_cast<uint4*>(p.hq + (size_t)out_row * p.b.Mg + c0);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float* a = acc + i * 16 + j * 4;
                w[j] = fp8::codes4(a[0] * sc.inv, a[1] * sc.inv, a[2] * sc.inv, a[3] * sc.inv);
              }
              dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (half == 0) p.hs[(size_t)out_row * pitch_of(p.b.Mg) + tile] = sc.scale;
          }
        }
      } else {
        if (live) {
          const int c0 = tile * 256 + half * 128, cols = min(p.b.Mg - c0, 128);  // 0 or less: none
          __nv_bfloat16* dst = p.y + (size_t)out_row * p.b.Mg + c0;
          const bool wide = (reinterpret_cast<uintptr_t>(p.y) & 31u) == 0;  // rows are: d % 64 == 0
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint64_t a = sum[i * 8 + j];
              const __nv_bfloat162 h = __floats2bfloat162_rn(lo_of(a) * slot_w, hi_of(a) * slot_w);
              w[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            if (16 * i < cols) {  // Mg is a multiple of 64
              if (wide) {
                st_global_v8(dst + 16 * i, w);
              } else {
                reinterpret_cast<uint4*>(dst)[2 * i] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4*>(dst)[2 * i + 1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// e4m3 matrix [rows, inner] (row-major), boxes of box_rows x 128, 128-byte swizzle;
// columns and rows beyond it are read as zero
bool make_tmap_f8(CUtensorMap* tm, const void* base, uint64_t inner, uint64_t rows,
                  uint32_t box_rows) {
  return make_tmap_2d(tm, base, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, inner, rows, kBK, box_rows,
                      CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int MODE, int STAGES>
cudaError_t launch_f8(const CUtensorMap& x, const CUtensorMap& xfull, const CUtensorMap& w0,
                      const CUtensorMap& w1, const F8Params& p, long long max_units,
                      const char* name, cudaStream_t s) {
  using C = Cfg<STAGES>;
  auto kern = fp8_grouped_gemm<MODE, STAGES>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  static std::mutex mu;
  static bool configured[64] = {};
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev]) {
      cudaFuncAttributes attr;
      if ((e = cudaFuncGetAttributes(&attr, kern)) != cudaSuccess) return e;
      if (!covers_split(attr.numRegs)) return cudaErrorInvalidConfiguration;
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_TOTAL);
      if (e != cudaSuccess) return e;
      configured[dev] = true;
    }
  }
  const long long grid = max_units < num_sms() ? max_units : num_sms();
  if (grid <= 0) return cudaSuccess;
  ProfScope pr(name, s);
  (void)launch_kernel(kern, (unsigned)grid, kThreads, C::SMEM_TOTAL, s, x, xfull, w0, w1, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ffn_fp8(const void* x8, const float* xs, const int32_t* offsets, int n_groups,
                           int P, int d, int I, const Fp8Weight& Wg, const Fp8Weight& Wu,
                           const Fp8Weight& Wd, const float* slot_w, void* h8, float* hs,
                           void* y_perm, int* err, cudaStream_t s) {
  if (P == 0) return cudaSuccess;
  const uint64_t cap = (uint64_t)tc_row_capacity(P);
  CUtensorMap tx, txf, th, thf, tg, tu, td;
  if (!make_tmap_f8(&tx, x8, d, cap, 32) || !make_tmap_f8(&txf, x8, d, cap, 128) ||
      !make_tmap_f8(&th, h8, I, cap, 32) || !make_tmap_f8(&thf, h8, I, cap, 128) ||
      !make_tmap_f8(&tg, Wg.q, d, (uint64_t)n_groups * I, 128) ||
      !make_tmap_f8(&tu, Wu.q, d, (uint64_t)n_groups * I, 128) ||
      !make_tmap_f8(&td, Wd.q, I, (uint64_t)n_groups * d, 128))
    return cudaErrorInvalidValue;
  F8Params p1{}, p2{};
  p1.b.offsets = p2.b.offsets = offsets;
  p1.b.n_groups = p2.b.n_groups = n_groups;
  p1.b.max_rows = p2.b.max_rows = P;
  p1.b.err = p2.b.err = err;
  p1.b.Mg = I, p1.b.K = d;
  p1.xs = xs, p1.ws0 = Wg.scale, p1.ws1 = Wu.scale;
  p1.hq = static_cast<uint8_t*>(h8), p1.hs = hs;
  p2.b.Mg = d, p2.b.K = I;
  p2.b.row_scale = slot_w;
  p2.xs = hs, p2.ws0 = p2.ws1 = Wd.scale;
  p2.y = static_cast<__nv_bfloat16*>(y_perm);
  const long long tiles = (long long)(P + kRows - 1) / kRows + n_groups;
  const cudaError_t e = launch_f8<MODE_GATEUP, 4>(tx, txf, tg, tu, p1, (I + 127) / 128 * tiles,
                                                  "ffn_gateup_fp8", s);
  if (e != cudaSuccess) return e;
  return launch_f8<MODE_DOWN, 4>(th, thf, td, td, p2, (d + 255) / 256 * tiles, "ffn_down_fp8", s);
}

}  // namespace moe
