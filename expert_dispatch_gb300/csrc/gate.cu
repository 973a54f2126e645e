// gate.cu -- from router logits: the gate weights of given slots, the per-expert
// counts and the balance loss, and the gradient of both with respect to the
// logits ("Distributed MoE" (tenzro docs), router-families paragraph, for the two
// gating families; the loss is what training adds).
//
//   p       softmax(l), or s / sum(s) with s = sigmoid(l), per token
//   counts  c_e = pairs (t, j) whose id is e;  n = tokens with any id in [0, E)
//   prob_e  = sum of p_e over those n tokens / n
//   loss    = E / (k n) * <c, prob>      (1 where tokens and probability are even)
//   dl      = dloss * E / (k n^2) * p (c - <c, p>)   (sigmoid: times 1 - s)
//             + the gate weights' part (gate_backward_kernel)
// The counts are whole numbers and take no gradient.  Everything is fp32, sums
// in a fixed order (integers by atomics, whose order is of no matter).
//
// One warp a token, expert e on lane e % 32: a token's logits are read once, the
// next token's while these are worked on, and all sums over experts are warp
// butterflies.  By its bytes a pass is short (16384 x 256 fp32: 2.5 us forward, 5 us
// backward at the copy's rate; 11.8 and 12.2 us on the GPU); what is left is latency: the
// load, three butterflies and the exponentials of a token one after the other, and for
// the forward pass the joining of the blocks' sums, a launch of its own where there are
// several blocks.
#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

// Forward: warps a block, all that registers allow (one block an SM: few blocks' sums are
// left to join).
__host__ __device__ constexpr int warps_of(int PL) { return PL <= 8 ? 32 : 16; }
constexpr int kBackWarps = 8;
// Forward by one block and one launch up to so many tokens a warp: the joining launch is 2.4 us
// of the host's time and of the GPU's, a token of a warp about 2.5 us (64 x 384 by one block,
// four a warp, 11.3 us, by several 6.9 us).
constexpr int kOneBlockTokens = 2;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
// The fast division is off by 2 steps at most, and 0 where the divisor is above 2^126: the
// sigmoid left out there is below 2^-126.
__device__ __forceinline__ float sigmoid(float l) { return __fdividef(1.0f, 1.0f + expf(-l)); }

// s = sigmoid(l) and 1 - s for its slope s (1 - s).  With e = exp(-|l|) they are 1 / (1 + e)
// and e / (1 + e), whichever is which: neither is a difference, so 1 - s keeps its digits where
// s is next to 1 (subtracted it was 1 % off at l = 12 and nothing from 17 on).
struct Sigmoid {
  float s, rest;
};
__device__ __forceinline__ Sigmoid sigmoid_and_rest(float l) {
  const float e = expf(-fabsf(l));
  const float large = __fdividef(1.0f, 1.0f + e), small = e * large;
  return l < 0.f ? Sigmoid{small, large} : Sigmoid{large, small};
}

// Below this logit a sigmoid is exp(l) to 26 digits; where all logits of a sum
// lie below it the sum is formed of exp(l - max), which does not underflow.
constexpr float kSmallLogit = -60.f;

// A token's probabilities: pr[i] of expert lane + 32 i (softmax, or sigmoid over
// the sum of sigmoids); rest[i] = 1 - the sigmoid (SIGMOID and REST only).
// l[i] = -inf past E.
struct Softmax {
  float max, inv;  // of the softmax: p = exp(l - max) * inv
};
template <int PL, bool SIGMOID, bool REST>
__device__ __forceinline__ Softmax probabilities(const float (&l)[PL], float (&pr)[PL],
                                                 float (&rest)[PL]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < PL; ++i) m = fmaxf(m, l[i]);
  m = warp_max(m);
  float z = 0.f;
  const bool shift = !SIGMOID || m < kSmallLogit;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    float sg = 0.f;
    if (SIGMOID && REST) {
      const Sigmoid f = sigmoid_and_rest(l[i]);
      sg = f.s, rest[i] = f.rest;
    } else if (SIGMOID) {
      sg = sigmoid(l[i]);
    }
    pr[i] = shift ? expf(l[i] - m) : sg;
    z += pr[i];
  }
  const float inv = 1.0f / warp_sum(z);
#pragma unroll
  for (int i = 0; i < PL; ++i) pr[i] = pr[i] * inv;
  return {m, inv};
}

// Lane j < k holds slot j: its expert (-1: none) and that expert's logit.
struct Slot {
  int id;
  float logit;
};
template <typename T>
__device__ __forceinline__ Slot load_slot(const T* __restrict__ row,
                                          const int32_t* __restrict__ ids, size_t t, int E, int k,
                                          int lane) {
  Slot s{-1, -INFINITY};
  if (lane < k) {
    const int id = ids[t * k + lane];
    if (id >= 0 && id < E) {
      s.id = id;
      s.logit = load_as_f32(row, id);
    }
  }
  return s;
}

// Slot weights over the selection, q_j = score_j / sum of the slots' scores
// (exp(l - max) for softmax: the normaliser over all experts cancels).
template <bool SIGMOID>
__device__ __forceinline__ float normalised(const Slot& s) {
  const float m = warp_max(s.logit);
  const bool shift = !SIGMOID || m < kSmallLogit;
  float v = 0.f;
  if (s.id >= 0) v = shift ? expf(s.logit - m) : sigmoid(s.logit);
  return v / warp_sum(v);
}

// A token of the warp's sequence (forward: loaded before the one ahead of it is worked on;
// backward, where eight blocks an SM hide the loads, that cost 13.8 -> 16.5 us).
template <int PL, typename T>
struct Token {
  float l[PL];
  Slot s;
  __device__ __forceinline__ void load(const T* __restrict__ logits,
                                       const int32_t* __restrict__ ids, long long t, long long n,
                                       int E, int k, int lane) {
    if (t >= n) return;
    const T* row = logits + (size_t)t * E;
    s = load_slot(row, ids, (size_t)t, E, k, lane);
#pragma unroll
    for (int i = 0; i < PL; ++i)
      l[i] = lane + 32 * i < E ? load_as_f32(row, lane + 32 * i) : -INFINITY;
  }
};

// Blocks' sums: part_p [blocks][E], part_c [blocks][E + 1] (counts, tokens); or, for a
// single block with a thread for every expert, the results.
template <int PL, bool SIGMOID, bool NORM, typename T>
__global__ void __launch_bounds__(32 * warps_of(PL))
    gate_forward_kernel(const T* __restrict__ logits, const int32_t* __restrict__ ids, int T_,
                        int E, int k, float rs, float* __restrict__ w, float* __restrict__ part_p,
                        int32_t* __restrict__ part_c, int32_t* __restrict__ counts,
                        float* __restrict__ prob, float* __restrict__ loss,
                        unsigned* __restrict__ ticket) {
  pdl_wait();
  pdl_trigger();
  constexpr int kWarps = warps_of(PL), kThreads = 32 * kWarps;
  extern __shared__ float sum_s[];  // [kWarps][32 * PL]
  __shared__ int32_t count_s[32 * PL + 1];
  __shared__ float dot_s[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e <= E; e += kThreads) count_s[e] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *ticket = 0;  // of the launch that follows
  __syncthreads();
  float sum[PL] = {};
  int tokens = 0;
  const long long step = (long long)gridDim.x * kWarps;
  long long t = (long long)blockIdx.x * kWarps + warp;
  Token<PL, T> next;
  next.load(logits, ids, t, T_, E, k, lane);
  for (; t < T_; t += step) {
    const Token<PL, T> now = next;
    next.load(logits, ids, t + step, T_, E, k, lane);
    const Slot s = now.s;
    float v = 0.f;
    if (__any_sync(0xffffffffu, s.id >= 0)) {
      float pr[PL], rest[PL];
      const Softmax f = probabilities<PL, SIGMOID, false>(now.l, pr, rest);
#pragma unroll
      for (int i = 0; i < PL; ++i) sum[i] += pr[i];
      ++tokens;
      if (s.id >= 0) atomicAdd(&count_s[s.id], 1);
      if (w) {
        if (NORM)
          v = normalised<SIGMOID>(s);
        else
          v = SIGMOID ? sigmoid(s.logit) : expf(s.logit - f.max) * f.inv;
      }
    }
    if (w && lane < k) w[(size_t)t * k + lane] = s.id >= 0 ? rs * v : 0.f;
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) sum_s[warp * 32 * PL + lane + 32 * i] = sum[i];
  if (lane == 0) atomicAdd(&count_s[E], tokens);
  __syncthreads();
  auto block_sum = [&](int e) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) v += sum_s[i * 32 * PL + e];
    return v;
  };
  if (gridDim.x == 1 && E <= kThreads) {
    const int e = threadIdx.x, n = count_s[E];
    const float p = n > 0 && e < E ? block_sum(e) / (float)n : 0.f;
    if (e < E) {
      if (counts) counts[e] = count_s[e];
      if (prob) prob[e] = p;
    }
    if (counts && e == 0) counts[E] = n;
    const float dot = warp_sum(e < E ? (float)count_s[e] * p : 0.f);
    if (lane == 0) dot_s[warp] = dot;
    __syncthreads();
    if (warp == 0 && loss) {
      const float v = warp_sum(lane < kWarps ? dot_s[lane] : 0.f);
      if (lane == 0) *loss = n > 0 ? v * ((float)E / ((float)k * (float)n)) : 0.f;
    }
    return;
  }
  for (int e = threadIdx.x; e <= E; e += kThreads) {
    part_c[(size_t)blockIdx.x * (E + 1) + e] = count_s[e];
    if (e < E) part_p[(size_t)blockIdx.x * E + e] = block_sum(e);
  }
}

// The blocks' sums together.  32 experts a block, 32 threads an expert, so that all loads
// are under way at once; sums in a fixed order.  The block that comes last (by a ticket
// that the launch before has set to 0) adds up the loss.
__global__ void __launch_bounds__(1024) gate_finish_kernel(
    const float* __restrict__ part_p, const int32_t* __restrict__ part_c, int blocks, int E, int k,
    int32_t* __restrict__ counts, float* __restrict__ prob, float* __restrict__ loss,
    volatile float* __restrict__ dots, unsigned* __restrict__ ticket) {
  pdl_wait();
  pdl_trigger();
  __shared__ float p_s[32][33];
  __shared__ int c_s[32][33];
  __shared__ int n_s;
  const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  int c = 0;
  float p = 0.f;
  if (e < E) {
#pragma unroll 8
    for (int b = share; b < blocks; b += 32) {
      c += part_c[(size_t)b * (E + 1) + e];
      p += part_p[(size_t)b * E + e];
    }
  }
  p_s[share][lane] = p;
  c_s[share][lane] = c;
  if (share == 31) {
    int n = 0;
    for (int b = lane; b < blocks; b += 32) n += part_c[(size_t)b * (E + 1) + E];
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) n_s = n;
  }
  __syncthreads();
  if (share != 0) return;
  const int n = n_s;
  for (int i = 1; i < 32; ++i) {
    p += p_s[i][lane];
    c += c_s[i][lane];
  }
  p = n > 0 ? p / (float)n : 0.f;
  if (e < E) {
    if (counts) counts[e] = c;
    if (prob) prob[e] = p;
  }
  if (counts && e == 0) counts[E] = n;
  const float dot = warp_sum(e < E ? (float)c * p : 0.f);
  unsigned nth = 0;
  if (lane == 0) {
    dots[blockIdx.x] = dot;
    __threadfence();
    nth = atomicAdd(ticket, 1u);
  }
  nth = __shfl_sync(0xffffffffu, nth, 0);
  if (nth != gridDim.x - 1 || !loss) return;
  __threadfence();
  const float v = warp_sum(lane < (int)gridDim.x ? dots[lane] : 0.f);
  if (lane == 0) *loss = n > 0 ? v * ((float)E / ((float)k * (float)n)) : 0.f;
}

template <int PL, bool SIGMOID, bool NORM, typename T>
__global__ void __launch_bounds__(32 * kBackWarps)
    gate_backward_kernel(const T* __restrict__ logits, const int32_t* __restrict__ ids,
                         const int32_t* __restrict__ counts, const float* __restrict__ dw,
                         const float* __restrict__ dloss, int T_, int E, int k, float rs,
                         T* __restrict__ dlogits) {
  pdl_wait();
  pdl_trigger();
  __shared__ float add_s[kBackWarps][32 * PL];  // the selected experts' part, per warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long step = (long long)gridDim.x * kBackWarps;
  long long t = (long long)blockIdx.x * kBackWarps + warp;
  float a = 0.f;  // dloss * E / (k n^2)
  float c[PL];
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    c[i] = dloss && lane + 32 * i < E ? (float)counts[lane + 32 * i] : 0.f;
    add_s[warp][lane + 32 * i] = 0.f;
  }
  if (dloss && counts[E] > 0) {
    const float n = (float)counts[E];
    a = *dloss * ((float)E / ((float)k * n)) / n;
  }
  __syncwarp();
  for (; t < T_; t += step) {
    Token<PL, T> now;
    now.load(logits, ids, t, T_, E, k, lane);
    const Slot s = now.s;
    const float g = dw && s.id >= 0 ? rs * dw[(size_t)t * k + lane] : 0.f;
    T* out = dlogits + (size_t)t * E;
    if (!__any_sync(0xffffffffu, s.id >= 0)) {
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (lane + 32 * i < E) out[lane + 32 * i] = (T)0.f;
      continue;
    }
    float pr[PL], rest[PL];
    const Softmax f = probabilities<PL, SIGMOID, true>(now.l, pr, rest);
    float mean = 0.f;  // <c, p>
#pragma unroll
    for (int i = 0; i < PL; ++i) mean += c[i] * pr[i];
    mean = warp_sum(mean);
    float pull = 0.f;  // softmax weights: the part -<g, p> p of every expert
    if (dw) {
      float v = 0.f;  // slot j's own part, on lane j
      if (NORM) {
        const float q = normalised<SIGMOID>(s);
        const float dot = warp_sum(s.id >= 0 ? g * q : 0.f);
        v = q * (g - dot);
        if (SIGMOID) v *= sigmoid_and_rest(s.logit).rest;
      } else if (SIGMOID) {
        const Sigmoid sj = sigmoid_and_rest(s.logit);
        v = g * sj.s * sj.rest;
      } else {
        v = g;  // times p_e, known on the expert's lane
        pull = warp_sum(s.id >= 0 ? g * (expf(s.logit - f.max) * f.inv) : 0.f);
      }
      // an id may come twice: then its slots are added in their order
      const unsigned same = __match_any_sync(0xffffffffu, s.id);
      if (__any_sync(0xffffffffu, s.id >= 0 && (same & (same - 1u)) != 0)) {
        for (int j = 0; j < k; ++j) {
          const int id = __shfl_sync(0xffffffffu, s.id, j);
          const float vj = __shfl_sync(0xffffffffu, v, j);
          if (id >= 0 && (id & 31) == lane) add_s[warp][id] += vj;
        }
      } else if (s.id >= 0) {
        add_s[warp][s.id] = v;
      }
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      float v = a * pr[i] * (c[i] - mean);
      if (SIGMOID) v *= rest[i];
      if (dw) {
        const float add = add_s[warp][lane + 32 * i];
        v += !NORM && !SIGMOID ? pr[i] * (add - pull) : add;
      }
      if (lane + 32 * i < E) out[lane + 32 * i] = (T)v;
    }
    if (dw) {
      __syncwarp();
      if (s.id >= 0) add_s[warp][s.id] = 0.f;
      __syncwarp();
    }
  }
}

template <int PL, bool SIGMOID, bool NORM, typename T>
struct Kernels {
  static void forward(const void* logits, const int32_t* ids, const moe_layer_desc& D, float* w,
                      float* part_p, int32_t* part_c, int32_t* counts, float* prob, float* loss,
                      unsigned* ticket, int blocks, cudaStream_t s) {
    constexpr int smem = warps_of(PL) * 32 * PL * 4;
    if (smem > 48 * 1024 - 8192 &&
        cudaFuncSetAttribute(gate_forward_kernel<PL, SIGMOID, NORM, T>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return;
    (void)launch_kernel(gate_forward_kernel<PL, SIGMOID, NORM, T>, blocks, 32 * warps_of(PL), smem,
                        s, static_cast<const T*>(logits), ids, D.T, D.E, D.k, D.routed_scaling, w,
                        part_p, part_c, counts, prob, loss, ticket);
  }
  static void backward(const void* logits, const int32_t* ids, const moe_layer_desc& D,
                       const int32_t* counts, const float* dw, const float* dloss, void* dlogits,
                       int blocks, cudaStream_t s) {
    (void)launch_kernel(gate_backward_kernel<PL, SIGMOID, NORM, T>, blocks, 32 * kBackWarps, 0, s,
                        static_cast<const T*>(logits), ids, counts, dw, dloss, D.T, D.E, D.k,
                        D.routed_scaling, static_cast<T*>(dlogits));
  }
};

int per_lane(int E) { return E <= 64 ? 2 : E <= 128 ? 4 : E <= 256 ? 8 : E <= 512 ? 16 : 32; }

// f(Kernels<...>) of the layer's experts a lane, gating and logits' type
template <typename F>
void choose(const moe_layer_desc& D, int dtype, const F& f) {
  auto by_type = [&](auto pl, auto sig, auto norm) {
    constexpr int PL = decltype(pl)::value;
    constexpr bool S = decltype(sig)::value, N = decltype(norm)::value;
    if (dtype == MOE_BF16)
      f(Kernels<PL, S, N, __nv_bfloat16>{});
    else
      f(Kernels<PL, S, N, float>{});
  };
  auto by_gate = [&](auto pl) {
    using Y = std::true_type;
    using No = std::false_type;
    if (D.gate == MOE_GATE_SIGMOID_BIAS)
      D.norm_topk ? by_type(pl, Y{}, Y{}) : by_type(pl, Y{}, No{});
    else
      D.norm_topk ? by_type(pl, No{}, Y{}) : by_type(pl, No{}, No{});
  };
  switch (per_lane(D.E)) {
    case 2: return by_gate(std::integral_constant<int, 2>{});
    case 4: return by_gate(std::integral_constant<int, 4>{});
    case 8: return by_gate(std::integral_constant<int, 8>{});
    case 16: return by_gate(std::integral_constant<int, 16>{});
    default: return by_gate(std::integral_constant<int, 32>{});
  }
}

// Forward blocks.  Goes by no device: the workspace's size goes by it.
int grid_of(const moe_layer_desc& D) {
  const int warps = warps_of(per_lane(D.E));
  if (D.T > 0 && D.T <= kOneBlockTokens * warps) return 1;
  const int need = (D.T + warps - 1) / warps;
  return need < 152 ? need : 152;
}

// One block that has a thread for every expert gives the results itself.
bool one_launch(const moe_layer_desc& D) {
  return grid_of(D) == 1 && D.E <= 32 * warps_of(per_lane(D.E));
}

}  // namespace

size_t gate_workspace_bytes(const moe_layer_desc& D) {
  // the blocks' sums, 32 parts of the loss and the ticket
  return D.T == 0 ? 0 : ((size_t)grid_of(D) * (2 * (size_t)D.E + 1) + 33) * 4;
}

cudaError_t launch_gate_forward(const moe_layer_desc& D, int dtype, const void* logits,
                                const int32_t* ids, float* w, int32_t* counts, float* prob,
                                float* loss, void* ws, cudaStream_t s) {
  const int blocks = grid_of(D);
  float* part_p = static_cast<float*>(ws);
  int32_t* part_c = reinterpret_cast<int32_t*>(part_p + (size_t)blocks * D.E);
  float* dots = reinterpret_cast<float*>(part_c + (size_t)blocks * (D.E + 1));
  unsigned* ticket = reinterpret_cast<unsigned*>(dots + 32);
  {
    ProfScope pr("gate_forward", s);
    choose(D, dtype, [&](auto kernels) {
      decltype(kernels)::forward(logits, ids, D, w, part_p, part_c, counts, prob, loss, ticket,
                                 blocks, s);
    });
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (one_launch(D) || (!counts && !prob && !loss)) return cudaSuccess;
  ProfScope pr("gate_finish", s);
  (void)launch_kernel(gate_finish_kernel, (D.E + 31) / 32, 1024, 0, s, (const float*)part_p,
                      (const int32_t*)part_c, blocks, D.E, D.k, counts, prob, loss, dots, ticket);
  return cudaGetLastError();
}

cudaError_t launch_gate_backward(const moe_layer_desc& D, int dtype, const void* logits,
                                 const int32_t* ids, const int32_t* counts, const float* dw,
                                 const float* dloss, void* dlogits, cudaStream_t s) {
  const int need = (D.T + kBackWarps - 1) / kBackWarps, most = num_sms() * 8;
  ProfScope pr("gate_backward", s);
  choose(D, dtype, [&](auto kernels) {
    decltype(kernels)::backward(logits, ids, D, counts, dw, dloss, dlogits,
                                need < most ? need : most, s);
  });
  return cudaGetLastError();
}

}  // namespace moe
