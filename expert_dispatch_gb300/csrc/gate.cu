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
// One warp a token, expert e on lane e % 32: a token's logits are read once, all
// sums over experts are warp butterflies.  Bound by the logits' bytes.
#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

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

// Below this logit a sigmoid is exp(l) to 26 digits; where all logits of a sum
// lie below it the sum is formed of exp(l - max), which does not underflow.
constexpr float kSmallLogit = -60.f;

// A token's probabilities: pr[i] of expert lane + 32 i (softmax, or sigmoid over
// the sum of sigmoids); sg[i] = the sigmoid (SIGMOID only).  l[i] = -inf past E.
template <int PL, bool SIGMOID>
__device__ __forceinline__ void probabilities(const float (&l)[PL], float (&pr)[PL],
                                              float (&sg)[PL]) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < PL; ++i) m = fmaxf(m, l[i]);
  m = warp_max(m);
  float z = 0.f;
  const bool shift = !SIGMOID || m < kSmallLogit;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    if (SIGMOID) sg[i] = 1.0f / (1.0f + expf(-l[i]));
    pr[i] = shift ? expf(l[i] - m) : sg[i];
    z += pr[i];
  }
  z = warp_sum(z);
#pragma unroll
  for (int i = 0; i < PL; ++i) pr[i] = pr[i] / z;
}

// Lane j < k holds slot j: its expert (-1: none) and that expert's logit.
struct Slot {
  int id;
  float logit;
};
template <typename T>
__device__ __forceinline__ Slot load_slot(const T* __restrict__ row, const int32_t* __restrict__ ids,
                                          size_t t, int E, int k, int lane) {
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
  if (s.id >= 0) v = shift ? expf(s.logit - m) : 1.0f / (1.0f + expf(-s.logit));
  return v / warp_sum(v);
}

template <int PL, typename T>
__device__ __forceinline__ void load_logits(const T* __restrict__ row, int E, int lane,
                                            float (&l)[PL]) {
#pragma unroll
  for (int i = 0; i < PL; ++i)
    l[i] = lane + 32 * i < E ? load_as_f32(row, lane + 32 * i) : -INFINITY;
}

// Blocks' sums: part_p [blocks][E], part_c [blocks][E + 1] (counts, tokens).
template <int PL, bool SIGMOID, bool NORM, typename T>
__global__ void __launch_bounds__(kThreads)
    gate_forward_kernel(const T* __restrict__ logits, const int32_t* __restrict__ ids, int T_, int E,
                        int k, float rs, float* __restrict__ w, float* __restrict__ part_p,
                        int32_t* __restrict__ part_c) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sum_s[kWarps][32 * PL];
  __shared__ int32_t count_s[32 * PL + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e <= E; e += kThreads) count_s[e] = 0;
  __syncthreads();
  float sum[PL] = {};
  int tokens = 0;
  for (long long t = (long long)blockIdx.x * kWarps + warp; t < T_;
       t += (long long)gridDim.x * kWarps) {
    const T* row = logits + (size_t)t * E;
    const Slot s = load_slot(row, ids, (size_t)t, E, k, lane);
    const bool live = __any_sync(0xffffffffu, s.id >= 0);
    if (live) {
      float l[PL], pr[PL], sg[PL];
      load_logits<PL>(row, E, lane, l);
      probabilities<PL, SIGMOID>(l, pr, sg);
#pragma unroll
      for (int i = 0; i < PL; ++i) sum[i] += pr[i];
      ++tokens;
      if (s.id >= 0) atomicAdd(&count_s[s.id], 1);
      if (w) {
        float v;
        if (NORM) {
          v = normalised<SIGMOID>(s);
        } else if (SIGMOID) {
          v = 1.0f / (1.0f + expf(-s.logit));
        } else {  // the slot's probability, from the lane that has it
          v = 0.f;
          for (int j = 0; j < k; ++j) {
            const int id = __shfl_sync(0xffffffffu, s.id, j);
            float have = 0.f;
#pragma unroll
            for (int i = 0; i < PL; ++i)
              if (id >> 5 == i) have = pr[i];
            have = __shfl_sync(0xffffffffu, have, id & 31);
            if (lane == j) v = have;
          }
        }
        if (lane < k) w[(size_t)t * k + lane] = s.id >= 0 ? rs * v : 0.f;
      }
    } else if (w && lane < k) {
      w[(size_t)t * k + lane] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) sum_s[warp][lane + 32 * i] = sum[i];
  if (lane == 0) atomicAdd(&count_s[E], tokens);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kThreads) {
    part_c[(size_t)blockIdx.x * (E + 1) + e] = count_s[e];
    if (e < E) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) v += sum_s[i][e];
      part_p[(size_t)blockIdx.x * E + e] = v;
    }
  }
}

// The blocks' sums together: counts [E + 1], prob [E], loss [1] (prob, loss may
// be null).  One block; a thread an expert, blocks in order.
__global__ void __launch_bounds__(1024) gate_finish_kernel(const float* __restrict__ part_p,
                                                           const int32_t* __restrict__ part_c,
                                                           int blocks, int E, int k,
                                                           int32_t* __restrict__ counts,
                                                           float* __restrict__ prob,
                                                           float* __restrict__ loss) {
  pdl_wait();
  pdl_trigger();
  __shared__ float dot_s[32];
  __shared__ int n_s;
  const int e = threadIdx.x, lane = e & 31;
  if (e < 32) {
    int n = 0;
    for (int b = lane; b < blocks; b += 32) n += part_c[(size_t)b * (E + 1) + E];
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) n_s = n;
  }
  int c = 0;
  float p = 0.f;
  if (e < E)
    for (int b = 0; b < blocks; ++b) {
      c += part_c[(size_t)b * (E + 1) + e];
      p += part_p[(size_t)b * E + e];
    }
  __syncthreads();
  const int n = n_s;
  p = n > 0 ? p / (float)n : 0.f;
  if (e < E) {
    if (counts) counts[e] = c;
    if (prob) prob[e] = p;
  }
  if (counts && e == 0) counts[E] = n;
  const float dot = warp_sum(e < E ? (float)c * p : 0.f);
  if (lane == 0) dot_s[e >> 5] = dot;
  __syncthreads();
  if (e < 32 && loss) {
    const float v = warp_sum(lane < (int)blockDim.x / 32 ? dot_s[lane] : 0.f);
    if (lane == 0) *loss = n > 0 ? v * ((float)E / ((float)k * (float)n)) : 0.f;
  }
}

template <int PL, bool SIGMOID, bool NORM, typename T>
__global__ void __launch_bounds__(kThreads)
    gate_backward_kernel(const T* __restrict__ logits, const int32_t* __restrict__ ids,
                         const int32_t* __restrict__ counts, const float* __restrict__ dw,
                         const float* __restrict__ dloss, int T_, int E, int k, float rs,
                         T* __restrict__ dlogits) {
  pdl_wait();
  pdl_trigger();
  __shared__ float add_s[kWarps][32 * PL];  // the selected experts' part, per warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
  for (long long t = (long long)blockIdx.x * kWarps + warp; t < T_;
       t += (long long)gridDim.x * kWarps) {
    const T* row = logits + (size_t)t * E;
    T* out = dlogits + (size_t)t * E;
    const Slot s = load_slot(row, ids, (size_t)t, E, k, lane);
    if (!__any_sync(0xffffffffu, s.id >= 0)) {
#pragma unroll
      for (int i = 0; i < PL; ++i)
        if (lane + 32 * i < E) out[lane + 32 * i] = (T)0.f;
      continue;
    }
    float l[PL], pr[PL], sg[PL];
    load_logits<PL>(row, E, lane, l);
    probabilities<PL, SIGMOID>(l, pr, sg);
    float mean = 0.f;  // <c, p>
#pragma unroll
    for (int i = 0; i < PL; ++i) mean += c[i] * pr[i];
    mean = warp_sum(mean);
    float pull = 0.f;  // softmax weights: the part -<g, p> p of every expert
    if (dw) {
      const float g = s.id >= 0 ? rs * dw[(size_t)t * k + lane] : 0.f;
      float v = 0.f;  // slot j's own part, on lane j
      if (NORM) {
        const float q = normalised<SIGMOID>(s);
        const float dot = warp_sum(s.id >= 0 ? g * q : 0.f);
        v = q * (g - dot);
        if (SIGMOID) v *= 1.0f - 1.0f / (1.0f + expf(-s.logit));
      } else if (SIGMOID) {
        const float sj = 1.0f / (1.0f + expf(-s.logit));
        v = g * sj * (1.0f - sj);
      } else {
        v = g;  // times p_e, known on the expert's lane
      }
      for (int j = 0; j < k; ++j) {  // in slot order: an id may come twice
        const int id = __shfl_sync(0xffffffffu, s.id, j);
        const float vj = __shfl_sync(0xffffffffu, v, j);
        if (id >= 0 && (id & 31) == lane) add_s[warp][id] += vj;
      }
      __syncwarp();
      if (!NORM && !SIGMOID) {
#pragma unroll
        for (int i = 0; i < PL; ++i) pull += add_s[warp][lane + 32 * i] * pr[i];
        pull = warp_sum(pull);
      }
    }
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      float v = a * pr[i] * (c[i] - mean);
      if (SIGMOID) v *= 1.0f - sg[i];
      const float add = add_s[warp][lane + 32 * i];
      v += !NORM && !SIGMOID ? pr[i] * (add - pull) : add;
      add_s[warp][lane + 32 * i] = 0.f;
      if (lane + 32 * i < E) out[lane + 32 * i] = (T)v;
    }
    __syncwarp();
  }
}

template <int PL, bool SIGMOID, bool NORM, typename T>
struct Kernels {
  static void forward(const void* logits, const int32_t* ids, const moe_layer_desc& D, float* w,
                      float* part_p, int32_t* part_c, int blocks, cudaStream_t s) {
    (void)launch_kernel(gate_forward_kernel<PL, SIGMOID, NORM, T>, blocks, kThreads, 0, s,
                        static_cast<const T*>(logits), ids, D.T, D.E, D.k, D.routed_scaling, w,
                        part_p, part_c);
  }
  static void backward(const void* logits, const int32_t* ids, const moe_layer_desc& D,
                       const int32_t* counts, const float* dw, const float* dloss, void* dlogits,
                       int blocks, cudaStream_t s) {
    (void)launch_kernel(gate_backward_kernel<PL, SIGMOID, NORM, T>, blocks, kThreads, 0, s,
                        static_cast<const T*>(logits), ids, counts, dw, dloss, D.T, D.E, D.k,
                        D.routed_scaling, static_cast<T*>(dlogits));
  }
};

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
  if (D.E <= 64)
    by_gate(std::integral_constant<int, 2>{});
  else if (D.E <= 128)
    by_gate(std::integral_constant<int, 4>{});
  else if (D.E <= 256)
    by_gate(std::integral_constant<int, 8>{});
  else if (D.E <= 512)
    by_gate(std::integral_constant<int, 16>{});
  else
    by_gate(std::integral_constant<int, 32>{});
}

int grid_of(const moe_layer_desc& D) {
  // does not depend on the device: the workspace's size goes by it
  const int need = (D.T + kWarps - 1) / kWarps;
  return need < 304 ? need : 304;
}

}  // namespace

size_t gate_workspace_bytes(const moe_layer_desc& D) {
  return (size_t)grid_of(D) * (2 * (size_t)D.E + 1) * 4;
}

cudaError_t launch_gate_forward(const moe_layer_desc& D, int dtype, const void* logits,
                                const int32_t* ids, float* w, int32_t* counts, float* prob,
                                float* loss, void* ws, cudaStream_t s) {
  const int blocks = grid_of(D);
  float* part_p = static_cast<float*>(ws);
  int32_t* part_c = reinterpret_cast<int32_t*>(part_p + (size_t)blocks * D.E);
  {
    ProfScope pr("gate_forward", s);
    choose(D, dtype, [&](auto kernels) {
      decltype(kernels)::forward(logits, ids, D, w, part_p, part_c, blocks, s);
    });
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (!counts && !prob && !loss) return cudaSuccess;
  ProfScope pr("gate_finish", s);
  (void)launch_kernel(gate_finish_kernel, 1, (D.E + 31) / 32 * 32, 0, s, (const float*)part_p,
                      (const int32_t*)part_c, blocks, D.E, D.k, counts, prob, loss);
  return cudaGetLastError();
}

cudaError_t launch_gate_backward(const moe_layer_desc& D, int dtype, const void* logits,
                                 const int32_t* ids, const int32_t* counts, const float* dw,
                                 const float* dloss, void* dlogits, cudaStream_t s) {
  const int need = (D.T + kWarps - 1) / kWarps, most = num_sms() * 8;
  ProfScope pr("gate_backward", s);
  choose(D, dtype, [&](auto kernels) {
    decltype(kernels)::backward(logits, ids, D, counts, dw, dloss, dlogits,
                                need < most ? need : most, s);
  });
  return cudaGetLastError();
}

}  // namespace moe
