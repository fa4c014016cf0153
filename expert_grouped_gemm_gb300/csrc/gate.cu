// gate.cu -- routing from router logits, forward and backward.
//
// A warp per token; lane l holds the experts e = l + 32 i (i < EPL) in registers. A choice
// score becomes an order-preserving 32-bit key, so the largest score of the warp is one
// integer reduction and, among equal scores, the lowest expert another: ties need no care
// and a token's selection is the same on every run. Key 1 is a masked expert (logit -inf or
// NaN, or a choice score that is -inf or NaN), key 0 one that cannot be chosen (already
// taken, in a group that was not kept, or past E).
//
// The softmax sums run over a fixed tree: lane l adds its experts by halves (i with
// i + EPL/2), then the lanes by butterflies, i.e. element j of the padded row with element
// j + n/2 at each step.
#include "block.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ uint32_t order_key(float c) {
  const uint32_t u = __float_as_uint(c + 0.0f);  // -0 and +0 are one value
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
constexpr uint32_t kKeyNone = 0, kKeyMasked = 1;

struct GateArgs {
  const void* logits;
  const float* bias;
  int* idx;
  float* w;
  int* count;
  const int* idx_in;
  const float* dw;
  void* dlogits;
  int T, E, k, G, Kg, take, renorm;
  float scale;
};

// Scores of one token: s[i] for expert lane + 32 i (0 where masked or past E).
template <int EPL, bool SOFTMAX, typename TL>
__device__ __forceinline__ void scores(const TL* row, int E, int lane, float (&l)[EPL], float (&s)[EPL]) {
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    const float v = e < E ? io<TL>::to_f(row[e]) : -INFINITY;
    l[i] = v != v ? -INFINITY : v;  // NaN masks its expert as -inf does
  }
  if constexpr (SOFTMAX) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) m = fmaxf(m, l[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    // l == m covers +inf (where l - m is NaN); a row without any expert left has m = -inf
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = l[i] == -INFINITY ? 0.0f : (l[i] == m ? 1.0f : expf(l[i] - m));
    float t[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) t[i] = s[i];
#pragma unroll
    for (int h = EPL / 2; h > 0; h >>= 1)
#pragma unroll
      for (int i = 0; i < h; ++i) t[i] += t[i + h];
    const float z = warp_sum(t[0]);
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = z > 0.0f ? s[i] / z : 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = l[i] == -INFINITY ? 0.0f : 1.0f / (1.0f + expf(-l[i]));
  }
}

// Largest key of the warp and the lowest expert that has it; the owner's copy is cleared.
template <int EPL>
__device__ __forceinline__ int take_best(uint32_t (&key)[EPL], int lane, uint32_t* best) {
  uint32_t b = key[0];
  int be = lane;
#pragma unroll
  for (int i = 1; i < EPL; ++i)
    if (key[i] > b) {
      b = key[i];
      be = lane + 32 * i;
    }
  const uint32_t m = __reduce_max_sync(kFull, b);
  const uint32_t e = __reduce_min_sync(kFull, b == m ? (uint32_t)be : 0xffffffffu);
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if ((int)e == lane + 32 * i) key[i] = kKeyNone;
  *best = m;
  return (int)e;
}

template <int EPL, bool SOFTMAX, typename TL>
__global__ void __launch_bounds__(256) k_gate_fwd(const GateArgs a) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  float l[EPL], s[EPL];
  scores<EPL, SOFTMAX>(reinterpret_cast<const TL*>(a.logits) + (int64_t)t * a.E, a.E, lane, l, s);
  uint32_t key[EPL];
  float c[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    c[i] = s[i] + (a.bias && e < a.E ? a.bias[e] : 0.0f);
    const bool masked = l[i] == -INFINITY || !(c[i] > -INFINITY);
    key[i] = e >= a.E ? kKeyNone : masked ? kKeyMasked : order_key(c[i]);
  }
  if (a.Kg < a.G) {
    const int per = a.E / a.G;
    // lane g keeps group g's score
    uint32_t gkey = lane < a.G ? kKeyMasked : kKeyNone;
    for (int g = 0; g < a.G; ++g) {
      uint32_t gk[EPL];
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        gk[i] = e >= g * per && e < (g + 1) * per ? key[i] : kKeyNone;
      }
      float score = 0.0f;
      bool any = false;
      for (int r = 0; r < a.take; ++r) {
        uint32_t b;
        const int e = take_best<EPL>(gk, lane, &b);
        if (b <= kKeyMasked) break;
        float ce = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if ((e >> 5) == i) ce = c[i];
        ce = __shfl_sync(kFull, ce, e & 31);
        score = any ? score + ce : ce;
        any = true;
      }
      if (lane == g && any) gkey = order_key(score);
    }
    uint32_t kept = 0;
    uint32_t gk1[1] = {gkey};
    for (int r = 0; r < a.Kg; ++r) {
      uint32_t b;
      kept |= 1u << take_best<1>(gk1, lane, &b);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E && !((kept >> (e / per)) & 1u)) key[i] = kKeyNone;
    }
  }
  int my_e = 0;
  float my_s = 0.0f, my_l = -INFINITY;
  for (int j = 0; j < a.k; ++j) {
    uint32_t b;
    const int e = take_best<EPL>(key, lane, &b);
    float se = 0.0f, le = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if ((e >> 5) == i) {
        se = s[i];
        le = l[i];
      }
    se = __shfl_sync(kFull, se, e & 31);
    le = __shfl_sync(kFull, le, e & 31);
    if (lane == j) {
      my_e = e;
      my_s = se;
      my_l = le;
    }
  }
  if (a.renorm) {
    if constexpr (SOFTMAX) {  // s / S over the chosen is the softmax of the chosen logits: it cannot underflow to 0 / 0
      float m = my_l;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      my_s = my_l == -INFINITY ? 0.0f : (my_l == m ? 1.0f : expf(my_l - m));
    }
    const float S = warp_sum(my_s);
    my_s = S > 0.0f ? my_s / S : 0.0f;
  }
  if (lane < a.k) {
    a.idx[(int64_t)t * a.k + lane] = my_e;
    a.w[(int64_t)t * a.k + lane] = my_s * a.scale;
    if (a.count) atomicAdd(a.count + my_e, 1);  // whole numbers: the order of the additions does not matter
  }
}

template <int EPL, bool SOFTMAX, typename TL, typename TG>
__global__ void __launch_bounds__(256) k_gate_bwd(const GateArgs a) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  float l[EPL], s[EPL], ds[EPL];
  scores<EPL, SOFTMAX>(reinterpret_cast<const TL*>(a.logits) + (int64_t)t * a.E, a.E, lane, l, s);
#pragma unroll
  for (int i = 0; i < EPL; ++i) ds[i] = 0.0f;
  int my_e = -1;
  float my_dw = 0.0f;
  if (lane < a.k) {
    my_e = a.idx_in[(int64_t)t * a.k + lane];
    my_dw = a.dw[(int64_t)t * a.k + lane] * a.scale;
    if (my_e < 0 || my_e >= a.E) my_e = -1;
  }
  // the chosen score (and logit) in its slot's lane
  float my_s = 0.0f, my_l = -INFINITY;
  for (int j = 0; j < a.k; ++j) {
    const int e = __shfl_sync(kFull, my_e, j);
    if (e < 0) continue;
    float se = 0.0f, le = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if ((e >> 5) == i) {
        se = s[i];
        le = l[i];
      }
    se = __shfl_sync(kFull, se, e & 31);
    le = __shfl_sync(kFull, le, e & 31);
    if (lane == j) {
      my_s = se;
      my_l = le;
    }
  }
  if (my_l == -INFINITY) my_dw = 0.0f;  // a masked or skipped slot takes no part
  if (SOFTMAX && a.renorm) {
    // the weights are the softmax of the chosen logits: dl_j = w_j (dw_j - sum_i w_i dw_i)
    float m = my_l;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    const float ex = my_l == -INFINITY ? 0.0f : (my_l == m ? 1.0f : expf(my_l - m));
    const float S = warp_sum(ex);
    const float wj = S > 0.0f ? ex / S : 0.0f;
    my_dw = wj * (my_dw - warp_sum(wj * my_dw));
  } else if (a.renorm) {
    const float S = warp_sum(my_s);
    const float dot = warp_sum(my_dw * my_s);
    my_dw = S > 0.0f ? (my_dw - dot / S) / S * my_s * (1.0f - my_s) : 0.0f;
  } else if (!SOFTMAX) {
    my_dw = my_dw * my_s * (1.0f - my_s);
  }
  for (int j = 0; j < a.k; ++j) {
    const int e = __shfl_sync(kFull, my_e, j);
    const float d = __shfl_sync(kFull, my_dw, j);
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (e == lane + 32 * i) ds[i] += d;
  }
  if (SOFTMAX && !a.renorm) {
    const float dot = warp_sum(my_dw * my_s);
#pragma unroll
    for (int i = 0; i < EPL; ++i) ds[i] = s[i] * (ds[i] - dot);
  }
  TG* out = reinterpret_cast<TG*>(a.dlogits) + (int64_t)t * a.E;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    if (e < a.E) out[e] = io<TG>::cvt(ds[i]);
  }
}

GateArgs args_of(const moe_gate_dims& d) {
  GateArgs a = {};
  a.T = (int)d.T;
  a.E = (int)d.E;
  a.k = (int)d.k;
  a.G = (int)d.n_group;
  a.Kg = (int)d.topk_group;
  a.take = d.group_take;
  a.renorm = d.renorm != 0;
  a.scale = d.scale;
  return a;
}

// f(std::integral_constant<int, EPL>) for the smallest supported number of experts per lane
template <typename F>
cudaError_t with_epl(int64_t E, F&& f) {
  const int epl = (int)((E + 31) / 32);
  if (epl <= 1) return f(std::integral_constant<int, 1>());
  if (epl <= 2) return f(std::integral_constant<int, 2>());
  if (epl <= 4) return f(std::integral_constant<int, 4>());
  if (epl <= 8) return f(std::integral_constant<int, 8>());
  if (epl <= 16) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}

template <int EPL, bool SOFTMAX>
cudaError_t bwd_typed(const moe_gate_dims& d, const GateArgs& a, int grid, cudaStream_t st) {
  if (d.dtype == MOE_BF16) {
    if (d.grad_dtype == MOE_BF16) MOE_LAUNCH(k_gate_bwd<EPL, SOFTMAX, __nv_bfloat16, __nv_bfloat16>, grid, 256, 0, st, a);
    else MOE_LAUNCH(k_gate_bwd<EPL, SOFTMAX, __nv_bfloat16, float>, grid, 256, 0, st, a);
  } else {
    if (d.grad_dtype == MOE_BF16) MOE_LAUNCH(k_gate_bwd<EPL, SOFTMAX, float, __nv_bfloat16>, grid, 256, 0, st, a);
    else MOE_LAUNCH(k_gate_bwd<EPL, SOFTMAX, float, float>, grid, 256, 0, st, a);
  }
  return cudaSuccess;
}

template <int EPL, bool SOFTMAX>
cudaError_t fwd_typed(const moe_gate_dims& d, const GateArgs& a, int grid, cudaStream_t st) {
  if (d.dtype == MOE_BF16) MOE_LAUNCH(k_gate_fwd<EPL, SOFTMAX, __nv_bfloat16>, grid, 256, 0, st, a);
  else MOE_LAUNCH(k_gate_fwd<EPL, SOFTMAX, float>, grid, 256, 0, st, a);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_gate_fwd(const moe_gate_dims& d, const void* logits, const float* bias, int* topk_idx, float* topk_w,
                            int* count, int sms, cudaStream_t st, int* launches) {
  GateArgs a = args_of(d);
  a.logits = logits;
  a.bias = bias;
  a.idx = topk_idx;
  a.w = topk_w;
  a.count = count;
  if (count) {
    const cudaError_t e = cudaMemsetAsync(count, 0, (size_t)d.E * sizeof(int), st);
    if (e != cudaSuccess) return e;
  }
  *launches += 1;
  const int grid = (int)((d.T + 7) / 8);
  return with_epl(d.E, [&](auto epl) {
    return d.score == MOE_SCORE_SOFTMAX ? fwd_typed<epl.value, true>(d, a, grid, st)
                                        : fwd_typed<epl.value, false>(d, a, grid, st);
  });
}

cudaError_t launch_gate_bwd(const moe_gate_dims& d, const void* logits, const int* topk_idx, const float* dw,
                            void* dlogits, int sms, cudaStream_t st, int* launches) {
  GateArgs a = args_of(d);
  a.logits = logits;
  a.idx_in = topk_idx;
  a.dw = dw;
  a.dlogits = dlogits;
  *launches += 1;
  const int grid = (int)((d.T + 7) / 8);
  return with_epl(d.E, [&](auto epl) {
    return d.score == MOE_SCORE_SOFTMAX ? bwd_typed<epl.value, true>(d, a, grid, st)
                                        : bwd_typed<epl.value, false>(d, a, grid, st);
  });
}

}  // namespace moe
