// gate.cu -- routing from router logits, forward and backward.
//
// A warp per token. The experts of a group lie on L = 2^n consecutive lanes, R consecutive
// experts a lane, so everything a group needs is a butterfly over its lanes and the lowest lane
// with a value holds the lowest expert with it. A choice score becomes an order-preserving
// 32-bit key: the largest of the warp is one integer reduction, and ties fall to the lower expert
// by the lane order. Key 1 is a masked expert (logit -inf or NaN, or a choice score that is -inf
// or NaN), key 0 one that cannot be chosen (taken, in a group that was not kept, or absent).
//
// Without a bias the scores are ordered as the logits are, so the logits themselves are compared
// and only the chosen experts' scores are computed; a group's sum of two scores and a bias need
// every score. The kernels are bound by latency: the logits are read once (T = 8192, E = 256 is
// 8.4 MB, 1.2 us of HBM time), the rest is a chain of k warp reductions that a warp runs for one token with nothing of
// its own beside it. There, with 8 groups and a bias, 1024 blocks go over 760 places (45 registers, five a SM) in two
// waves, issue in half of their cycles, and the counts are a second launch: 13.4 us together with logits that change
// from call to call, 12.2 with the same ones in L2. 8 tokens of 128 experts 2.3 us; backward of 4097 x 160 2.9 us.
#include <algorithm>
#include <type_traits>

#include "act.cuh"
#include "block.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kKeyNone = 0, kKeyMasked = 1;
template <int EPL>
constexpr int one_block_tokens = EPL <= 4 ? 32 : EPL <= 16 ? 16 : 8;  // tokens one block may take by itself

__device__ __forceinline__ uint32_t order_key(float c) {
  const uint32_t u = __float_as_uint(c + 0.0f);  // -0 and +0 are one value
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

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
  int per;     // experts of a group
  int L, R;    // lanes of a group, experts of a lane
  int vec;     // the lanes' experts can be read (and written) 16 bytes at a time
  int vec_bias;  // and their biases
  int direct;  // the logits decide the order
  float scale;
};

// The lane's n logits (of at most EPL) at p; NaN masks its expert as -inf does.
template <int EPL, typename TL>
__device__ __forceinline__ void load_logits(const TL* p, int n, bool vec, float (&l)[EPL]) {
  constexpr int V = 16 / (int)sizeof(TL);
  if constexpr (EPL % V == 0) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < EPL; i += V) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (i < n) u = *reinterpret_cast<const uint4*>(p + i);
        const TL* e = reinterpret_cast<const TL*>(&u);
#pragma unroll
        for (int q = 0; q < V; ++q) l[i + q] = i < n ? io<TL>::to_f(e[q]) : -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i) l[i] = l[i] != l[i] ? -INFINITY : l[i];
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const float v = i < n ? io<TL>::to_f(p[i]) : -INFINITY;
    l[i] = v != v ? -INFINITY : v;
  }
}

template <int EPL>
__device__ __forceinline__ void load_bias(const float* p, int n, bool vec, float (&b)[EPL]) {
  if constexpr (EPL % 4 == 0) {
    if (p && vec) {
#pragma unroll
      for (int i = 0; i < EPL; i += 4) {
        const float4 u = i < n ? *reinterpret_cast<const float4*>(p + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        b[i] = u.x;
        b[i + 1] = u.y;
        b[i + 2] = u.z;
        b[i + 3] = u.w;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) b[i] = p && i < n ? p[i] : 0.0f;
}

// e^{l - m} of a softmax with maximum m: 0 for masked experts, 1 at the maximum (which may be +inf)
__device__ __forceinline__ float soft(float l, float m) {
  return l == -INFINITY ? 0.0f : (l == m ? 1.0f : expf(l - m));
}
__device__ __forceinline__ float logistic(float l) { return l == -INFINITY ? 0.0f : 1.0f / (1.0f + expf(-l)); }

// Maximum over the warp (one reduction of order-preserving keys).
__device__ __forceinline__ float warp_max(float v) { return key_value(__reduce_max_sync(kFull, order_key(v))); }

// Softmax over a token's logits: l becomes the scores, *m the largest logit and *inv the factor of
// e^{l - m} (0 when every expert is masked).
template <int EPL>
__device__ __forceinline__ void softmax_row(float (&l)[EPL], float* m, float* inv) {
  float v = l[0];
#pragma unroll
  for (int i = 1; i < EPL; ++i) v = fmaxf(v, l[i]);
  *m = warp_max(v);
  float z = 0.0f;
  if (fabsf(*m) < INFINITY) {  // the usual row: e^{-inf - m} = 0 needs no care
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      l[i] = expf(l[i] - *m);
      z += l[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      l[i] = soft(l[i], *m);
      z += l[i];
    }
  }
  z = warp_sum(z);
  *inv = z > 0.0f ? 1.0f / z : 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) l[i] *= *inv;
}

// Keys of a lane in descending order (equal ones in ascending expert order), with their places.
// An odd-even transposition network: neighbours change places only when the later one is larger.
template <int EPL>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[EPL], int (&at)[EPL]) {
#pragma unroll
  for (int i = 0; i < EPL; ++i) at[i] = i;
#pragma unroll
  for (int r = 0; r < EPL; ++r)
#pragma unroll
    for (int i = r & 1; i + 1 < EPL; i += 2) {
      const bool sw = key[i + 1] > key[i];
      const uint32_t hi = sw ? key[i + 1] : key[i], lo = sw ? key[i] : key[i + 1];
      const int ah = sw ? at[i + 1] : at[i], al = sw ? at[i] : at[i + 1];
      key[i] = hi;
      key[i + 1] = lo;
      at[i] = ah;
      at[i + 1] = al;
    }
}

// Bitonic sort of one (key, expert) a lane: keys descending, equal keys by ascending expert.
__device__ __forceinline__ void warp_sort(uint32_t& key, int& e, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const uint32_t ok = __shfl_xor_sync(kFull, key, o);
      const int oe = __shfl_xor_sync(kFull, e, o);
      const bool mine_first = key > ok || (key == ok && e < oe);
      // the lower lane of the pair keeps the first in a descending run, the last in an ascending one
      const bool keep_first = ((lane & o) == 0) == ((lane & size) == 0);
      if (mine_first != keep_first) {
        key = ok;
        e = oe;
      }
    }
}
// The same for keys alone.
__device__ __forceinline__ uint32_t warp_sort(uint32_t key, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const uint32_t ok = __shfl_xor_sync(kFull, key, o);
      const bool larger = ((lane & o) == 0) == ((lane & size) == 0);
      key = larger ? max(key, ok) : min(key, ok);
    }
  return key;
}

constexpr int kCountBlocks = 8;  // largest cluster that counts

// The blocks' histograms added over the cluster that is the grid, each block a share of the experts
// (a grid of one block has them all).
__device__ __forceinline__ void cluster_counts(const int* hist, int E, int* count) {
  if (gridDim.x == 1) {
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) count[e] = hist[e];
    return;
  }
  cluster_sync_all();
  const int blocks = (int)gridDim.x, share = (E + blocks - 1) / blocks;
  const int end = min(E, ((int)blockIdx.x + 1) * share);
  for (int e = (int)blockIdx.x * share + (int)threadIdx.x; e < end; e += blockDim.x) {
    const uint32_t at = smem_u32(hist + e);
    int v[kCountBlocks], s = 0;
#pragma unroll
    for (int r = 0; r < kCountBlocks; ++r) {
      v[r] = 0;
      if (r < blocks)
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v[r]) : "r"(mapa_shared(at, r)) : "memory");
    }
#pragma unroll
    for (int r = 0; r < kCountBlocks; ++r) s += v[r];
    count[e] = s;
  }
  cluster_sync_all();  // no block leaves while another still reads its histogram
}

template <int EPL, bool SOFTMAX, typename TL>
__global__ void __launch_bounds__(32 * one_block_tokens<EPL>) k_gate_fwd(const GateArgs a) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  __shared__ uint2 candidates[EPL <= 8 ? 1 : one_block_tokens<EPL>][32];
  __shared__ int hist[1024];  // the grid is one cluster: it has every token and writes the counts itself
  const bool one = gridDim.x <= kCountBlocks && a.count;
  if (one) {
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t < a.T) {
    const int grp = lane / a.L;
    const int e0 = grp * a.per + (lane & (a.L - 1)) * a.R;  // this lane's first expert
    const int n = grp < a.G ? max(0, min(a.R, (grp + 1) * a.per - e0)) : 0;
    const TL* row = reinterpret_cast<const TL*>(a.logits) + (int64_t)t * a.E;
    uint32_t key[EPL];
    float m = 0.0f, inv = 0.0f;
    {
      float l[EPL];
      load_logits<EPL, TL>(row + e0, n, a.vec, l);
      if (a.direct) {
        if constexpr (SOFTMAX) {  // beside a +inf logit every other score is zero, and they tie
          bool inf = false;
#pragma unroll
          for (int i = 0; i < EPL; ++i) inf |= l[i] == INFINITY;
          if (__any_sync(kFull, inf)) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
              if (l[i] > -INFINITY) l[i] = l[i] == INFINITY ? 1.0f : 0.0f;
          }
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = i >= n ? kKeyNone : l[i] == -INFINITY ? kKeyMasked : order_key(l[i]);
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = l[i] == -INFINITY;
        if constexpr (SOFTMAX) {
          softmax_row<EPL>(l, &m, &inv);
        } else {
          // within three ulp of fp32, whatever the logit: the exponent of a base-2 form would be rounded to 2^-24 of the
          // logit, which turns over close scores of e^-30 (0.25 us less at T = 8192, E = 256). The weights' scores are
          // divided out below; here one below 2^-126 counts as zero.
#pragma unroll
          for (int i = 0; i < EPL; ++i) l[i] = rcp_approx(1.0f + expf(-l[i]));
        }
        float bias[EPL];
        load_bias<EPL>(a.bias ? a.bias + e0 : nullptr, n, a.vec_bias, bias);
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          const float c = l[i] + bias[i];
          key[i] = i >= n ? kKeyNone : (key[i] || !(c > -INFINITY)) ? kKeyMasked : order_key(c);
        }
      }
    }
    if (a.Kg < a.G) {
      uint32_t m1 = kKeyNone, m2 = kKeyNone;  // the group's two largest
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        m2 = max(m2, min(m1, key[i]));
        m1 = max(m1, key[i]);
      }
      for (int o = 1; o < a.L; o <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(kFull, m1, o), o2 = __shfl_xor_sync(kFull, m2, o);
        m2 = max(max(m2, o2), min(m1, o1));
        m1 = max(m1, o1);
      }
      uint32_t gk = m1;
      if (a.take == 2 && m2 > kKeyMasked) gk = order_key(key_value(m1) + key_value(m2));
      int rank = 0;  // groups in front of this one
      for (int g = 0; g < a.G; ++g) {
        const uint32_t o = __shfl_sync(kFull, gk, g * a.L);
        rank += o > gk || (o == gk && g < grp);
      }
      if (rank >= a.Kg) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) key[i] = kKeyNone;
      }
    }
    int my_e = 0;
    if constexpr (EPL <= 8) {
      // Lanes with few experts sort them once; k rounds take the largest key of the warp, in its
      // lowest lane, and that lane drops its first. (Gathering as below: E = 128, k = 8 at 8192
      // tokens 7.2 us, so 5.2; E = 1024 at 2000 tokens 9.9, so 13; logits in L2, without counts.)
      int at[EPL];
      sort_keys<EPL>(key, at);
      for (int j = 0; j < a.k; ++j) {
        const uint32_t top = __reduce_max_sync(kFull, key[0]);
        const int who = __ffs(__ballot_sync(kFull, key[0] == top)) - 1;
        const int e = __shfl_sync(kFull, e0 + at[0], who);
        if (lane == j) my_e = e;
        if (lane == who) {
#pragma unroll
          for (int i = 0; i + 1 < EPL; ++i) {
            key[i] = key[i + 1];
            at[i] = at[i + 1];
          }
          key[EPL - 1] = kKeyNone;
        }
      }
    } else {
      // The k-th largest of the lanes' maxima bounds the k-th largest key from below, so the keys at or
      // above it hold the k chosen ones and, as a rule, few others: they are gathered, one a lane, and
      // sorted. More than 32 of them (many equal keys, few lanes with any) are taken one by one.
      uint32_t half[2] = {kKeyNone, kKeyNone};  // the maxima of the lane's two halves
#pragma unroll
      for (int i = 0; i < EPL; ++i) half[2 * i / EPL] = max(half[2 * i / EPL], key[i]);
      uint32_t top = warp_sort(max(half[0], half[1]), lane);
      if (a.Kg < a.G) {
        // lanes of dropped groups hold nothing: the 32 largest of both halves' maxima bound more
        // tightly (one list against the other reversed; 16 of 2 x 128 experts at 16384 tokens: 30 us, 51 without)
        const uint32_t low = warp_sort(min(half[0], half[1]), lane);
        top = warp_sort(max(top, __shfl_sync(kFull, low, 31 - lane)), lane);
      }
      const uint32_t bound = max(__shfl_sync(kFull, top, a.k - 1), kKeyMasked);
      uint2* cand = candidates[threadIdx.x >> 5];
      int count = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const uint32_t m = __ballot_sync(kFull, key[i] >= bound);
        if (m) {
          const int pos = count + __popc(m & ((1u << lane) - 1u));
          if (key[i] >= bound && pos < 32) cand[pos] = make_uint2(key[i], (uint32_t)(e0 + i));
          count += __popc(m);
        }
      }
      if (count <= 32) {
        __syncwarp();
        const uint2 c = lane < count ? cand[lane] : make_uint2(kKeyNone, 0x7fffffffu);
        uint32_t ck = c.x;
        my_e = (int)c.y;
        warp_sort(ck, my_e, lane);
      } else {
        uint32_t best;  // this lane's largest key, the first expert that has it
        int bi;
        auto search = [&]() {
          best = key[0];
          bi = 0;
#pragma unroll
          for (int i = 1; i < EPL; ++i)
            if (key[i] > best) {
              best = key[i];
              bi = i;
            }
        };
        search();
        for (int j = 0; j < a.k; ++j) {
          const uint32_t top = __reduce_max_sync(kFull, best);
          const int who = __ffs(__ballot_sync(kFull, best == top)) - 1;
          const int e = __shfl_sync(kFull, e0 + bi, who);
          if (lane == j) my_e = e;
          if (lane == who) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
              if (i == bi) key[i] = kKeyNone;
            search();
          }
        }
      }
    }
    // weights: lane j reads its chosen logit again (a line that is still in L1)
    float lj = lane < a.k ? io<TL>::to_f(row[my_e]) : -INFINITY;
    if (lj != lj) lj = -INFINITY;
    float s;
    if (SOFTMAX) {
      // s / S over the chosen is the softmax of the chosen logits: it cannot become 0 / 0
      if (a.renorm) {
        m = warp_max(lj);
      } else if (a.direct) {  // the row's sum has not been needed so far
        float l[EPL];
        load_logits<EPL, TL>(row + e0, n, a.vec, l);
        softmax_row<EPL>(l, &m, &inv);
      }
      s = soft(lj, m);
      if (!a.renorm) s *= inv;
    } else {
      s = logistic(lj);
    }
    if (a.renorm) {
      const float S = warp_sum(s);
      s = S > 0.0f ? s / S : 0.0f;
    }
    if (lane < a.k) {
      a.idx[(int64_t)t * a.k + lane] = my_e;
      a.w[(int64_t)t * a.k + lane] = s * a.scale;
      if (one) atomicAdd(&hist[my_e], 1);  // whole numbers: the order does not matter
    }
  }
  if (one) cluster_counts(hist, a.E, a.count);
}

// How often each expert stands in idx[n], for grids of more than one cluster. (Counting with atomics
// on global memory as the tokens are routed took as long again as the routing: the counters of all
// experts share a few L2 lines.)
__global__ void __launch_bounds__(1024) __cluster_dims__(kCountBlocks) k_gate_count(const int* idx, int64_t n, int E,
                                                                                    int* count) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  __shared__ int hist[1024];
  hist[threadIdx.x] = 0;
  __syncthreads();
  constexpr int U = 8;
  for (int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x; i < n; i += (int64_t)kCountBlocks * 1024 * U) {
    int e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = i + (int64_t)u * kCountBlocks * 1024;
      e[u] = at < n ? idx[at] : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (e[u] >= 0) atomicAdd(&hist[e[u]], 1);
  }
  cluster_counts(hist, E, count);
}

template <int EPL, bool SOFTMAX, typename TL, typename TG>
__global__ void __launch_bounds__(256) k_gate_bwd(const GateArgs a) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int e0 = lane * a.R, n = max(0, min(a.R, a.E - e0));
  // what the slots add to each expert's gradient, in the lanes' order
  __shared__ __align__(16) float sums[8][32 * EPL];
  float* sum = sums[threadIdx.x >> 5];
#pragma unroll
  for (int i = 0; i < EPL; ++i) sum[lane + 32 * i] = 0.0f;
  const TL* row = reinterpret_cast<const TL*>(a.logits) + (int64_t)t * a.E;
  // slot j in lane j; a skipped or masked slot takes no part
  int my_e = -1;
  float dw = 0.0f;
  if (lane < a.k) {
    my_e = a.idx_in[(int64_t)t * a.k + lane];
    dw = a.dw[(int64_t)t * a.k + lane] * a.scale;
    if (my_e < 0 || my_e >= a.E) my_e = -1;
  }
  const bool dense = SOFTMAX && !a.renorm;
  float l[EPL], m = 0.0f, inv = 0.0f;
  if (dense) {
    load_logits<EPL, TL>(row + e0, n, a.vec, l);
    softmax_row<EPL>(l, &m, &inv);
  }
  float lj = my_e >= 0 ? io<TL>::to_f(row[my_e]) : -INFINITY;
  if (lj != lj) lj = -INFINITY;
  if (lj == -INFINITY) dw = 0.0f;
  float d;          // what slot j adds to its expert's gradient
  float dot = 0.0f; // dense: sum of ds s over the chosen
  if (dense) {
    d = dw;
    dot = warp_sum(dw * soft(lj, m) * inv);
  } else if (SOFTMAX) {
    // the weights are the softmax of the chosen logits: dl_j = w_j (dw_j - sum_i w_i dw_i)
    const float s = soft(lj, warp_max(lj));
    const float S = warp_sum(s);
    const float w = S > 0.0f ? s / S : 0.0f;
    d = w * (dw - warp_sum(w * dw));
  } else {
    const float s = logistic(lj);
    if (a.renorm) {
      // ds_j s_j with s_j / S taken first: 1 / S of denormal scores would be infinite
      const float S = warp_sum(s);
      const float w = S > 0.0f ? s / S : 0.0f;
      d = w * (dw - warp_sum(w * dw)) * (1.0f - s);
    } else {
      d = dw * s * (1.0f - s);
    }
  }
  // expert e is lane e / R's element e % R; its sum stands at [e % R][lane], free of bank conflicts
  const int at = my_e >= 0 ? (my_e % a.R) * 32 + my_e / a.R : -1;
  const bool first = (__ffs(__match_any_sync(kFull, my_e)) - 1) == lane;
  __syncwarp();
  if (at >= 0 && first) sum[at] = d;
  if (__any_sync(kFull, at >= 0 && !first)) {  // an expert listed twice: the others add to it in slot order
    for (int j = 0; j < a.k; ++j) {
      __syncwarp();
      if (lane == j && at >= 0 && !first) sum[at] += d;
    }
  }
  __syncwarp();
  float out[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) out[i] = sum[i * 32 + lane];
  if (dense) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) out[i] = l[i] * (out[i] - dot);
  }
  TG* o = reinterpret_cast<TG*>(a.dlogits) + (int64_t)t * a.E + e0;
  constexpr int V = 16 / (int)sizeof(TG);
  if constexpr (EPL % V == 0) {
    if (a.vec) {
#pragma unroll
      for (int i = 0; i < EPL; i += V)
        if (i < n) {
          uint4 u;
          TG* e = reinterpret_cast<TG*>(&u);
#pragma unroll
          for (int q = 0; q < V; ++q) e[q] = io<TG>::cvt(out[i + q]);
          *reinterpret_cast<uint4*>(o + i) = u;
        }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (i < n) o[i] = io<TG>::cvt(out[i]);
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
  a.per = a.E / a.G;
  return a;
}

// f(integral_constant<EPL>) for the smallest number of experts per lane that holds R. Numbers that
// are multiples of 8 are read 16 bytes at a time in either type; 4 in fp32.
template <typename F>
cudaError_t with_epl(int R, F&& f) {
  if (R <= 1) return f(std::integral_constant<int, 1>());
  if (R <= 2) return f(std::integral_constant<int, 2>());
  if (R <= 4) return f(std::integral_constant<int, 4>());
  if (R <= 8) return f(std::integral_constant<int, 8>());
  if (R <= 16) return f(std::integral_constant<int, 16>());
  if (R <= 32) return f(std::integral_constant<int, 32>());
  return f(std::integral_constant<int, 64>());  // groups that are no power of two leave lanes empty
}

template <int EPL, bool SOFTMAX>
cudaError_t bwd_typed(const moe_gate_dims& d, const GateArgs& a, cudaStream_t st) {
  const int grid = (int)((d.T + 7) / 8);
  if (d.dtype == MOE_BF16) {
    if (d.grad_dtype == MOE_BF16) MOE_LAUNCH(k_gate_bwd<EPL, SOFTMAX, __nv_bfloat16, __nv_bfloat16>, grid, 256, 0, st, a);
    else MOE_LAUNCH(k_gate_bwd<EPL, SOFTMAX, __nv_bfloat16, float>, grid, 256, 0, st, a);
  } else {
    if (d.grad_dtype == MOE_BF16) MOE_LAUNCH(k_gate_bwd<EPL, SOFTMAX, float, __nv_bfloat16>, grid, 256, 0, st, a);
    else MOE_LAUNCH(k_gate_bwd<EPL, SOFTMAX, float, float>, grid, 256, 0, st, a);
  }
  return cudaSuccess;
}

template <int EPL, bool SOFTMAX, typename TL>
cudaError_t fwd_typed(const moe_gate_dims& d, const GateArgs& a, cudaStream_t st, int* launches) {
  // As many tokens as one cluster of full blocks holds are routed and counted by it; more by blocks
  // of eight and a second kernel for the counts. (Without counts: eight a block.)
  constexpr int kTokens = one_block_tokens<EPL>;
  const bool one = a.count && d.T <= kTokens * kCountBlocks;
  const int warps = one ? (int)std::min<int64_t>(d.T, kTokens) : 8;
  unsigned grid = (unsigned)((d.T + warps - 1) / warps);
  *launches += 1;
  if (one) {
    while (grid & (grid - 1)) ++grid;  // clusters of 1, 2, 4 or 8 blocks (one may have no token)
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    unsigned n = 0;
    if (MOE_PDL) {
      at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (grid > 1) {
      at[n].id = cudaLaunchAttributeClusterDimension;
      at[n].val.clusterDim.x = grid;
      at[n].val.clusterDim.y = 1;
      at[n++].val.clusterDim.z = 1;
    }
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)warps * 32);
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, k_gate_fwd<EPL, SOFTMAX, TL>, a);
  }
  // (a small grid without counts must not take itself for the counting cluster: a.count is null)
  MOE_LAUNCH(k_gate_fwd<EPL, SOFTMAX, TL>, grid, warps * 32, 0, st, a);
  if (a.count) {
    *launches += 1;
    MOE_LAUNCH(k_gate_count, kCountBlocks, 1024, 0, st, (const int*)a.idx, (int64_t)a.T * a.k, a.E, a.count);
  }
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
  a.L = 1;
  while (a.L * 2 * a.G <= 32) a.L *= 2;
  a.R = (a.per + a.L - 1) / a.L;
  const int V = d.dtype == MOE_BF16 ? 8 : 4;
  a.vec = a.E % V == 0 && a.per % V == 0 && a.R % V == 0;
  a.vec_bias = a.E % 4 == 0 && a.per % 4 == 0 && a.R % 4 == 0 && reinterpret_cast<uintptr_t>(bias) % 16 == 0;
  a.direct = !bias && (a.Kg == a.G || a.take == 1);
  return with_epl(a.R, [&](auto epl) {
    constexpr int EPL = decltype(epl)::value;
    if (d.dtype == MOE_BF16)
      return d.score == MOE_SCORE_SOFTMAX ? fwd_typed<EPL, true, __nv_bfloat16>(d, a, st, launches)
                                          : fwd_typed<EPL, false, __nv_bfloat16>(d, a, st, launches);
    return d.score == MOE_SCORE_SOFTMAX ? fwd_typed<EPL, true, float>(d, a, st, launches) : fwd_typed<EPL, false, float>(d, a, st, launches);
  });
}

cudaError_t launch_gate_bwd(const moe_gate_dims& d, const void* logits, const int* topk_idx, const float* dw,
                            void* dlogits, int sms, cudaStream_t st, int* launches) {
  GateArgs a = args_of(d);
  a.logits = logits;
  a.idx_in = topk_idx;
  a.dw = dw;
  a.dlogits = dlogits;
  // groups play no part here: R consecutive experts a lane, in whole 16-byte pieces where E allows
  a.R = (a.E + 31) / 32;
  const int V = d.dtype == MOE_BF16 || d.grad_dtype == MOE_BF16 ? 8 : 4;
  a.vec = a.E % V == 0;
  if (a.vec) a.R = (a.R + V - 1) / V * V;
  *launches += 1;
  return with_epl(a.R, [&](auto epl) {
    constexpr int EPL = decltype(epl)::value <= 32 ? decltype(epl)::value : 32;  // E <= 1024
    return d.score == MOE_SCORE_SOFTMAX ? bwd_typed<EPL, true>(d, a, st) : bwd_typed<EPL, false>(d, a, st);
  });
}

}  // namespace moe
