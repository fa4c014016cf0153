// balance.cu -- balance loss and z loss of router logits, forward and backward.
//
// With p = softmax(l), or sigmoid(l) over their sum, n_s the tokens of sequence s, N those of all sequences:
//   count_se = chosen experts, prob_se = mean of p over the sequence,
//   loss = alpha E / (k N) sum_se count_se prob_se,   z loss = z / N sum_t lse_t^2,
//   dl = p (1 - sigma) (c - p.c) + 2 z / N lse p   with c_e = alpha E / (k N) count_se / n_s  ((1 - sigma): sigmoid only).
//
// Forward: tokens are cut into chunks of equal length, a block each; a block walks the sequences that its chunk
// meets and writes one row of sums (p, counts, lse^2) for each. Row c + s holds chunk c of sequence s: along the
// tokens either index only grows, so no two share a row and chunks + S rows are enough. A second kernel adds a
// sequence's rows in order, so results do not depend on timing. Few tokens of one or two sequences are one block's and
// need neither rows nor a second kernel.
//
// Exponentials and reciprocals are the hardware's, for fp32 logits too (with expf and divisions 16384 x 256 in 37 sequences
// 16.2 us for 13.2, backward of 8192 x 128 4.0 for 3.8). A score is off by 2^-22 of itself and, since the exponent's argument is
// rounded, by 2^-23 for each unit that its logit is below the row's largest: 1e-6 of itself at 8, and where it is off by
// more it is small beside the others. One below 2^-126 is zero.
//
// Bound by what a warp does for a token and by latency, not by HBM: 16384 x 256 in 37 sequences 13 us (17 MB are 2.6),
// 64 x 128 4.2, backward of 8192 x 128 3.8.
#include <algorithm>
#include <type_traits>

#include "act.cuh"
#include "block.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = 8;  // of a block of the backward

struct BalanceArgs {
  const void* logits;
  const int* idx;
  const int* start;   // [S + 1] or null
  int T, E, k, S;
  int R, vec;         // experts of a lane; whether in fours
  int chunk, chunks;
  bool one;           // a single block: its sums are the results
  float alpha, z;
  float* row_p;       // [chunks + S][E]
  int* row_n;         // [chunks + S][E]
  float* row_z;       // [chunks + S]
  float* part;        // [S * column blocks][2]: parts of the losses
  unsigned* done;
  int* status;
  float* loss;
  int* count;
  float* prob;
  // backward
  const int* count_in;
  const float* dloss;
  const void* add;
  void* dlogits;
};

__device__ __forceinline__ int seq_at(const BalanceArgs& a, int s) {
  return a.start ? min(max(a.start[s], 0), a.T) : (s ? a.T : 0);
}
// The last sequence that begins at or before token t (the first if none does), by the whole warp: 32 offsets are looked
// at together, since each look waits for memory. Offsets that are not ascending give some sequence in [0, S).
__device__ __forceinline__ int seq_of(const BalanceArgs& a, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = a.S;
  while (n > 1) {
    const int step = (n + 31) / 32, at = lane * step;
    const uint32_t before = __ballot_sync(kFull, at < n && (lane == 0 || seq_at(a, lo + at) <= t));
    const int skip = (__popc(before) - 1) * step;
    lo += skip;
    n = min(step, n - skip);
  }
  return lo;
}
__device__ __forceinline__ float tokens_of_all(const BalanceArgs& a) {
  return fmaxf(1.0f, (float)(seq_at(a, a.S) - seq_at(a, 0)));
}

// A lane's experts: slot i holds expert first + (i / 4) 128 + (i % 4) step, four neighbours or every 32nd, so that a warp's
// accesses are of whole lines (backward of 65536 x 1024 100 us, with a lane's experts next to each other 373; of
// 8192 x 128 3.8 and 4.9).
struct Lane {
  int first, step, E;
  __device__ __forceinline__ Lane(const BalanceArgs& a)
      : first((threadIdx.x & 31) * (a.vec ? 4 : 1)), step(a.vec ? 1 : 32), E(a.E) {}
  __device__ __forceinline__ int at(int i) const { return first + (i >> 2) * 128 + (i & 3) * step; }
  __device__ __forceinline__ bool has(int i) const { return at(i) < E; }
};

// Four neighbouring values at p, 16 bytes of floats or 8 of bf16.
template <typename T>
using Quad = std::conditional_t<sizeof(T) == 4, uint4, uint2>;

// The lane's logits of a row; NaN masks its expert as -inf does.
template <int EPL, typename TL>
__device__ __forceinline__ void load_row(const TL* row, const Lane& x, bool vec, float (&l)[EPL]) {
  bool done = false;
  if constexpr (EPL % 4 == 0) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < EPL; i += 4) {
        Quad<TL> u = {};
        if (x.has(i)) u = *reinterpret_cast<const Quad<TL>*>(row + x.at(i));
        const TL* e = reinterpret_cast<const TL*>(&u);
#pragma unroll
        for (int q = 0; q < 4; ++q) l[i + q] = x.has(i) ? io<TL>::to_f(e[q]) : -INFINITY;
      }
      done = true;
    }
  }
  if (!done) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = x.has(i) ? io<TL>::to_f(row[x.at(i)]) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) l[i] = fmaxf(l[i], -INFINITY);  // of NaN and a number: the number
}

// Whether a row has a z loss: not where every logit is masked, by -inf or by its type's lowest value (the square of
// such an lse is no float), nor where one is +inf.
__device__ __forceinline__ bool has_lse(float lse) { return fabsf(lse) < 9.2e18f; }

__device__ __forceinline__ float warp_max(float v) {
  const uint32_t u = __float_as_uint(v), key = u & 0x80000000u ? ~u : u | 0x80000000u;
  const uint32_t m = __reduce_max_sync(kFull, key);
  return __uint_as_float(m & 0x80000000u ? m ^ 0x80000000u : ~m);
}

// l becomes p. softmax: returns the row's lse (not finite where the row has no finite logit, or a +inf). sigmoid:
// away (where given) receives 1 - sigma; scores are taken relative to the largest, so that a row of logits far
// below zero, whose scores are denormal, has a sum that can be divided by. A masked row is all zeros.
template <int EPL, bool SOFTMAX>
__device__ __forceinline__ float probs(float (&l)[EPL], float* away) {
  float m = l[0], sum = 0.0f;
#pragma unroll
  for (int i = 1; i < EPL; ++i) m = fmaxf(m, l[i]);
  if constexpr (SOFTMAX) {
    m = warp_max(m);
    if (fabsf(m) < INFINITY) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) sum += l[i] = ex2_approx((l[i] - m) * kLog2e);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) sum += l[i] = l[i] == INFINITY ? 1.0f : 0.0f;
    }
  } else {
    float low = 0.0f;
    if (!__any_sync(kFull, m >= 0.0f)) {  // the whole row is below zero
      m = warp_max(m);
      if (m > -INFINITY) low = m;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      float e = ex2_approx(-kLog2e * fabsf(l[i]));
      const float r = rcp_approx(1.0f + e);  // sigma(|l|)
      if (away) away[i] = l[i] > 0.0f ? e * r : r;
      if (low < 0.0f) e = ex2_approx((l[i] - low) * kLog2e);
      l[i] = l[i] > 0.0f ? r : e * r;
      sum += l[i];
    }
  }
  sum = warp_sum(sum);
  const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int i = 0; i < EPL; ++i) l[i] *= inv;
  return SOFTMAX ? m + logf(sum) : 0.0f;
}

// The rows of sequence s added for experts e0 .. e0 + COLS - 1, a column a lane and 32 / COLS rows a warp at a time.
// Returns the columns' sum of count prob (warp 0).
template <int WARPS, int COLS>
__device__ __forceinline__ float sum_columns(const BalanceArgs& a, int s, int e0, float (*sp)[COLS], int (*sn)[COLS]) {
  constexpr int kRows = WARPS * 32 / COLS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cx = lane % COLS, ry = threadIdx.x / COLS, e = e0 + cx;
  const int t0 = seq_at(a, s), t1 = seq_at(a, s + 1);
  const int r0 = t0 < t1 ? t0 / a.chunk + s : 0, r1 = t0 < t1 ? (t1 - 1) / a.chunk + s + 1 : 0;
  float p = 0.0f, dot = 0.0f;
  int c = 0;
  if (e < a.E) {
#pragma unroll 4
    for (int r = r0 + ry; r < r1; r += kRows) {
      p += __ldcg(a.row_p + (int64_t)r * a.E + e);
      c += __ldcg(a.row_n + (int64_t)r * a.E + e);
    }
  }
#pragma unroll
  for (int o = COLS; o < 32; o <<= 1) {
    p += __shfl_xor_sync(kFull, p, o);
    c += __shfl_xor_sync(kFull, c, o);
  }
  if (lane < COLS) {
    sp[warp][cx] = p;
    sn[warp][cx] = c;
  }
  __syncthreads();
  if (warp == 0) {
    if (lane < COLS && e < a.E) {
#pragma unroll
      for (int w = 1; w < WARPS; ++w) {
        p += sp[w][cx];
        c += sn[w][cx];
      }
      p /= (float)max(t1 - t0, 1);
      a.count[(int64_t)s * a.E + e] = c;
      if (a.prob) a.prob[(int64_t)s * a.E + e] = p;
      dot = (float)c * p;
    }
    dot = warp_sum(dot);
  }
  return dot;
}

// Warp 0: the sum of lse^2 over the rows of sequence s.
__device__ __forceinline__ float sum_z(const BalanceArgs& a, int s) {
  const int t0 = seq_at(a, s), t1 = seq_at(a, s + 1);
  float z = 0.0f;
  if (t0 < t1)
    for (int r = t0 / a.chunk + s + (int)threadIdx.x; r <= (t1 - 1) / a.chunk + s; r += 32) z += __ldcg(a.row_z + r);
  return warp_sum(z);
}

__device__ __forceinline__ void check_seq(const BalanceArgs& a, int s) {
  if (a.start && threadIdx.x == 0 && (a.start[s] > a.start[s + 1] || a.start[s] < 0 || a.start[s + 1] > a.T))
    set_status(a.status, MOE_ERR_DEVICE_ARG);
}

__device__ __forceinline__ void store_losses(const BalanceArgs& a, float dot, float z) {
  const float N = tokens_of_all(a);
  a.loss[0] = dot * (a.alpha * ((float)a.E / (float)a.k) / N);
  a.loss[1] = z * (a.z / N);
}

// Whether this is the last block of the grid; what the others' first threads wrote before is visible to it.
__device__ __forceinline__ bool last_block(unsigned* done) {
  __shared__ bool last;
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(done, 1u) == gridDim.x * gridDim.y - 1;
    if (last) *done = 0;
    __threadfence();
  }
  __syncthreads();
  return last;
}

template <int EPL, bool SOFTMAX, typename TL, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) k_balance_fwd(const BalanceArgs a) {
  extern __shared__ float shared[];  // [WARPS][E] sums of p, [E] counts
  int* hist = reinterpret_cast<int*>(shared + WARPS * a.E);
  __shared__ float zsum[WARPS];
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Lane x(a);
  const int c0 = (int)blockIdx.x * a.chunk, c1 = min(c0 + a.chunk, a.T);
  const TL* logits = reinterpret_cast<const TL*>(a.logits);
  float dot = 0.0f, z_all = 0.0f;  // of the only block
  // Towards L2 while the sequences are looked for: a lane 128 bytes of the warp's rows and of the indices. Of short chunks
  // alone (rows not in L2: 64 x 128 4.9 us without, 4.6 with; 4096 x 64 in 8 sequences 11.0, 10.0; 16384 x 256 in 37, 27
  // rows a chunk, 15.0, 14.9). In longer ones the next row's loads, which are always under way, do better than requests for
  // all of them at once (32768 x 256, 54 rows a chunk, 17.4, 18.8; 65536 x 1024 60, 71; 2^20 x 256 245, 305).
  if (a.chunk <= 4 * WARPS) {
    for (int t = c0 + warp; t < c1; t += WARPS)
      if (lane * (128 / (int)sizeof(TL)) < a.E)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const TL*>(a.logits) + (int64_t)t * a.E + lane * (128 / sizeof(TL))));
    for (int64_t i = (int64_t)c0 * a.k + threadIdx.x * 32; i < (int64_t)c1 * a.k; i += WARPS * 32 * 32)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.idx + i));
  }
  for (int s = seq_of(a, c0); s < a.S;) {
    const int b0 = max(c0, seq_at(a, s)), b1 = min(c1, seq_at(a, s + 1));
    if (seq_at(a, s) >= c1) break;
    if (b0 >= b1) {  // past a run of empty sequences at once
      s = max(s + 1, seq_of(a, b0));
      continue;
    }
    for (int i = threadIdx.x; i < a.E; i += blockDim.x) hist[i] = 0;
    float acc[EPL], z = 0.0f, next[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] = 0.0f;
    if (b0 + warp < b1) load_row<EPL>(logits + (int64_t)(b0 + warp) * a.E, x, a.vec, next);
    for (int t = b0 + warp; t < b1; t += WARPS) {
      float l[EPL];
#pragma unroll
      for (int i = 0; i < EPL; ++i) l[i] = next[i];
      if (t + WARPS < b1) load_row<EPL>(logits + (int64_t)(t + WARPS) * a.E, x, a.vec, next);
      const float lse = probs<EPL, SOFTMAX>(l, nullptr);
      if (SOFTMAX && has_lse(lse)) z += lse * lse;
#pragma unroll
      for (int i = 0; i < EPL; ++i) acc[i] += l[i];
    }
    if (lane == 0) zsum[warp] = z;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (x.has(i)) shared[warp * a.E + x.at(i)] = acc[i];
    __syncthreads();
    const int64_t i1 = (int64_t)b1 * a.k;
    for (int64_t i = (int64_t)b0 * a.k + threadIdx.x; i < i1; i += blockDim.x) {
      const int e = a.idx[i];
      if ((unsigned)e < (unsigned)a.E) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    const int64_t row = (int64_t)blockIdx.x + s;
    for (int i = threadIdx.x; i < a.E; i += blockDim.x) {
      float v = shared[i];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) v += shared[w * a.E + i];
      if (a.one) {  // these are the sequence's sums
        v /= (float)(b1 - b0);
        dot += (float)hist[i] * v;
        a.count[(int64_t)s * a.E + i] = hist[i];
        if (a.prob) a.prob[(int64_t)s * a.E + i] = v;
      } else {
        a.row_p[row * a.E + i] = v;
        a.row_n[row * a.E + i] = hist[i];
      }
    }
    if (threadIdx.x == 0) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) v += zsum[w];
      if (a.one) z_all += v;
      else a.row_z[row] = v;
    }
    __syncthreads();
    ++s;
  }
  if (!a.one) return;
  for (int s = 0; s < a.S; ++s) {
    check_seq(a, s);
    if (seq_at(a, s) < seq_at(a, s + 1)) continue;
    for (int i = threadIdx.x; i < a.E; i += blockDim.x) {
      a.count[(int64_t)s * a.E + i] = 0;
      if (a.prob) a.prob[(int64_t)s * a.E + i] = 0.0f;
    }
  }
  dot = warp_sum(dot);
  if (lane == 0) zsum[warp] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < WARPS; ++w) dot += zsum[w];
    store_losses(a, dot, z_all);
  }
}

// A block COLS experts of a sequence: its rows added; the last block adds the parts of the losses in a fixed order.
template <int kSumWarps, int COLS>
__global__ void __launch_bounds__(kSumWarps * 32) k_balance_sum(const BalanceArgs a) {
  __shared__ float sp[kSumWarps][COLS];
  __shared__ int sn[kSumWarps][COLS];
  __shared__ float2 red[kSumWarps];
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const int s = (int)blockIdx.x, at = s * (int)gridDim.y + (int)blockIdx.y;
  if (blockIdx.y == 0) check_seq(a, s);
  const float dot = sum_columns<kSumWarps, COLS>(a, s, (int)blockIdx.y * COLS, sp, sn);
  if (threadIdx.x < 32) {
    const float z = blockIdx.y == 0 ? sum_z(a, s) : 0.0f;
    if (threadIdx.x == 0) {
      a.part[2 * at] = dot;
      a.part[2 * at + 1] = z;
    }
  }
  if (!last_block(a.done)) return;
  float2 v = make_float2(0.0f, 0.0f);
  for (int i = threadIdx.x; i < (int)(gridDim.x * gridDim.y); i += kSumWarps * 32) {
    v.x += __ldcg(a.part + 2 * i);
    v.y += __ldcg(a.part + 2 * i + 1);
  }
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kSumWarps; ++w) {
      v.x += red[w].x;
      v.y += red[w].y;
    }
    store_losses(a, v.x, v.y);
  }
}

// A warp a token.
template <int EPL, bool SOFTMAX, typename TL, typename TG>
__global__ void __launch_bounds__(kWarps * 32) k_balance_bwd(const BalanceArgs a) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const int t = (int)blockIdx.x * kWarps + (int)(threadIdx.x >> 5);
  if (t >= a.T) return;
  const Lane x(a);
  const int64_t o = (int64_t)t * a.E;
  const int s = seq_of(a, t), t0 = seq_at(a, s), t1 = seq_at(a, s + 1);
  float l[EPL];
  if (t >= t0 && t < t1) {
    const float N = tokens_of_all(a), up = a.dloss ? *a.dloss : 1.0f;
    load_row<EPL>(reinterpret_cast<const TL*>(a.logits) + o, x, a.vec, l);
    float away[SOFTMAX ? 1 : EPL];
    const float lse = probs<EPL, SOFTMAX>(l, SOFTMAX ? nullptr : away);
    const float f = up * a.alpha * ((float)a.E / (float)a.k) / N / (float)(t1 - t0);
    float c[EPL], dot = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      c[i] = x.has(i) ? f * (float)a.count_in[(int64_t)s * a.E + x.at(i)] : 0.0f;
      dot += l[i] * c[i];
    }
    dot = warp_sum(dot);
    const float zf = SOFTMAX && has_lse(lse) ? up * 2.0f * a.z / N * lse : 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if constexpr (SOFTMAX) l[i] *= c[i] - dot + zf;
      else l[i] *= away[i] * (c[i] - dot);
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = 0.0f;
  }
  const TG* add = reinterpret_cast<const TG*>(a.add);
  TG* out = reinterpret_cast<TG*>(a.dlogits);
  if constexpr (EPL % 4 == 0) {
    if (a.vec) {
#pragma unroll
      for (int i = 0; i < EPL; i += 4) {
        if (!x.has(i)) break;
        Quad<TG> u;
        TG* q = reinterpret_cast<TG*>(&u);
        if (add) {
          u = *reinterpret_cast<const Quad<TG>*>(add + o + x.at(i));
#pragma unroll
          for (int j = 0; j < 4; ++j) l[i + j] += io<TG>::to_f(q[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = io<TG>::cvt(l[i + j]);
        *reinterpret_cast<Quad<TG>*>(out + o + x.at(i)) = u;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (x.has(i)) out[o + x.at(i)] = io<TG>::cvt(l[i] + (add ? io<TG>::to_f(add[o + x.at(i)]) : 0.0f));
}

// ---------------------------------------------------------------- host side
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
// One block takes what its warps get through in four tokens each, of at most two sequences, which it walks one after the
// other (64 tokens of 128 experts 4.2 us, 6.1 in two sequences, 30 in 16; in two kernels 6.0, 6.4 and 6.5). More go in
// chunks of 8-warp blocks, four an SM (16384 x 256 in 37 sequences 13 us; one block of 32 warps an SM 17), of two
// tokens a warp, or as many as a sequence has.
constexpr int kChunkBlocks = 608;
constexpr int kChunkWarps = 8;
int one_block_warps(int64_t E) { return E <= 256 ? 32 : E <= 512 ? 16 : 8; }  // as many as hold their sums in 32 KB
bool one_block(const moe_balance_dims& d) { return d.T <= 4 * one_block_warps(d.E) && d.S <= 2; }
int chunk_tokens(const moe_balance_dims& d) {
  if (one_block(d)) return (int)d.T;
  const int64_t each = std::clamp<int64_t>(d.T / std::max<int64_t>(d.S, 1), 1, 2 * kChunkWarps);
  return (int)std::max<int64_t>(each, (d.T + kChunkBlocks - 1) / kChunkBlocks);
}

struct BalanceWs {
  size_t p, n, z, part, total;
};
BalanceWs layout(const moe_balance_dims& d) {
  const size_t c = chunk_tokens(d), S = (size_t)std::max<int64_t>(d.S, 1), rows = ((size_t)d.T + c - 1) / c + S;
  BalanceWs L;
  size_t o = kBalanceHeader;
  L.p = o;
  o += up256(rows * d.E * 4);
  L.n = o;
  o += up256(rows * d.E * 4);
  L.z = o;
  o += up256(rows * 4);
  L.part = o;
  o += up256(S * ((d.E + 7) / 8) * 8);
  L.total = o;
  return L;
}

template <typename F>
cudaError_t with_epl(int R, F f) {
  if (R <= 1) return f(std::integral_constant<int, 1>());
  if (R <= 2) return f(std::integral_constant<int, 2>());
  if (R <= 4) return f(std::integral_constant<int, 4>());
  if (R <= 8) return f(std::integral_constant<int, 8>());
  if (R <= 16) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());  // E <= 1024
}

BalanceArgs args_of(const moe_balance_dims& d, const void* logits, const int* start) {
  BalanceArgs a = {};
  a.logits = logits;
  a.start = d.S ? start : nullptr;
  a.T = (int)d.T;
  a.E = (int)d.E;
  a.k = (int)d.k;
  a.S = (int)std::max<int64_t>(d.S, 1);
  a.alpha = d.alpha;
  a.z = d.z_coef;
  a.vec = a.E % 4 == 0 && a.E > 64;  // of up to 64, more lanes at work are better (65536 x 64 backward 20.6 us, in fours 23.1)
  a.R = a.vec ? (a.E + 127) / 128 * 4 : (a.E + 31) / 32;
  return a;
}

template <int EPL, bool SOFTMAX>
cudaError_t bwd_typed(const moe_balance_dims& d, const BalanceArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)((d.T + kWarps - 1) / kWarps);
  using bf = __nv_bfloat16;
  if (d.dtype == MOE_BF16) {
    if (d.grad_dtype == MOE_BF16) MOE_LAUNCH(k_balance_bwd<EPL, SOFTMAX, bf, bf>, grid, kWarps * 32, 0, st, a);
    else MOE_LAUNCH(k_balance_bwd<EPL, SOFTMAX, bf, float>, grid, kWarps * 32, 0, st, a);
  } else {
    if (d.grad_dtype == MOE_BF16) MOE_LAUNCH(k_balance_bwd<EPL, SOFTMAX, float, bf>, grid, kWarps * 32, 0, st, a);
    else MOE_LAUNCH(k_balance_bwd<EPL, SOFTMAX, float, float>, grid, kWarps * 32, 0, st, a);
  }
  return cudaSuccess;
}

template <int EPL, bool SOFTMAX, typename TL>
cudaError_t fwd_launch(const BalanceArgs& a, cudaStream_t st) {
  constexpr int W = EPL <= 8 ? 32 : EPL <= 16 ? 16 : 8;  // one_block_warps of every E that comes here
  if (a.one)
    MOE_LAUNCH(k_balance_fwd<EPL, SOFTMAX, TL, W>, 1, W * 32, (size_t)a.E * 4 * (W + 1), st, a);
  else
    MOE_LAUNCH(k_balance_fwd<EPL, SOFTMAX, TL, kChunkWarps>, a.chunks, kChunkWarps * 32, (size_t)a.E * 4 * (kChunkWarps + 1), st, a);
  return cudaSuccess;
}
template <int EPL, bool SOFTMAX>
cudaError_t fwd_typed(const moe_balance_dims& d, const BalanceArgs& a, cudaStream_t st) {
  return d.dtype == MOE_BF16 ? fwd_launch<EPL, SOFTMAX, __nv_bfloat16>(a, st) : fwd_launch<EPL, SOFTMAX, float>(a, st);
}

}  // namespace

size_t balance_workspace_bytes(const moe_balance_dims& d) { return layout(d).total; }

cudaError_t launch_balance_fwd(const moe_balance_dims& d, void* ws, const void* logits, const int* topk_idx,
                               const int* seq_start, float* loss, int* count, float* prob, cudaStream_t st,
                               int* launches) {
  BalanceArgs a = args_of(d, logits, seq_start);
  const BalanceWs L = layout(d);
  char* w = static_cast<char*>(ws);
  a.idx = topk_idx;
  a.chunk = chunk_tokens(d);
  a.chunks = (a.T + a.chunk - 1) / a.chunk;
  a.one = one_block(d);
  a.row_p = reinterpret_cast<float*>(w + L.p);
  a.row_n = reinterpret_cast<int*>(w + L.n);
  a.row_z = reinterpret_cast<float*>(w + L.z);
  a.part = reinterpret_cast<float*>(w + L.part);
  a.status = reinterpret_cast<int*>(w);
  a.done = reinterpret_cast<unsigned*>(w + 64);
  a.loss = loss;
  a.count = count;
  a.prob = prob;
  *launches += a.one ? 1 : 2;
  const cudaError_t e = with_epl(a.R, [&](auto epl) {
    constexpr int EPL = decltype(epl)::value;
    return d.score == MOE_SCORE_SOFTMAX ? fwd_typed<EPL, true>(d, a, st) : fwd_typed<EPL, false>(d, a, st);
  });
  if (e != cudaSuccess || a.one) return e;
  // few sequences have many rows each: 128 of them at a time, eight columns a block (8192 x 128 in one sequence 9.0 us
  // with the first kernel; as below 13). Many have few (16384 x 256 in 37 sequences 13; as above 23)
  if (a.chunks >= 64 * a.S) MOE_LAUNCH((k_balance_sum<32, 8>), dim3((unsigned)a.S, (unsigned)((a.E + 7) / 8)), 1024, 0, st, a);
  else MOE_LAUNCH((k_balance_sum<8, 32>), dim3((unsigned)a.S, (unsigned)((a.E + 31) / 32)), 256, 0, st, a);
  return cudaSuccess;
}

cudaError_t launch_balance_bwd(const moe_balance_dims& d, const void* logits, const int* count, const int* seq_start,
                               const float* dloss, const void* dlogits_add, void* dlogits, cudaStream_t st,
                               int* launches) {
  BalanceArgs a = args_of(d, logits, seq_start);
  a.count_in = count;
  a.dloss = dloss;
  a.add = dlogits_add;
  a.dlogits = dlogits;
  *launches += 1;
  return with_epl(a.R, [&](auto epl) {
    constexpr int EPL = decltype(epl)::value;
    return d.score == MOE_SCORE_SOFTMAX ? bwd_typed<EPL, true>(d, a, st) : bwd_typed<EPL, false>(d, a, st);
  });
}

}  // namespace moe
