// xent.cu -- softmax cross entropy of l = x w over a large vocabulary, and its gradients.
//
//   lse = log sum_v e^l;  loss = lse - l_target + z lse^2;  dl = d ((1 + 2 z lse) e^{l - lse} - onehot);
//   dx = dl w^T;  dw = x^T dl.
//
// bf16: the tensor-core products' epilogue turns a tile of logits into the rows' statistics (largest, sum of
// exponentials), or into dl, before anything is stored; the forward is one product over the whole vocabulary, the
// backward takes it a piece at a time: dl of the piece, then its two products. Bound by the products: 4096 x 2048 x 131072
// 5.4 to 5.6 ms (8 M H V flops at 1.6 PFLOP/s); statistics 1.15 ms by themselves, dl of 32768 columns 0.3. A few rows are a
// stream of w: 8 x 2048 x 65536 51 us, 44 of them at 6.1 TB/s. The target's logit is summed in fp32 on the CUDA cores:
// tensor cores truncate as they add, and a target's products are mostly of one sign. fp32: the logits of a piece are
// stored, then read.
#include <algorithm>

#include "act.cuh"
#include "block.h"
#include "common.cuh"
#include "linear_choice.h"
#include "linear_f32.h"
#include "linear_tc.h"

namespace moe {
namespace {

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int64_t up64(int64_t n) { return (n + 63) / 64 * 64; }
// Row lengths of the matrices that the products read. bf16: TMA wants multiples of 16 bytes, so odd rows are copied; a
// copy's rows are whole 128-byte lines, which a box's rows then do not straddle. x is copied for that alone where it is
// small beside the products (777 x 1000 x 50001 with an embedding table 331 -> 311 us; a copy of w as well 423).
int64_t row_of_w(const moe_xent_dims& d) {
  const int64_t C = d.tied ? d.H : d.V;
  return d.dtype == MOE_BF16 && C % 8 ? up64(C) : C;
}
int64_t row_of_x(const moe_xent_dims& d) {
  return d.dtype == MOE_BF16 && (d.H % 8 || (d.H % 64 && d.M >= 256 && d.V >= 8192)) ? up64(d.H) : d.H;
}

// (m, s) joined with (m2, s2): s e^m is the sum of both.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float big = fmaxf(m, m2);
  if (big == -INFINITY) return;  // both empty
  s = s * expf(m - big) + s2 * expf(m2 - big);
  m = big;
}

// A block a row: the piece's largest logit and sum joined to what earlier pieces left; the target's logit where it is
// among the piece's.
__global__ void __launch_bounds__(256) k_xent_piece(const float* l, int64_t ld, int cols, int v0, const int* target,
                                                    float2* stat, float* at_target, int first) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  __shared__ float2 red[8];
  const int64_t t = blockIdx.x;
  const float* row = l + t * ld;  // 16-byte aligned, as every row is
  float m = -INFINITY, s = 0.0f;
  constexpr int U = 4;  // 16-byte loads in flight
  for (int i0 = threadIdx.x * 4; i0 < cols; i0 += U * 1024) {
    float v[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * 1024;
      const float4 q = i < cols ? *reinterpret_cast<const float4*>(row + i) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      v[u][0] = q.x;
      v[u][1] = i + 1 < cols ? q.y : -INFINITY;
      v[u][2] = i + 2 < cols ? q.z : -INFINITY;
      v[u][3] = i + 3 < cols ? q.w : -INFINITY;
    }
    float big = m;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) big = fmaxf(big, v[u][j]);
    const float at = big == -INFINITY ? 0.0f : big;  // nothing but -inf so far: e^{-inf} = 0, and NaN stays
    s = m == -INFINITY ? s : s * expf(m - at);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) s += expf(v[u][j] - at);
    m = big;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    join(m, s, m2, s2);
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) join(m, s, red[w].x, red[w].y);
    if (!first) join(m, s, stat[t].x, stat[t].y);
    stat[t] = make_float2(m, s);
    const int64_t c = (int64_t)target[t] - v0;
    if (c >= 0 && c < cols) at_target[t] = row[c];
  }
}

// Eight rows' slots [first, end) of stat[slot][M] joined by a block, four slots of eight rows a warp; BASE2: a slot is
// (largest logit times log2 e, sum of powers of two), else of e. Warp i < 8 holds row i's result.
constexpr int kLossRows = 8, kLossWarps = 32;
template <bool BASE2>
__device__ __forceinline__ float2 join_slots(const float2* stat, int first, int end, int M, int64_t t0, float2 (*red)[kLossRows]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane & 7;
  const auto both = [](float& m, float& s, float m2, float s2) {
    if constexpr (BASE2) {
      const float big = fmaxf(m, m2);
      s = s * ex2_approx(m - big) + s2 * ex2_approx(m2 - big);
      m = big;
    } else {
      join(m, s, m2, s2);
    }
  };
  float m = BASE2 ? -3.0e38f : -INFINITY, s = 0.0f;
  if (t0 + r < M) {
#pragma unroll 8
    for (int i = first + warp * 4 + (lane >> 3); i < end; i += 4 * kLossWarps) {
      const float2 v = stat[(int64_t)i * M + t0 + r];
      both(m, s, v.x, v.y);
    }
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    both(m, s, m2, s2);
  }
  if (lane < 8) red[warp][lane] = make_float2(m, s);
  __syncthreads();
  if (warp < kLossRows) {
    const float2 v = red[lane][warp];
    m = v.x;
    s = v.y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      both(m, s, m2, s2);
    }
  }
  return make_float2(m, s);
}

// Slots [first, end) joined into slot 0.
__global__ void __launch_bounds__(kLossWarps * 32) k_xent_fold(float2* stat, int first, int end, int M) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  __shared__ float2 red[kLossWarps][kLossRows];
  const int64_t t0 = (int64_t)blockIdx.x * kLossRows;
  const float2 v = join_slots<true>(stat, first, end, M, t0, red);
  const int row = threadIdx.x >> 5;
  if (row < kLossRows && (threadIdx.x & 31) == 0 && t0 + row < M) stat[t0 + row] = v;
}

struct LossArgs {
  const float2* stat;  // [slots][M]
  const float* at;     // [M], the targets' logits as the product has them
  const float* dots;   // BASE2: [M][parts], their sums in fp32
  int first, end, M, V, parts;
  const int* target;
  float z;
  float* loss;
  float* lse;
  float2* part;
  unsigned* done;
  float* total;
  int* status;
};

// The targets' logits of bf16 products in fp32, a warp 256 features of a row; a kernel of its own, so that the columns of w, a line for
// every feature, are fetched by all SMs (8 rows of 2048 features: 20 us in one block of k_xent_loss, 3 us here).
constexpr int kDotCols = 256;
__device__ __forceinline__ float dot_part(const __nv_bfloat16* x, const __nv_bfloat16* w, int64_t swh, int h0, int H) {
  const int lane = threadIdx.x & 31;
  float a[kDotCols / 32], b[kDotCols / 32], dot = 0.0f;
#pragma unroll
  for (int i = 0; i < kDotCols / 32; ++i) {
    const int h = h0 + i * 32 + lane;
    a[i] = h < H ? __bfloat162float(x[h]) : 0.0f;
    b[i] = h < H ? __bfloat162float(w[h * swh]) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kDotCols / 32; ++i) dot = fmaf(a[i], b[i], dot);
  return warp_sum(dot);
}
__global__ void __launch_bounds__(256) k_xent_dots(const __nv_bfloat16* x, const __nv_bfloat16* w, int64_t ldx, int64_t swh,
                                                   int64_t swv, const int* target, int M, int H, int V, int parts,
                                                   float* dots) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t t = at / parts;
  if (t >= M) return;
  const int v = target[t], h0 = (int)(at - t * parts) * kDotCols;
  const float dot = v >= 0 && v < V ? dot_part(x + t * ldx, w + v * swv, swh, h0, H) : 0.0f;
  if ((threadIdx.x & 31) == 0) dots[at] = dot;
}

// log(s 2^m) + more
__device__ __forceinline__ float lse_of(float m, float s, float more) {
  constexpr float kLn2 = 0.6931471805599453f;
  return fmaf(m, kLn2, fmaf(log2f(s), kLn2, more));
}

// lse and loss of a row from its sum s 2^m of powers of two, with the target's logit `at` in fp32 in place of the product's
// own, `had`, in that sum:  loss = log(1 + e^y), y = log(e^L - 1) + had - at,  L = log(s 2^m) - had. The difference to had
// is taken before the logarithm's rounding, so that a likely target's small loss keeps its digits; no exponential here can
// overflow and no logarithm sees a negative number, whatever had and at are off (lse + log(1 + e^{at - lse} - e^{had - lse})
// was NaN where a large had rounded lse away from itself).
__device__ __forceinline__ void corrected(float m, float s, float had, float at, float* lse, float* loss) {
  constexpr float kLn2 = 0.6931471805599453f;
  float L = kLn2 * (log2f(s) + fmaf(-had, kLog2e, m));
  if (L < 0.0f) L = 0.0f;                         // had is in the sum; NaN stays
  const float others = logf(-expm1f(-L));         // log of the others' share
  const float off = had == at ? 0.0f : had - at;  // of two infinities as well
  const float y = (L + others) + off;
  const float t = log1pf(expf(-fabsf(y)));
  // the larger of the target's and the others' parts, and what the other adds; the small terms first
  *loss = y > 0.0f ? L + ((others + t) + off) : t;
  *lse = y > 0.0f ? lse_of(m, s, others + t) : at + t;
}

// lse and loss of eight rows a block; with BASE2 the targets' logits are exchanged (corrected). The blocks' totals are
// added in order by the last one.
template <bool BASE2>
__global__ void __launch_bounds__(kLossWarps * 32) k_xent_loss(const LossArgs a) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  __shared__ float2 red[kLossWarps][kLossRows];
  __shared__ float2 rows[kLossRows];
  __shared__ float sums[kLossWarps];
  __shared__ int counts[kLossWarps];
  __shared__ bool last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = (int64_t)blockIdx.x * kLossRows;
  const int64_t t = t0 + warp;  // of the first eight warps
  int v = -1;
  float at = 0.0f, had = 0.0f;
  if (warp < kLossRows && t < a.M) {
    v = a.target[t];
    if (v >= 0 && v < a.V) had = a.at[t];
    if constexpr (BASE2) {
      for (int i = lane; i < a.parts; i += 32) at += a.dots[t * a.parts + i];
      at = warp_sum(at);
    } else {
      at = had;
    }
  }
  const float2 st = join_slots<BASE2>(a.stat, a.first, a.end, a.M, t0, red);
  if (warp < kLossRows && lane == 0) {
    float sum = 0.0f, n = 0.0f;
    if (t < a.M) {
      float e = BASE2 ? lse_of(st.x, st.y, 0.0f) : st.x + logf(st.y);
      if (v >= a.V) set_status(a.status, MOE_ERR_DEVICE_ARG);
      if (v >= 0 && v < a.V) {
        sum = e - at;
        if (BASE2) corrected(st.x, st.y, had, at, &e, &sum);
        sum += a.z * e * e;
        n = 1.0f;
      }
      a.lse[t] = e;
      a.loss[t] = sum;
    }
    rows[warp] = make_float2(sum, n);
  }
  if (!a.total) return;
  __syncthreads();
  if (threadIdx.x == 0) {
    float sum = 0.0f, n = 0.0f;
#pragma unroll
    for (int i = 0; i < kLossRows; ++i) {
      sum += rows[i].x;
      n += rows[i].y;
    }
    if (gridDim.x == 1) {
      a.total[0] = sum;
      a.total[1] = n;
    } else {
      a.part[blockIdx.x] = make_float2(sum, n);
      __threadfence();
      last = atomicAdd(a.done, 1u) == gridDim.x - 1;
      __threadfence();
    }
  }
  if (gridDim.x == 1) return;
  __syncthreads();
  if (!last) return;
  // a thread's blocks in order, then trees: every sum of losses is of few and equal terms, the rows are counted as integers
  float sum = 0.0f;
  int n = 0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += kLossWarps * 32) {
    const float2 p = __ldcg(a.part + i);
    sum += p.x;
    n += (int)p.y;
  }
  sum = warp_sum(sum);
  n = (int)__reduce_add_sync(0xffffffffu, (unsigned)n);
  if (lane == 0) {
    sums[warp] = sum;
    counts[warp] = n;
  }
  __syncthreads();
  if (warp == 0) {
    sum = warp_sum(sums[lane]);
    n = (int)__reduce_add_sync(0xffffffffu, (unsigned)counts[lane]);
    if (lane == 0) {
      a.total[0] = sum;
      a.total[1] = (float)n;
      *a.done = 0;
    }
  }
}

// What the rows' gradients are made of.
struct XentRows {
  const int* target;
  const float* lse;
  const float* dloss;
  const float* total;
  int V;
  float z;
};
__device__ __forceinline__ float row_grad(const XentRows& r, int64_t t) {
  const int v = r.target[t];
  if (v < 0 || v >= r.V) return 0.0f;
  return r.dloss ? r.dloss[t] : 1.0f / r.total[1];
}

// bf16: the targets' gradients (without the mean's factor) from the logits that the forward's lse has in it, in every bit:
// k_xent_dots' parts in k_xent_loss' order. With the products' own logits the errors of the two do not cancel, and p - 1
// of a target was off by 5% at p = 1 - 9e-5 and by 13% at 1 - 5e-5; here by what lse's rounding is. A block a row.
__global__ void __launch_bounds__(256) k_xent_own(const __nv_bfloat16* x, const __nv_bfloat16* w, int64_t ldx, int64_t swh,
                                                  int64_t swv, XentRows r, int H, int parts, float* own) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  __shared__ float part[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x;
  const int v = r.target[t];
  if (v < 0 || v >= r.V) return;  // nobody reads it
  x += t * ldx;
  w += v * swv;
  float at = 0.0f;
  for (int p0 = 0; p0 < parts; p0 += 32) {
    for (int p = p0 + warp; p < min(parts, p0 + 32); p += 8) {
      const float dot = dot_part(x, w, swh, p * kDotCols, H);
      if (lane == 0) part[p - p0] = dot;
    }
    __syncthreads();
    if (warp == 0 && p0 + lane < parts) at += part[lane];
    __syncthreads();
  }
  if (warp) return;
  at = warp_sum(at);
  if (lane == 0) {
    const float d = r.dloss ? r.dloss[t] : 1.0f, lse = r.lse[t], u = at - lse;
    own[t] = d == 0.0f ? 0.0f : d * (expm1f(u) + 2.0f * r.z * lse * expf(u));  // f e^u - d
  }
}

// dl of a piece in place of its logits (fp32), a block 1024 columns of a row; zeros up to a multiple of four.
__global__ void __launch_bounds__(256) k_xent_dl(float* l, int64_t ld, int cols, int v0, XentRows r) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const int64_t t = blockIdx.x;
  const float d = row_grad(r, t), lse = r.lse[t], f = d * (1.0f + 2.0f * r.z * lse);
  const int at = r.target[t] - v0;
  for (int i = blockIdx.y * 1024 + threadIdx.x; i < min((cols + 3) / 4 * 4, ((int)blockIdx.y + 1) * 1024); i += 256) {
    const float p = d == 0.0f || i >= cols ? 0.0f : expf(l[t * ld + i] - lse) * f;
    l[t * ld + i] = i == at ? p - d : p;
  }
}

// dx from the sums of `parts` parts of K, in order, over *div where that is given.
__global__ void __launch_bounds__(256) k_xent_round(const float* a, __nv_bfloat16* o, int64_t n, int parts, const float* div) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const float by = div ? *div : 1.0f, f0 = by != 0.0f ? 1.0f / by : 0.0f;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n; i += (int64_t)gridDim.x * 1024) {
    float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n % 4 == 0) {  // a part begins at a 16-byte boundary
#pragma unroll 8
      for (int p = 0; p < parts; ++p) {
        const float4 v = *reinterpret_cast<const float4*>(a + p * n + i);
        f[0] += v.x;
        f[1] += v.y;
        f[2] += v.z;
        f[3] += v.w;
      }
      const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0] * f0, f[1] * f0), hi = __floats2bfloat162_rn(f[2] * f0, f[3] * f0);
      *reinterpret_cast<uint2*>(o + i) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
      for (int64_t j = i; j < min(n, i + 4); ++j) {
        float v = 0.0f;
        for (int p = 0; p < parts; ++p) v += a[p * n + j];
        o[j] = __float2bfloat16_rn(v * f0);
      }
    }
  }
}

// dx from the sums of fp32 parts, in order, added to what earlier pieces left (add).
__global__ void __launch_bounds__(256) k_xent_add(const float* a, float* o, int64_t n, int parts, int add) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    float v = 0.0f;
#pragma unroll 8
    for (int p = 0; p < parts; ++p) v += a[p * n + i];
    o[i] = add ? o[i] + v : v;
  }
}

// ---------------------------------------------------------------- host side
// Columns of a piece: a multiple of 256; about 2^27 values of dl in bf16, 2^24 logits in fp32 (4096 x 2048 x 131072
// 5.42 ms; with 2^26 5.60, 2^25 6.02, 2^28 5.38: the products of a piece have ragged last rounds).
int64_t piece_cols(const moe_xent_dims& d) {
  const int64_t want = std::max<int64_t>(1024, (1ll << (d.dtype == MOE_BF16 ? 27 : 24)) / d.M / 256 * 256);
  return std::min(want, up64(d.V));
}
// Parts of K of a piece's dx product in bf16: its K is a piece of the vocabulary and its tiles may be few. 0: as
// launch_xent_product does it, which is as good or better; else pairs of CTAs, each with a tile's part, whose fp32 sums are
// added afterwards (777 x 1000 over 50001 columns: 16 tiles for 76 pairs, 200 -> 93 us in 4 parts). Estimates as in
// linear_choice.h; a part costs its sums' way to memory and back.
int dx_parts(const moe_xent_dims& d) {
  constexpr int kSms = 152, kUnits = kSms / 2;
  const int64_t P = piece_cols(d);
  const int kb = (int)((std::min(P, d.V) + 63) / 64);
  const bool whole = P >= d.V;
  const double sums = (double)d.M * d.H * (whole ? 8 : 12) / 6.0e6;
  int best = 0;
  double t = choose_linear(d.M, d.H, std::min(P, d.V), false, kSms).us + (whole ? 0.0 : sums);
  const int64_t tiles = ((d.M + 255) / 256) * ((d.H + 255) / 256);
  for (int p = 1; p <= kUnits && kb / p >= 8; ++p) {
    const double rounds = (double)((tiles * p + kUnits - 1) / kUnits);
    const double e = 2.23 + rounds * (0.300 * ((kb + p - 1) / p) + 3.05) + p * sums + (whole ? 3.0 : 0.0);
    if (e < t) {
      t = e;
      best = p;
    }
  }
  return best;
}
// The same in fp32, 1: none but those that a cluster adds. While a cluster's part would last longer than the GPU's even
// share of both products, and than 32 steps, which its sums' way to memory and a launch cost (backward of
// 17 x 768 x 50257 505 -> 383 us, of 8 x 64 x 50257 280 -> 46).
int dx_parts_f32(const moe_xent_dims& d, int64_t cols) {
  constexpr int64_t kSlots = 152 * 4;
  const auto tiles = [](int64_t m, int64_t n) { return ((m + kF32Tile - 1) / kF32Tile) * ((n + kF32Tile - 1) / kF32Tile); };
  const auto steps = [](int64_t k) { return (k + kF32Slab - 1) / kF32Slab; };
  const int64_t all = tiles(d.M, d.H) * steps(cols) + tiles(d.H, cols) * steps(d.M);
  const int64_t most = std::max<int64_t>(all / kSlots, 32) * kF32Cluster;
  int parts = 1;
  while (parts < 64 && steps(cols) / parts > most) parts *= 2;
  return parts;
}
constexpr int kSlotCols = 64;  // the narrowest slot of the statistics
// Columns of a forward product in bf16: its statistics (with those of the columns before) stay below 256 MB, or 1 KB a row.
int64_t stat_cols(const moe_xent_dims& d) {
  return std::min(d.V, std::max<int64_t>(8192, (1ll << 31) / d.M / 256 * 256));
}

// Workspace: header, the rows' statistics, a piece's logits (fp32) or dl, dx in fp32, and copies of x and w with rows of a
// multiple of 16 bytes where the caller's are not.
struct XentWs {
  size_t stat, at, dots, part, piece, dx, xp, wp, total;
};
XentWs layout(const moe_xent_dims& d, bool backward) {
  const bool bf = d.dtype == MOE_BF16;
  const int64_t P = piece_cols(d), R = d.tied ? d.V : d.H, C = d.tied ? d.H : d.V;
  XentWs L;
  size_t o = kXentHeader;
  const auto take = [&](size_t bytes) {
    const size_t at = o;
    o += up256(bytes);
    return at;
  };
  L.stat = take((size_t)d.M * 8 * (bf ? 1 + (stat_cols(d) + kSlotCols - 1) / kSlotCols : 1));
  L.at = take((size_t)d.M * 4);
  L.dots = take(bf ? (size_t)d.M * ((d.H + kDotCols - 1) / kDotCols) * 4 : 0);
  L.part = take((size_t)((d.M + kLossRows - 1) / kLossRows) * 8);
  L.xp = take(row_of_x(d) != d.H ? (size_t)d.M * row_of_x(d) * 2 : 0);
  L.wp = take(row_of_w(d) != C ? (size_t)R * row_of_w(d) * 2 : 0);
  L.piece = take(bf ? (backward ? (size_t)d.M * P * 2 : 0) : (size_t)d.M * P * 4);
  const int parts = bf ? dx_parts(d) : dx_parts_f32(d, std::min(P, d.V));
  const bool sums = bf ? parts || d.V > P : parts > 1;
  L.dx = take(backward && sums ? (size_t)d.M * d.H * 4 * std::max(parts, 1) : 0);
  L.total = o;
  return L;
}

struct Xent {
  const moe_xent_dims& d;
  char* ws;
  XentWs L;
  const void* x;
  const void* w;
  int sms;
  cudaStream_t st;
  int* launches;
  int64_t P, ldx, ldw;

  // bf16: x and w with rows that TMA can read. fp32 reads them as they are (copies for 16-byte loads cost 22 us of
  // 500 x 768 x 10007, where a product's odd rows cost 12).
  cudaError_t prepare() {
    P = piece_cols(d);
    ldx = row_of_x(d);
    ldw = row_of_w(d);
    const cudaError_t e = launch_pack_rows(&x, ws + L.xp, d.M, d.H, ldx, sms, st, launches);
    if (e != cudaSuccess) return e;
    return launch_pack_rows(&w, ws + L.wp, d.tied ? d.V : d.H, d.tied ? d.H : d.V, ldw, sms, st, launches);
  }
  const void* w_at(int64_t v0) const {
    return static_cast<const char*>(w) + (d.tied ? v0 * ldw : v0) * (d.dtype == MOE_BF16 ? 2 : 4);
  }
  // the product of columns v0 .. v0 + cols - 1 of the logits
  XentGemm gemm(int64_t v0, int cols, void* out) const {
    return {{(int)d.M, cols, (int)d.H, x, w_at(v0), ldx, ldw, 0, !d.tied, nullptr, nullptr, out, nullptr, MOE_ACT_NONE, 0,
             reinterpret_cast<int*>(ws)}, P};
  }
  cudaError_t logits_f32(int64_t v0, int cols) {
    const int M = (int)d.M, H = (int)d.H;
    SimtGemm g = {static_cast<const float*>(x), static_cast<const float*>(w_at(v0)), ldx, 1, d.tied ? 1 : ldw,
                  d.tied ? ldw : 1, M, H, cols, nullptr, nullptr, piece(), nullptr, MOE_ACT_NONE, P};
    return launch_linear_f32(&g, 1, true, sms, st, launches);
  }
  static int up4(int n) { return (n + 3) / 4 * 4; }
  float* piece() const { return reinterpret_cast<float*>(ws + L.piece); }
  // div: bf16's dl is that of the sum of the losses, the products are divided by *div
  cudaError_t products(int64_t v0, int cols, void* dx, void* dw, const float* div) {
    const int M = (int)d.M, H = (int)d.H;
    if (d.dtype == MOE_BF16) {
      int* status = reinterpret_cast<int*>(ws);
      const void* dl = ws + L.piece;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(dw) + (dw ? (d.tied ? v0 * d.H : v0) : 0);
      const int parts = dx_parts(d);
      const bool direct = P >= d.V && !parts;
      XentGemm gx = {{M, H, cols, dl, w_at(v0), P, ldw, 0, d.tied, nullptr, nullptr, direct ? dx : ws + L.dx, nullptr,
                      MOE_ACT_NONE, !direct, status}, H, v0 > 0};
      if (direct) gx.div = div;
      if (parts) gx.parts = std::min(parts, (cols + 63) / 64);
      XentGemm gw = d.tied ? XentGemm{{cols, H, M, dl, x, P, ldx, 1, 1, nullptr, nullptr, out, nullptr, MOE_ACT_NONE, 0, status}}
                           : XentGemm{{H, cols, M, x, dl, ldx, P, 1, 1, nullptr, nullptr, out, nullptr, MOE_ACT_NONE, 0, status},
                                      d.V};
      gw.div = div;
      cudaError_t e = cudaSuccess;
      if (dx) {
        *launches += 1;
        e = parts ? launch_xent_parts(gx, sms, st) : launch_xent_product(gx, sms, st);
      }
      if (dw && e == cudaSuccess) {
        *launches += 1;
        e = launch_xent_product(gw, sms, st);
      }
      return e;
    }
    const float* dl = piece();
    const float *fx = static_cast<const float*>(x), *fw = static_cast<const float*>(w_at(v0));
    float* out = static_cast<float*>(dw) + (dw ? (d.tied ? v0 * d.H : v0) : 0);
    SimtGemm g[2];
    int n = 0;
    // no more than the workspace has room for: the last piece's share may be smaller
    const int parts = dx ? std::min(dx_parts_f32(d, cols), dx_parts_f32(d, std::min(P, d.V))) : 1;
    float* sums = reinterpret_cast<float*>(ws + L.dx);
    if (dx) {
      g[n] = {dl, fw, P, 1, d.tied ? ldw : 1, d.tied ? 1 : ldw, M, cols, H, nullptr,
              v0 && parts == 1 ? static_cast<const float*>(dx) : nullptr, parts == 1 ? static_cast<float*>(dx) : sums, nullptr,
              MOE_ACT_NONE};
      g[n].parts = parts;
      g[n++].ka = up4(cols);  // rows of dl end in zeros
    }
    if (dw && d.tied) {
      g[n] = {dl, fx, 1, P, ldx, 1, cols, M, H, nullptr, nullptr, out, nullptr, MOE_ACT_NONE};
      g[n++].ma = up4(cols);
    } else if (dw) {
      g[n] = {fx, dl, 1, ldx, P, 1, H, M, cols, nullptr, nullptr, out, nullptr, MOE_ACT_NONE, d.V};
      g[n++].nb = up4(cols);
    }
    const cudaError_t e = launch_linear_f32(g, n, true, sms, st, launches);
    if (e != cudaSuccess || parts == 1) return e;
    *launches += 1;
    const int64_t size = d.M * d.H;
    MOE_LAUNCH(k_xent_add, (unsigned)std::min<int64_t>((size + 255) / 256, (int64_t)sms * 8), 256, 0, st, sums,
               static_cast<float*>(dx), size, parts, (int)(v0 > 0));
    return cudaSuccess;
  }
};

}  // namespace

size_t xent_workspace_bytes(const moe_xent_dims& d, bool backward) { return layout(d, backward).total; }

cudaError_t launch_xent_fwd(const moe_xent_dims& d, void* ws, const void* x, const void* w, const int* target,
                            float* loss, float* lse, float* total, int sms, cudaStream_t st, int* launches) {
  Xent c = {d, static_cast<char*>(ws), layout(d, false), x, w, sms, st, launches, 0, 0, 0};
  cudaError_t e = c.prepare();
  if (e != cudaSuccess) return e;
  const bool bf = d.dtype == MOE_BF16;
  float2* stat = reinterpret_cast<float2*>(c.ws + c.L.stat);
  float* at = reinterpret_cast<float*>(c.ws + c.L.at);
  const unsigned grid = (unsigned)((d.M + kLossRows - 1) / kLossRows);
  float* dots = reinterpret_cast<float*>(c.ws + c.L.dots);
  const int parts = (int)((d.H + kDotCols - 1) / kDotCols);
  const int64_t swh = d.tied ? 1 : c.ldw, swv = d.tied ? c.ldw : 1, warps = d.M * parts;
  if (warps / 8 >= (1ll << 31) - 1) return cudaErrorInvalidValue;
  int first = 0, end = 1;  // the slots to join
  if (bf) {
    *launches += 1;
    MOE_LAUNCH(k_xent_dots, (unsigned)((warps + 7) / 8), 256, 0, st, (const __nv_bfloat16*)c.x, (const __nv_bfloat16*)c.w,
               c.ldx, swh, swv, target, (int)d.M, (int)d.H, (int)d.V, parts, dots);
    const int64_t cols = stat_cols(d);
    XentEpi epi = {};
    epi.part = stat + d.M;
    epi.at = at;
    epi.target = target;
    for (int64_t v0 = 0; v0 < d.V; v0 += cols) {
      if (v0) {  // what came before, into slot 0
        *launches += 1;
        MOE_LAUNCH(k_xent_fold, grid, kLossWarps * 32, 0, st, stat, first, end, (int)d.M);
      }
      const int n = (int)std::min(cols, d.V - v0);
      int width = 1;
      epi.v0 = (int)v0;
      *launches += 1;
      if ((e = launch_xent_stats(c.gemm(v0, n, nullptr), epi, sms, st, &width)) != cudaSuccess) return e;
      first = v0 ? 0 : 1;
      end = 1 + (n + width - 1) / width;
    }
  } else {
    for (int64_t v0 = 0; v0 < d.V; v0 += c.P) {
      const int cols = (int)std::min(c.P, d.V - v0);
      if ((e = c.logits_f32(v0, cols)) != cudaSuccess) return e;
      *launches += 1;
      MOE_LAUNCH(k_xent_piece, (unsigned)d.M, 256, 0, st, (const float*)c.piece(), c.P, cols, (int)v0, target,
                 stat, at, (int)(v0 == 0));
    }
  }
  LossArgs a = {};
  a.stat = stat;
  a.at = at;
  a.first = first;
  a.end = end;
  a.M = (int)d.M;
  a.V = (int)d.V;
  a.dots = dots;
  a.parts = parts;
  a.target = target;
  a.z = d.z_coef;
  a.loss = loss;
  a.lse = lse;
  a.part = reinterpret_cast<float2*>(c.ws + c.L.part);
  a.done = reinterpret_cast<unsigned*>(c.ws + 64);
  a.total = total;
  a.status = reinterpret_cast<int*>(c.ws);
  *launches += 1;
  if (bf) MOE_LAUNCH(k_xent_loss<true>, grid, kLossWarps * 32, 0, st, a);
  else MOE_LAUNCH(k_xent_loss<false>, grid, kLossWarps * 32, 0, st, a);
  return cudaSuccess;
}

cudaError_t launch_xent_bwd(const moe_xent_dims& d, void* ws, const void* x, const void* w, const int* target,
                            const float* lse, const float* dloss, const float* total, void* dx, void* dw, int sms,
                            cudaStream_t st, int* launches) {
  Xent c = {d, static_cast<char*>(ws), layout(d, true), x, w, sms, st, launches, 0, 0, 0};
  cudaError_t e = c.prepare();
  if (e != cudaSuccess) return e;
  const XentRows r = {target, lse, dloss, total, (int)d.V, d.z_coef};
  const bool bf = d.dtype == MOE_BF16;
  // The mean's gradient has one factor for all rows: in bf16 its rounding in dl would be one error of up to 2^-9 of
  // everything. There dl is that of the sum, at most 1 (and nearly -1 at a target that is not expected), and the products
  // are divided (4096 rows, dx 0.0029 -> 0.0019 of its size from 64 bits).
  const float* div = bf && !dloss ? total + 1 : nullptr;
  XentEpi epi = {};
  epi.target = target;
  epi.lse = lse;
  epi.dloss = dloss;
  epi.z = d.z_coef;
  epi.V = (int)d.V;
  if (bf) {
    float* own = reinterpret_cast<float*>(c.ws + c.L.at);
    epi.own = own;
    *launches += 1;
    MOE_LAUNCH(k_xent_own, (unsigned)d.M, 256, 0, st, (const __nv_bfloat16*)c.x, (const __nv_bfloat16*)c.w, c.ldx,
               d.tied ? 1 : c.ldw, d.tied ? c.ldw : 1, r, (int)d.H, (int)((d.H + kDotCols - 1) / kDotCols), own);
  }
  for (int64_t v0 = 0; v0 < d.V; v0 += c.P) {
    const int cols = (int)std::min(c.P, d.V - v0);
    *launches += 1;
    if (bf) {
      epi.v0 = (int)v0;
      if ((e = launch_xent_grad(c.gemm(v0, cols, c.piece()), epi, sms, st)) != cudaSuccess) return e;
    } else {
      if ((e = c.logits_f32(v0, cols)) != cudaSuccess) return e;
      MOE_LAUNCH(k_xent_dl, dim3((unsigned)d.M, (unsigned)((cols + 1023) / 1024)), 256, 0, st, c.piece(), c.P, cols, (int)v0, r);
    }
    if ((e = c.products(v0, cols, dx, dw, div)) != cudaSuccess) return e;
  }
  const int parts = bf ? dx_parts(d) : 0;
  if (bf && dx && (parts || c.P < d.V)) {
    *launches += 1;
    const int64_t n = d.M * d.H;
    MOE_LAUNCH(k_xent_round, (unsigned)std::min<int64_t>((n + 1023) / 1024, (int64_t)sms * 16), 256, 0, st,
               (const float*)(c.ws + c.L.dx), static_cast<__nv_bfloat16*>(dx), n, std::max(parts, 1), div);
  }
  return cudaSuccess;
}

}  // namespace moe
