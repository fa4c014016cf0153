// xent.cu -- softmax cross entropy of l = x w over a large vocabulary, and its gradients.
//
//   lse = log sum_v e^l;  loss = lse - l_target + z lse^2;  dl = d ((1 + 2 z lse) e^{l - lse} - onehot);
//   dx = dl w^T;  dw = x^T dl.
//
// The logits exist for a piece of the vocabulary at a time: their largest and the sum of exponentials are carried from
// piece to piece; the backward computes each piece again, turns it into dl and multiplies that by w and x.
#include <algorithm>

#include "block.h"
#include "common.cuh"
#include "linear_f32.h"
#include "linear_tc.h"

namespace moe {
namespace {

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }

// sum over the warp of e^{m} parts: (m, s) joined with lanes' (m, s)
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float big = fmaxf(m, m2);
  if (big == -INFINITY) return;  // both empty
  s = s * expf(m - big) + s2 * expf(m2 - big);
  m = big;
}

// A block a row: the piece's largest logit and sum joined to what earlier pieces left; the target's logit where it
// lies in the piece.
__global__ void __launch_bounds__(256) k_xent_piece(const float* l, int64_t ld, int cols, int v0, const int* target,
                                                    float2* stat, float* at_target, int first) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  __shared__ float2 red[8];
  const int64_t t = blockIdx.x;
  const float* row = l + t * ld;
  float m = -INFINITY, s = 0.0f;
  for (int i = threadIdx.x; i < cols; i += 256) {
    const float v = row[i];
    if (v > m) {
      s = s * expf(m - v) + 1.0f;
      m = v;
    } else {
      s += v == -INFINITY ? 0.0f : expf(v - m);
    }
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

// lse and loss of 256 rows a block; the blocks' totals are added in order by the last one.
__global__ void __launch_bounds__(256) k_xent_loss(const float2* stat, const float* at_target, const int* target, int M,
                                                   int V, float z, float* loss, float* lse, float2* part, unsigned* done,
                                                   float* total, int* status) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  __shared__ float2 red[8];
  __shared__ bool last;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  float sum = 0.0f, n = 0.0f;
  if (t < M) {
    const float2 st = stat[t];
    const float e = st.x + logf(st.y);
    lse[t] = e;
    const int v = target[t];
    if (v >= V) set_status(status, MOE_ERR_DEVICE_ARG);
    if (v >= 0 && v < V) {
      sum = e - at_target[t] + z * e * e;
      n = 1.0f;
    }
    loss[t] = sum;
  }
  if (!total) return;
  sum = warp_sum(sum);
  n = warp_sum(n);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(sum, n);
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) {
      sum += red[w].x;
      n += red[w].y;
    }
    part[blockIdx.x] = make_float2(sum, n);
    __threadfence();
    last = atomicAdd(done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  __shared__ double2 wide[256];
  double a = 0.0, b = 0.0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += 256) {
    const float2 p = __ldcg(part + i);
    a += p.x;
    b += p.y;
  }
  wide[threadIdx.x] = make_double2(a, b);
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 256; ++i) {
      a += wide[i].x;
      b += wide[i].y;
    }
    total[0] = (float)a;
    total[1] = (float)b;
    *done = 0;
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

// dl of a piece from its logits, a block 1024 columns of a row.
template <typename T>
__global__ void __launch_bounds__(256) k_xent_dl(const float* l, int64_t ld, int cols, int v0, XentRows r, T* dl) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const int64_t t = blockIdx.x;
  const float d = row_grad(r, t), lse = r.lse[t], f = d * (1.0f + 2.0f * r.z * lse);
  const int at = r.target[t] - v0;
  for (int i = blockIdx.y * 1024 + threadIdx.x; i < min(cols, ((int)blockIdx.y + 1) * 1024); i += 256) {
    const float p = d == 0.0f ? 0.0f : expf(l[t * ld + i] - lse) * f;
    dl[t * ld + i] = io<T>::cvt(i == at ? p - d : p);
  }
}

__global__ void __launch_bounds__(256) k_xent_round(const float* a, __nv_bfloat16* o, int64_t n) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 2048) {
    if (i + 8 <= n) {
      const float4 x = *reinterpret_cast<const float4*>(a + i), y = *reinterpret_cast<const float4*>(a + i + 4);
      const float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      *reinterpret_cast<uint4*>(o + i) = f_to_bf16x8(f);
    } else {
      for (int64_t j = i; j < n; ++j) o[j] = __float2bfloat16_rn(a[j]);
    }
  }
}

// ---------------------------------------------------------------- host side
// Columns of a piece: a multiple of 256, about 2^24 logits.
int64_t piece_cols(const moe_xent_dims& d) {
  const int64_t want = std::max<int64_t>(1024, (1 << 24) / d.M / 256 * 256);
  return std::min(want, up8(d.V));
}

// Workspace: header, the rows' statistics, a piece's logits and dl, dx in fp32, and copies of x and w with rows of a
// multiple of 16 bytes where the caller's are not.
struct XentWs {
  size_t stat, at, part, logits, dl, dx, xp, wp, total;
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
  L.stat = take((size_t)d.M * 8);
  L.at = take((size_t)d.M * 4);
  L.part = take((size_t)((d.M + 255) / 256) * 8);
  L.xp = take(bf && d.H % 8 ? (size_t)d.M * up8(d.H) * 2 : 0);
  L.wp = take(bf && C % 8 ? (size_t)R * up8(C) * 2 : 0);
  L.logits = take((size_t)d.M * P * 4);
  if (backward) {
    L.dl = take(bf ? (size_t)d.M * P * 2 : 0);
    L.dx = take(bf && d.V > P ? (size_t)d.M * d.H * 4 : 0);
  }
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

  // x and w with rows that TMA can read
  cudaError_t prepare() {
    P = piece_cols(d);
    const bool bf = d.dtype == MOE_BF16;
    ldx = bf ? up8(d.H) : d.H;
    ldw = d.tied ? ldx : bf ? up8(d.V) : d.V;
    if (!bf) return cudaSuccess;
    cudaError_t e = launch_pack_rows(&x, ws + L.xp, d.M, d.H, sms, st, launches);
    if (e != cudaSuccess) return e;
    return launch_pack_rows(&w, ws + L.wp, d.tied ? d.V : d.H, d.tied ? d.H : d.V, sms, st, launches);
  }
  const void* w_at(int64_t v0) const {
    return static_cast<const char*>(w) + (d.tied ? v0 * ldw : v0) * (d.dtype == MOE_BF16 ? 2 : 4);
  }
  cudaError_t logits(int64_t v0, int cols) {
    float* l = reinterpret_cast<float*>(ws + L.logits);
    const int M = (int)d.M, H = (int)d.H;
    if (d.dtype == MOE_BF16) {
      LinearGemm g = {M, cols, H, x, w_at(v0), ldx, ldw, 0, !d.tied, nullptr, nullptr, l, nullptr, MOE_ACT_NONE, 1,
                      reinterpret_cast<int*>(ws), P};
      *launches += 1;
      return launch_linear_tc(g, sms, st);
    }
    SimtGemm g = {static_cast<const float*>(x), static_cast<const float*>(w_at(v0)), H, 1, d.tied ? 1 : ldw,
                  d.tied ? ldw : 1, M, H, cols, nullptr, nullptr, l, nullptr, MOE_ACT_NONE, P};
    return launch_linear_f32(&g, 1, sms, st, launches);
  }
  cudaError_t products(int64_t v0, int cols, void* dx, void* dw) {
    const int M = (int)d.M, H = (int)d.H;
    if (d.dtype == MOE_BF16) {
      int* status = reinterpret_cast<int*>(ws);
      const void* dl = ws + L.dl;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(dw) + (dw ? (d.tied ? v0 * d.H : v0) : 0);
      const bool whole = P >= d.V;
      LinearGemm gx = {M, H, cols, dl, w_at(v0), P, ldw, 0, d.tied, nullptr, nullptr, whole ? dx : ws + L.dx, nullptr,
                       MOE_ACT_NONE, !whole, status, 0, v0 > 0};
      LinearGemm gw = d.tied ? LinearGemm{cols, H, M, dl, x, P, ldx, 1, 1, nullptr, nullptr, out, nullptr, MOE_ACT_NONE,
                                          0, status}
                             : LinearGemm{H, cols, M, x, dl, ldx, P, 1, 1, nullptr, nullptr, out, nullptr, MOE_ACT_NONE,
                                          0, status, d.V};
      cudaError_t e = cudaSuccess;
      if (dx) {
        *launches += 1;
        e = launch_linear_tc(gx, sms, st);
      }
      if (dw && e == cudaSuccess) {
        *launches += 1;
        e = launch_linear_tc(gw, sms, st);
      }
      return e;
    }
    const float* dl = reinterpret_cast<const float*>(ws + L.logits);
    const float *fx = static_cast<const float*>(x), *fw = static_cast<const float*>(w_at(v0));
    float* out = static_cast<float*>(dw) + (dw ? (d.tied ? v0 * d.H : v0) : 0);
    SimtGemm g[2];
    int n = 0;
    if (dx) g[n++] = {dl, fw, P, 1, d.tied ? ldw : 1, d.tied ? 1 : ldw, M, cols, H, nullptr,
                      v0 ? static_cast<const float*>(dx) : nullptr, static_cast<float*>(dx), nullptr, MOE_ACT_NONE};
    if (dw && d.tied) g[n++] = {dl, fx, 1, P, ldx, 1, cols, M, H, nullptr, nullptr, out, nullptr, MOE_ACT_NONE};
    if (dw && !d.tied) g[n++] = {fx, dl, 1, ldx, P, 1, H, M, cols, nullptr, nullptr, out, nullptr, MOE_ACT_NONE, d.V};
    return launch_linear_f32(g, n, sms, st, launches);
  }
};

}  // namespace

size_t xent_workspace_bytes(const moe_xent_dims& d, bool backward) { return layout(d, backward).total; }

cudaError_t launch_xent_fwd(const moe_xent_dims& d, void* ws, const void* x, const void* w, const int* target,
                            float* loss, float* lse, float* total, int sms, cudaStream_t st, int* launches) {
  Xent c = {d, static_cast<char*>(ws), layout(d, false), x, w, sms, st, launches, 0, 0, 0};
  cudaError_t e = c.prepare();
  if (e != cudaSuccess) return e;
  float2* stat = reinterpret_cast<float2*>(c.ws + c.L.stat);
  float* at = reinterpret_cast<float*>(c.ws + c.L.at);
  for (int64_t v0 = 0; v0 < d.V; v0 += c.P) {
    const int cols = (int)std::min(c.P, d.V - v0);
    if ((e = c.logits(v0, cols)) != cudaSuccess) return e;
    *launches += 1;
    MOE_LAUNCH(k_xent_piece, (unsigned)d.M, 256, 0, st, (const float*)(c.ws + c.L.logits), c.P, cols, (int)v0, target,
               stat, at, (int)(v0 == 0));
  }
  *launches += 1;
  MOE_LAUNCH(k_xent_loss, (unsigned)((d.M + 255) / 256), 256, 0, st, (const float2*)stat, (const float*)at, target,
             (int)d.M, (int)d.V, d.z_coef, loss, lse, reinterpret_cast<float2*>(c.ws + c.L.part),
             reinterpret_cast<unsigned*>(c.ws + 64), total, reinterpret_cast<int*>(c.ws));
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
  float* l = reinterpret_cast<float*>(c.ws + c.L.logits);
  for (int64_t v0 = 0; v0 < d.V; v0 += c.P) {
    const int cols = (int)std::min(c.P, d.V - v0);
    if ((e = c.logits(v0, cols)) != cudaSuccess) return e;
    const dim3 grid((unsigned)d.M, (unsigned)((cols + 1023) / 1024));
    *launches += 1;
    if (bf) MOE_LAUNCH(k_xent_dl<__nv_bfloat16>, grid, 256, 0, st, (const float*)l, c.P, cols, (int)v0, r,
                       reinterpret_cast<__nv_bfloat16*>(c.ws + c.L.dl));
    else MOE_LAUNCH(k_xent_dl<float>, grid, 256, 0, st, (const float*)l, c.P, cols, (int)v0, r, l);
    if ((e = c.products(v0, cols, dx, dw)) != cudaSuccess) return e;
  }
  if (bf && dx && c.P < d.V) {
    *launches += 1;
    const int64_t n = d.M * d.H;
    MOE_LAUNCH(k_xent_round, (unsigned)std::min<int64_t>((n + 2047) / 2048, (int64_t)sms * 16), 256, 0, st,
               (const float*)(c.ws + c.L.dx), static_cast<__nv_bfloat16*>(dx), n);
  }
  return cudaSuccess;
}

}  // namespace moe
