// norm.cu -- layer norm and RMS norm of rows, forward and backward.
//
// h = x + residual, y = (h - mean) rstd w + b. Sums are fp32 throughout; the variance is
// the mean of the squared deviations, taken in a second pass over the row (the one-pass
// form sum(h^2) - mean^2 loses every digit when the mean is large against the spread).
// Both directions are bound by HBM: each tensor is read or written once. Measured with inputs that change from call
// to call (400 MB in turn), layer norm:
//   8192 x 4096 with a residual   bf16 forward 46 us (5.8 TB/s), backward 49 (5.5, weight gradients included); fp32
//                                 forward 87 (6.1); fp32 backward without a residual 66 (6.1)
//   4096 x 2048 with a residual   bf16 forward 14.2, backward 19.9; fp32 forward 22, backward 27
// Without a residual the bf16 forward is held by the sums' instructions instead (8192 x 4096: 31.5 us, 4.3 TB/s; RMS
// 24.7). One row of 2048 forward 1.5 us.
#include <algorithm>
#include <atomic>

#include "block.h"
#include "common.cuh"

namespace moe {
namespace {

// VEC consecutive elements as one 16-byte (or, VEC = 1, one-element) access.
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
  T v[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ void unpack(const Vec<T, VEC>& a, float (&f)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) f[i] = io<T>::to_f(a.v[i]);
}
template <typename T, int VEC>
__device__ __forceinline__ Vec<T, VEC> pack(const float (&f)[VEC]) {
  Vec<T, VEC> a;
#pragma unroll
  for (int i = 0; i < VEC; ++i) a.v[i] = io<T>::cvt(f[i]);
  return a;
}

// v += s and out = v s, two elements an instruction (packed fp32, each rounded as the single one would be).
template <int VEC>
__device__ __forceinline__ void add_all(float (&v)[VEC], float s) {
  uint64_t ss;
  asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
#pragma unroll
  for (int i = 0; i < VEC; i += 2) {
    uint64_t t;
    asm("mov.b64 %0, {%1, %2};" : "=l"(t) : "f"(v[i]), "f"(v[i + 1]));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(t) : "l"(ss));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v[i]), "=f"(v[i + 1]) : "l"(t));
  }
}
template <int VEC>
__device__ __forceinline__ void scale_all(const float (&v)[VEC], float s, float (&out)[VEC]) {
  uint64_t ss;
  asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
#pragma unroll
  for (int i = 0; i < VEC; i += 2) {
    uint64_t t;
    asm("mov.b64 %0, {%1, %2};" : "=l"(t) : "f"(v[i]), "f"(v[i + 1]));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(t) : "l"(ss));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(out[i]), "=f"(out[i + 1]) : "l"(t));
  }
}

// Sums over a group of G threads (a warp, or G / 32 warps that meet at barrier `id`) of one value or
// two; every thread gets them. `slots` is the group's own, two sets of G / 32 entries used in turn,
// so one barrier a call is enough; behind it every thread adds the warps' sums in order (a few
// 16-byte shared loads, where a second butterfly costs ten shuffles and additions).
template <int G>
__device__ __forceinline__ float group_sum(float a, float2* slots, int* turn, int id) {
  a = warp_sum(a);
  if constexpr (G > 32) {
    constexpr int W = G / 32;
    float* s = reinterpret_cast<float*>(slots + *turn * W);
    *turn ^= 1;
    if ((threadIdx.x & 31) == 0) s[(threadIdx.x % G) >> 5] = a;
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(G) : "memory");
    a = 0.0f;
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(s + i);
      a += (v.x + v.y) + (v.z + v.w);
    }
  }
  return a;
}
template <int G>
__device__ __forceinline__ float2 group_sum2(float a, float b, float2* slots, int* turn, int id) {
  a = warp_sum(a);
  b = warp_sum(b);
  if constexpr (G > 32) {
    constexpr int W = G / 32;
    float2* s = slots + *turn * W;
    *turn ^= 1;
    if ((threadIdx.x & 31) == 0) s[(threadIdx.x % G) >> 5] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(G) : "memory");
    a = b = 0.0f;
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      const float4 v = *reinterpret_cast<const float4*>(s + i);
      a += v.x + v.z;
      b += v.y + v.w;
    }
  }
  return make_float2(a, b);
}

// Block-wide sums of two values; every thread gets both (fixed tree: same result each run).
__device__ __forceinline__ float2 block_sum2(float a, float b) {
  __shared__ float2 part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  a = warp_sum(a);
  b = warp_sum(b);
  __syncthreads();  // the previous call's reads of part
  if (lane == 0) part[warp] = make_float2(a, b);
  __syncthreads();
  float2 v = lane < nw ? part[lane] : make_float2(0.0f, 0.0f);
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  return v;
}

// Rows too long for a block's registers (16384 elements; backward 8192 in fp32 or
// without 16-byte alignment): block per row, three passes over it.
template <typename T>
__global__ void __launch_bounds__(256) k_norm_fwd_long(const T* x, const T* res, const T* w, const T* b, T* y, T* sum,
                                                  float* mean, float* rstd, int rows, int H, int rms, float eps) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  for (int t = blockIdx.x; t < rows; t += gridDim.x) {
    const int64_t o = (int64_t)t * H;
    auto h_at = [&](int i) { return io<T>::to_f(x[o + i]) + (res ? io<T>::to_f(res[o + i]) : 0.0f); };
    float s = 0.0f, q = 0.0f;
    if (!rms)
      for (int i = threadIdx.x; i < H; i += blockDim.x) s += h_at(i);
    const float mu = rms ? 0.0f : block_sum2(s, 0.0f).x / (float)H;
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      const float d = h_at(i) - mu;
      q = fmaf(d, d, q);
    }
    const float rs = 1.0f / sqrtf(block_sum2(q, 0.0f).x / (float)H + eps);
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      const float h = h_at(i);
      const float v = fmaf((h - mu) * rs, io<T>::to_f(w[i]), b ? io<T>::to_f(b[i]) : 0.0f);
      if (sum) sum[o + i] = io<T>::cvt(h);
      y[o + i] = io<T>::cvt(v);
    }
    if (threadIdx.x == 0) {
      if (mean) mean[t] = mu;
      if (rstd) rstd[t] = rs;
    }
  }
}

// dx of such rows, block per row.
template <typename T>
__global__ void __launch_bounds__(256) k_norm_dx_long(const T* dy, const T* dsum, const T* x, const T* w, const float* mean,
                                                 const float* rstd, T* dx, int rows, int H) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  for (int t = blockIdx.x; t < rows; t += gridDim.x) {
    const int64_t o = (int64_t)t * H;
    const float mu = mean ? mean[t] : 0.0f, rs = rstd[t];
    float s = 0.0f, q = 0.0f;
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      const float g = io<T>::to_f(dy[o + i]) * io<T>::to_f(w[i]);
      s += g;
      q = fmaf(g, (io<T>::to_f(x[o + i]) - mu) * rs, q);
    }
    const float2 r = block_sum2(s, q);
    const float ms = mean ? r.x / (float)H : 0.0f, mq = r.y / (float)H;
    for (int i = threadIdx.x; i < H; i += blockDim.x) {
      const float g = io<T>::to_f(dy[o + i]) * io<T>::to_f(w[i]);
      const float xh = (io<T>::to_f(x[o + i]) - mu) * rs;
      const float v = rs * (g - ms - xh * mq) + (dsum ? io<T>::to_f(dsum[o + i]) : 0.0f);
      dx[o + i] = io<T>::cvt(v);
    }
  }
}

constexpr int kNormChunks = 128;  // row chunks of the weight-gradient partial sums

// Partial sums over one chunk of rows: part[c][0][i] = sum dy xh, part[c][1][i] = sum dy.
template <typename T>
__global__ void __launch_bounds__(256) k_norm_dw_long(const T* dy, const T* x, const float* mean, const float* rstd,
                                                 float* part, int rows, int H, int per) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= H) return;
  const int t0 = blockIdx.y * per, t1 = min(rows, t0 + per);
  float aw = 0.0f, ab = 0.0f;
  for (int t = t0; t < t1; ++t) {
    const float g = io<T>::to_f(dy[(int64_t)t * H + i]);
    const float xh = (io<T>::to_f(x[(int64_t)t * H + i]) - (mean ? mean[t] : 0.0f)) * rstd[t];
    aw = fmaf(g, xh, aw);
    ab += g;
  }
  part[((int64_t)blockIdx.y * 2) * H + i] = aw;
  part[((int64_t)blockIdx.y * 2 + 1) * H + i] = ab;
}

// The chunks' partial sums added: 32 chunk lanes a column, each in chunk order, then the lanes in
// order. A lane has few chunks (five of 152), whose loads travel together.
template <typename T>
__global__ void __launch_bounds__(1024) k_norm_dw_sum(const float* part, int chunks, int H, T* dw, T* db) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  __shared__ float red[2][32][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + cx;
  float aw = 0.0f, ab = 0.0f;
  if (i < H) {
#pragma unroll 5
    for (int c = ry; c < chunks; c += 32) {
      aw += part[((int64_t)c * 2) * H + i];
      if (db) ab += part[((int64_t)c * 2 + 1) * H + i];
    }
  }
  red[0][ry][cx] = aw;
  red[1][ry][cx] = ab;
  __syncthreads();
  // warp 0 adds the weight sums, warp 1 the bias sums
  if (ry < 2 && i < H && (ry == 0 || db)) {
    float v = red[ry][0][cx];
#pragma unroll
    for (int r = 1; r < 32; ++r) v += red[ry][r][cx];
    (ry ? db : dw)[i] = io<T>::cvt(v);
  }
}


// ---------------------------------------------------------------- rows held in registers
template <int G>
constexpr int kFwdThreads = G < 256 ? 256 : G;

struct FwdArgs {
  const void *x, *res, *w, *b;
  void *y, *sum;
  float *mean, *rstd;
  int rows, H, rms;
  float eps;
};

// A group of G threads per row, VPT vectors of VEC elements a thread; every tensor is read or
// written once, in 16-byte accesses where H allows. The row waits in registers (fp32) for its
// mean and then its variance. Blocks stay and walk the rows.
template <typename T, int VEC, int VPT, int G>
__global__ void __launch_bounds__(kFwdThreads<G>) k_norm_fwd(const FwdArgs a) {
  using V = Vec<T, VEC>;
  pdl_wait();  // the previous kernel has completed and its writes are visible
  constexpr int GROUPS = kFwdThreads<G> / G;
  __shared__ __align__(16) float2 slots[GROUPS][G > 32 ? 2 * (G / 32) : 2];
  const int grp = threadIdx.x / G, j = threadIdx.x % G;
  int turn = 0;
  const int nv = a.H / VEC;
  const float inv_h = 1.0f / (float)a.H;
  const V* w = reinterpret_cast<const V*>(a.w);
  const V* bias = reinterpret_cast<const V*>(a.b);
  for (int t = blockIdx.x * GROUPS + grp; t < a.rows; t += gridDim.x * GROUPS) {
    const int64_t o = (int64_t)t * nv;
    const V* x = reinterpret_cast<const V*>(a.x) + o;
    const V* res = reinterpret_cast<const V*>(a.res) + o;
    float h[VPT][VEC];
    {
      V xv[VPT], rv[VPT];
#pragma unroll
      for (int p = 0; p < VPT; ++p)
        if (j + p * G < nv) xv[p] = x[j + p * G];
      if (a.res) {
#pragma unroll
        for (int p = 0; p < VPT; ++p)
          if (j + p * G < nv) rv[p] = res[j + p * G];
      }
#pragma unroll
      for (int p = 0; p < VPT; ++p) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) h[p][i] = 0.0f;
        if (j + p * G < nv) {
          unpack<T, VEC>(xv[p], h[p]);
          if (a.res) {
            float r[VEC];
            unpack<T, VEC>(rv[p], r);
#pragma unroll
            for (int i = 0; i < VEC; ++i) h[p][i] += r[i];
          }
        }
      }
    }
    float mu = 0.0f;
    if (!a.rms) {
      float s = 0.0f;
#pragma unroll
      for (int p = 0; p < VPT; ++p)
#pragma unroll
        for (int i = 0; i < VEC; ++i) s += h[p][i];
      mu = group_sum<G>(s, slots[grp], &turn, 1 + grp) * inv_h;
    }
    V* y = reinterpret_cast<V*>(a.y) + o;
    V* sum = reinterpret_cast<V*>(a.sum) + o;
    float q = 0.0f;
#pragma unroll
    for (int p = 0; p < VPT; ++p)
      if (j + p * G < nv) {
        if (a.sum) sum[j + p * G] = pack<T, VEC>(h[p]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          h[p][i] -= mu;
          q = fmaf(h[p][i], h[p][i], q);
        }
      }
    const float rs = 1.0f / sqrtf(group_sum<G>(q, slots[grp], &turn, 1 + grp) * inv_h + a.eps);
#pragma unroll
    for (int p = 0; p < VPT; ++p)
      if (j + p * G < nv) {
        float wf[VEC], v[VEC];
        unpack<T, VEC>(w[j + p * G], wf);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = h[p][i] * rs * wf[i];
        if (bias) {
          float bf[VEC];
          unpack<T, VEC>(bias[j + p * G], bf);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[i] += bf[i];
        }
        y[j + p * G] = pack<T, VEC>(v);
      }
    if (j == 0) {
      if (a.mean) a.mean[t] = mu;
      if (a.rstd) a.rstd[t] = rs;
    }
  }
}

// The same for many aligned rows: the rows come through a ring of STAGES slots in shared memory
// filled by 16-byte asynchronous copies, a row or more ahead of the sums. A thread copies exactly
// the vectors it reads, so the ring needs no barrier.
template <typename T, int VPT, int G, int STAGES>
__global__ void __launch_bounds__(512, sizeof(T) == 2 ? 2 : 1) k_norm_fwd_ring(const FwdArgs a) {
  constexpr int VEC = 16 / sizeof(T);
  using V = Vec<T, VEC>;
  pdl_wait();  // the previous kernel has completed and its writes are visible
  constexpr int GROUPS = 512 / G;
  __shared__ __align__(16) float2 slots[GROUPS][G > 32 ? 2 * (G / 32) : 2];
  extern __shared__ __align__(16) uint8_t ring[];  // [STAGES][2 tensors][VPT][512 threads] vectors
  const int grp = threadIdx.x / G, j = threadIdx.x % G;
  int turn = 0;
  const int nv = a.H / VEC;
  const float inv_h = 1.0f / (float)a.H;
  const V* x = reinterpret_cast<const V*>(a.x);
  const V* res = reinterpret_cast<const V*>(a.res);
  V wv[VPT], bv[VPT];
#pragma unroll
  for (int p = 0; p < VPT; ++p)
    if (j + p * G < nv) {
      wv[p] = reinterpret_cast<const V*>(a.w)[j + p * G];
      if (a.b) bv[p] = reinterpret_cast<const V*>(a.b)[j + p * G];
    }
  const uint32_t base = smem_u32(ring) + threadIdx.x * 16;
  auto slot = [&](int st, int tensor, int p) { return base + (uint32_t)(((st * 2 + tensor) * VPT + p) * 512 * 16); };
  auto fetch = [&](int t, int st) {
    if (t < a.rows) {
      const int64_t o = (int64_t)t * nv + j;
#pragma unroll
      for (int p = 0; p < VPT; ++p)
        if (j + p * G < nv) {
          cp_async16(slot(st, 0, p), x + o + p * G);
          if (res) cp_async16(slot(st, 1, p), res + o + p * G);
        }
    }
    cp_async_commit();
  };
  auto read = [&](int st, int tensor, int p, float (&f)[VEC]) {
    const uint4 u = ld_shared_v4(slot(st, tensor, p));
    unpack<T, VEC>(*reinterpret_cast<const V*>(&u), f);
  };
  const int step = gridDim.x * GROUPS;
  int t = blockIdx.x * GROUPS + grp, st = 0;
#pragma unroll
  for (int s = 0; s < STAGES; ++s) fetch(t + s * step, s);
  for (; t < a.rows; t += step) {
    cp_async_wait<STAGES - 1>();
    float h[VPT][VEC];
    float s = 0.0f;
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) h[p][i] = 0.0f;
      if (j + p * G < nv) {
        read(st, 0, p, h[p]);
        if (res) {
          float r[VEC];
          read(st, 1, p, r);
#pragma unroll
          for (int i = 0; i < VEC; ++i) h[p][i] += r[i];
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) s += h[p][i];
      }
    }
    fetch(t + STAGES * step, st);
    st = st + 1 == STAGES ? 0 : st + 1;
    const float mu = a.rms ? 0.0f : group_sum<G>(s, slots[grp], &turn, 1 + grp) * inv_h;
    V* y = reinterpret_cast<V*>(a.y) + (int64_t)t * nv + j;
    V* sum = reinterpret_cast<V*>(a.sum) + (int64_t)t * nv + j;
    float q = 0.0f;
#pragma unroll
    for (int p = 0; p < VPT; ++p)
      if (j + p * G < nv) {
        if (a.sum) sum[p * G] = pack<T, VEC>(h[p]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          h[p][i] -= mu;
          q = fmaf(h[p][i], h[p][i], q);
        }
      }
    const float rs = 1.0f / sqrtf(group_sum<G>(q, slots[grp], &turn, 1 + grp) * inv_h + a.eps);
#pragma unroll
    for (int p = 0; p < VPT; ++p)
      if (j + p * G < nv) {
        float wf[VEC], v[VEC];
        unpack<T, VEC>(wv[p], wf);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = h[p][i] * rs * wf[i];
        if (a.b) {
          float bf[VEC];
          unpack<T, VEC>(bv[p], bf);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[i] += bf[i];
        }
        y[p * G] = pack<T, VEC>(v);
      }
    if (j == 0) {
      if (a.mean) a.mean[t] = mu;
      if (a.rstd) a.rstd[t] = rs;
    }
  }
  cp_async_wait<0>();
}

struct BwdArgs {
  const void *dy, *dsum, *x, *w;
  const float *mean, *rstd;
  void *dx, *dweight, *dbias;
  float* part;
  int rows, H;
};

// The groups' column sums are added in order through shared memory ([element][thread], free of bank
// conflicts) and written as one row of partial sums a block; a grid of one block writes the
// gradients themselves.
template <typename T, int VEC, int VPT, int G, int THREADS>
__device__ __forceinline__ void write_part(const BwdArgs& a, float (&aw)[VPT][VEC], float (&ab)[VPT][VEC],
                                           float* smem) {
  constexpr int GROUPS = THREADS / G, COLS = G * VPT * VEC;
  const int grp = threadIdx.x / G, j = threadIdx.x % G;
  for (int k = 1; k < GROUPS; ++k) {  // group 0 collects the others', one group at a time
    __syncthreads();
    if (grp == k) {
#pragma unroll
      for (int p = 0; p < VPT; ++p)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          smem[(p * VEC + i) * G + j] = aw[p][i];
          smem[COLS + (p * VEC + i) * G + j] = ab[p][i];
        }
    }
    __syncthreads();
    if (grp == 0) {
#pragma unroll
      for (int p = 0; p < VPT; ++p)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          aw[p][i] += smem[(p * VEC + i) * G + j];
          ab[p][i] += smem[COLS + (p * VEC + i) * G + j];
        }
    }
  }
  if (grp == 0 && gridDim.x == 1) {
    Vec<T, VEC>* dw = reinterpret_cast<Vec<T, VEC>*>(a.dweight);
    Vec<T, VEC>* db = reinterpret_cast<Vec<T, VEC>*>(a.dbias);
#pragma unroll
    for (int p = 0; p < VPT; ++p)
      if (j + p * G < a.H / VEC) {
        dw[j + p * G] = pack<T, VEC>(aw[p]);
        if (db) db[j + p * G] = pack<T, VEC>(ab[p]);
      }
  } else if (grp == 0) {
    Vec<float, VEC>* pw = reinterpret_cast<Vec<float, VEC>*>(a.part + (int64_t)blockIdx.x * 2 * a.H);
    Vec<float, VEC>* pb = reinterpret_cast<Vec<float, VEC>*>(a.part + ((int64_t)blockIdx.x * 2 + 1) * a.H);
#pragma unroll
    for (int p = 0; p < VPT; ++p)
      if (j + p * G < a.H / VEC) {
        pw[j + p * G] = pack<float, VEC>(aw[p]);
        if (a.dbias) pb[j + p * G] = pack<float, VEC>(ab[p]);
      }
  }
}

// One pass over dy, x (and dsum): dx, and the block's share of the weight gradients. A group of G
// threads per row; a thread keeps its columns for every row, so dweight and dbias add up in its
// registers. Rows come through a ring of STAGES slots in shared memory filled by 16-byte
// asynchronous copies. A thread copies exactly the vectors it reads, so the ring needs no barrier,
// the loads run a row or more ahead of the sums, and the values can be read again after the row's
// sums instead of being held in registers.
// xh is (x - mean) rstd: the subtraction of near values is exact, where x rstd - mean rstd would carry the
// rounding of a large mean into every element of the row.
template <typename T, int VPT, int G, int STAGES>
__global__ void __launch_bounds__(512) k_norm_bwd_ring(const BwdArgs a) {
  constexpr int VEC = 16 / sizeof(T);
  using V = Vec<T, VEC>;
  pdl_wait();  // the previous kernel has completed and its writes are visible
  constexpr int GROUPS = 512 / G;
  __shared__ __align__(16) float2 slots[GROUPS][G > 32 ? 2 * (G / 32) : 2];
  extern __shared__ __align__(16) uint8_t ring[];  // [STAGES][3 tensors][VPT][512 threads] vectors
  const int grp = threadIdx.x / G, j = threadIdx.x % G;
  int turn = 0;
  const int nv = a.H / VEC;
  const float inv_h = 1.0f / (float)a.H;
  const V* dy = reinterpret_cast<const V*>(a.dy);
  const V* ds = reinterpret_cast<const V*>(a.dsum);
  const V* x = reinterpret_cast<const V*>(a.x);
  V* dx = reinterpret_cast<V*>(a.dx);
  V wv[VPT];
  float aw[VPT][VEC], ab[VPT][VEC];
#pragma unroll
  for (int p = 0; p < VPT; ++p) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) aw[p][i] = ab[p][i] = 0.0f;
    if (j + p * G < nv) wv[p] = reinterpret_cast<const V*>(a.w)[j + p * G];
  }
  const uint32_t base = smem_u32(ring) + threadIdx.x * 16;
  auto slot = [&](int st, int tensor, int p) { return base + (uint32_t)(((st * 3 + tensor) * VPT + p) * 512 * 16); };
  auto fetch = [&](int t, int st) {
    if (t < a.rows) {
      const int64_t o = (int64_t)t * nv + j;
#pragma unroll
      for (int p = 0; p < VPT; ++p)
        if (j + p * G < nv) {
          cp_async16(slot(st, 0, p), dy + o + p * G);
          cp_async16(slot(st, 1, p), x + o + p * G);
          if (ds) cp_async16(slot(st, 2, p), ds + o + p * G);
        }
    }
    cp_async_commit();
  };
  auto read = [&](int st, int tensor, int p, float (&f)[VEC]) {
    const uint4 u = ld_shared_v4(slot(st, tensor, p));
    unpack<T, VEC>(*reinterpret_cast<const V*>(&u), f);
  };
  const int step = gridDim.x * GROUPS;
  int t = blockIdx.x * GROUPS + grp;
#pragma unroll
  for (int s = 0; s < STAGES; ++s) fetch(t + s * step, s);
  int st = 0;
  float nmu = 0.0f, nrs = 0.0f;  // the next row's statistics
  auto stats = [&](int r) {
    if (r < a.rows) {
      nmu = a.mean ? a.mean[r] : 0.0f;
      nrs = a.rstd[r];
    }
  };
  stats(t);
  for (; t < a.rows; t += step) {
    const float rs = nrs, mu = nmu;
    stats(t + step);
    cp_async_wait<STAGES - 1>();
    float s = 0.0f, q = 0.0f;
#pragma unroll
    for (int p = 0; p < VPT; ++p)
      if (j + p * G < nv) {
        float d[VEC], xv[VEC], wf[VEC];
        read(st, 0, p, d);
        read(st, 1, p, xv);
        unpack<T, VEC>(wv[p], wf);
        add_all<VEC>(xv, -mu);
        scale_all<VEC>(xv, rs, xv);  // xh
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          aw[p][i] = fmaf(d[i], xv[i], aw[p][i]);
          ab[p][i] += d[i];
          const float g = d[i] * wf[i];
          s += g;
          q = fmaf(g, xv[i], q);
        }
      }
    const float2 r = group_sum2<G>(s, q, slots[grp], &turn, 1 + grp);
    // dx = rs (g - (x - mean) rs (mean g xh)) - rs (mean g)
    const float ms = a.mean ? rs * r.x * inv_h : 0.0f, mq = rs * r.y * inv_h;
    V* o = dx + (int64_t)t * nv + j;
#pragma unroll
    for (int p = 0; p < VPT; ++p)
      if (j + p * G < nv) {
        float d[VEC], xv[VEC], wf[VEC];
        read(st, 0, p, d);
        read(st, 1, p, xv);
        unpack<T, VEC>(wv[p], wf);
        add_all<VEC>(xv, -mu);
#pragma unroll
        for (int i = 0; i < VEC; ++i) d[i] = fmaf(fmaf(-xv[i], mq, d[i] * wf[i]), rs, -ms);
        if (ds) {
          read(st, 2, p, xv);
#pragma unroll
          for (int i = 0; i < VEC; ++i) d[i] += xv[i];
        }
        o[p * G] = pack<T, VEC>(d);
      }
    fetch(t + STAGES * step, st);
    st = st + 1 == STAGES ? 0 : st + 1;
  }
  cp_async_wait<0>();
  write_part<T, VEC, VPT, G, 512>(a, aw, ab, reinterpret_cast<float*>(ring));
}

// The same for rows without 16-byte alignment, element by element: thread j keeps the columns
// j + p G, and the next row's loads travel in registers while this row's sums meet. Slots past the
// row are skipped by the whole group. Bound by the latency of these 4- and 2-byte loads, one block an SM: 1001 x 1111
// in fp32 9.9 us with its second kernel (1.4 TB/s). The variant for 4097 to 8192 columns keeps 16 of each array a
// thread and spills 144 to 168 bytes: 1001 x 5001 61 us in fp32, 53 in bf16.
template <int G>
constexpr int odd_threads = G < 256 ? 256 : G;

template <typename T, int VPT, int G>
__global__ void __launch_bounds__(odd_threads<G>) k_norm_bwd_odd(const BwdArgs a) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  constexpr int GROUPS = odd_threads<G> / G;
  __shared__ __align__(16) float2 slots[GROUPS][G > 32 ? 2 * (G / 32) : 2];
  extern __shared__ float acc_smem[];  // [2][columns of a group], only with several groups
  const int grp = threadIdx.x / G, j = threadIdx.x % G;
  int turn = 0;
  const int H = a.H;
  const float inv_h = 1.0f / (float)H;
  const T* dy = reinterpret_cast<const T*>(a.dy);
  const T* ds = reinterpret_cast<const T*>(a.dsum);
  const T* x = reinterpret_cast<const T*>(a.x);
  T* dx = reinterpret_cast<T*>(a.dx);
  float w[VPT], aw[VPT][1], ab[VPT][1];
#pragma unroll
  for (int p = 0; p < VPT; ++p) {
    aw[p][0] = ab[p][0] = 0.0f;
    w[p] = j + p * G < H ? io<T>::to_f(reinterpret_cast<const T*>(a.w)[j + p * G]) : 0.0f;
  }
  T ndy[VPT], nx[VPT], nds[VPT];
  float nmu = 0.0f, nrs = 0.0f;
  auto fetch = [&](int t) {
    if (t >= a.rows) return;
    const int64_t o = (int64_t)t * H + j;
    nmu = a.mean ? a.mean[t] : 0.0f;
    nrs = a.rstd[t];
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      if (p * G >= H) break;
      if (j + p * G < H) {
        ndy[p] = dy[o + p * G];
        nx[p] = x[o + p * G];
        if (ds) nds[p] = ds[o + p * G];
      }
    }
  };
  const int step = gridDim.x * GROUPS;
  int t = blockIdx.x * GROUPS + grp;
  fetch(t);
  for (; t < a.rows; t += step) {
    const float rs = nrs, mu = nmu;
    float d[VPT], xh[VPT], e[VPT];
    float s = 0.0f, q = 0.0f;
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      if (p * G >= H) break;
      const bool in = j + p * G < H;
      d[p] = in ? io<T>::to_f(ndy[p]) : 0.0f;
      xh[p] = in ? (io<T>::to_f(nx[p]) - mu) * rs : 0.0f;
      e[p] = in && ds ? io<T>::to_f(nds[p]) : 0.0f;
      aw[p][0] = fmaf(d[p], xh[p], aw[p][0]);
      ab[p][0] += d[p];
      d[p] *= w[p];
      s += d[p];
      q = fmaf(d[p], xh[p], q);
    }
    fetch(t + step);
    const float2 r = group_sum2<G>(s, q, slots[grp], &turn, 1 + grp);
    const float ms = a.mean ? rs * r.x * inv_h : 0.0f, mq = rs * r.y * inv_h;
    T* o = dx + (int64_t)t * H + j;
#pragma unroll
    for (int p = 0; p < VPT; ++p) {
      if (p * G >= H) break;
      if (j + p * G < H) o[p * G] = io<T>::cvt(fmaf(-xh[p], mq, fmaf(d[p], rs, -ms)) + e[p]);
    }
  }
  write_part<T, 1, VPT, G, odd_threads<G>>(a, aw, ab, acc_smem);
}

// ---------------------------------------------------------------- choice of the variant
constexpr int kMaxParts = 512;  // rows of partial sums the workspace holds

// Blocks of a persistent kernel: as many as fit on the GPU at once, or as the rows need.
// The occupancy is asked once per kernel (`cache`): it only sets the grid.
template <typename K>
int resident_blocks(K kern, std::atomic<int>* cache, int threads, size_t smem, int64_t need, int sms, int cap) {
  int per = cache->load(std::memory_order_relaxed);
  if (per < 1) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, threads, smem) != cudaSuccess || per < 1) per = 1;
    cache->store(per, std::memory_order_relaxed);
  }
  return (int)std::max<int64_t>(1, std::min<int64_t>({need, (int64_t)per * sms, (int64_t)cap}));
}

template <typename T, int VEC, int VPT, int G>
cudaError_t fwd_regs(const FwdArgs& a, int sms, cudaStream_t st) {
  constexpr int threads = kFwdThreads<G>, groups = threads / G;
  static std::atomic<int> cache{0};
  auto kern = k_norm_fwd<T, VEC, VPT, G>;
  const int grid = resident_blocks(kern, &cache, threads, 0, ((int64_t)a.rows + groups - 1) / groups, sms, 1 << 30);
  MOE_LAUNCH(kern, grid, threads, 0, st, a);
  return cudaSuccess;
}

template <typename T, int EPT, int G>
cudaError_t fwd_ring(const FwdArgs& a, int sms, cudaStream_t st) {
  constexpr int VPT = EPT * (int)sizeof(T) / 16, stage = 2 * VPT * 512 * 16, groups = 512 / G;
  constexpr int room = sizeof(T) == 2 ? 98304 : 131072;  // two blocks an SM in bf16, one in fp32
  constexpr int stages = room / stage < 4 ? room / stage : 4;
  static_assert(stages >= 2, "ring too small");
  static std::atomic<int> cache{0};
  auto kern = k_norm_fwd_ring<T, VPT, G, stages>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, stages * stage);
  if (e != cudaSuccess) return e;
  const int grid = resident_blocks(kern, &cache, 512, stages * stage, ((int64_t)a.rows + groups - 1) / groups, sms, 1 << 30);
  MOE_LAUNCH(kern, grid, 512, stages * stage, st, a);
  return cudaSuccess;
}

// Many aligned rows go through the ring (16 rows an SM and more: 6000 rows of 1024 in bf16 take
// 10.4 us, 14.2 in registers; 3000 rows of 2048 and fewer leave a group about a row, where the
// registers are as fast). Else thirty-two elements a thread at most (they stay in registers) and
// the smallest group that covers the row; with few rows the latency of one row counts, and the
// whole block takes the row, eight elements a thread where that covers it.
template <typename T, int VEC>
cudaError_t fwd_vec(const FwdArgs& a, int sms, cudaStream_t st, bool* taken) {
  constexpr int P = 8 / VEC;  // vectors of eight elements
  const int h = a.H;
  *taken = true;
  if constexpr (VEC > 1) {
    if (a.rows >= sms * 16) {
      if (h <= 256) return fwd_ring<T, 8, 32>(a, sms, st);
      if (h <= 512) return fwd_ring<T, 16, 32>(a, sms, st);
      if (h <= 1024) return fwd_ring<T, 8, 128>(a, sms, st);
      if (h <= 2048) return fwd_ring<T, 16, 128>(a, sms, st);
      if (h <= 4096) return fwd_ring<T, 16, 256>(a, sms, st);
      if (h <= 8192) return fwd_ring<T, 16, 512>(a, sms, st);
    }
  }
  if (h <= 256) return fwd_regs<T, VEC, P, 32>(a, sms, st);
  if (a.rows < sms * 2) {
    if (h <= 2048) return fwd_regs<T, VEC, P, 256>(a, sms, st);
    if (h <= 4096) return fwd_regs<T, VEC, P, 512>(a, sms, st);
  }
  if (h <= 512) return fwd_regs<T, VEC, 2 * P, 32>(a, sms, st);
  if (h <= 1024) return fwd_regs<T, VEC, 4 * P, 32>(a, sms, st);
  if (h <= 2048) return fwd_regs<T, VEC, 2 * P, 128>(a, sms, st);
  if (h <= 4096) return fwd_regs<T, VEC, 4 * P, 128>(a, sms, st);
  if (h <= 8192) return fwd_regs<T, VEC, 2 * P, 512>(a, sms, st);
  if (h <= 16384) return fwd_regs<T, VEC, 4 * P, 512>(a, sms, st);
  *taken = false;
  return cudaSuccess;
}

template <typename T>
cudaError_t fwd(const moe_norm_dims& d, const void* x, const void* res, const void* w, const void* b, void* y,
                void* sum, float* mean, float* rstd, int sms, cudaStream_t st, int* launches) {
  FwdArgs a = {x, res, w, b, y, sum, mean, rstd, (int)d.T, (int)d.H, d.kind == MOE_NORM_RMS, d.eps};
  *launches += 1;
  constexpr int V = 16 / sizeof(T);
  bool taken;
  const cudaError_t e = d.H % V ? fwd_vec<T, 1>(a, sms, st, &taken) : fwd_vec<T, V>(a, sms, st, &taken);
  if (taken) return e;
  const int grid = (int)std::min<int64_t>(d.T, (int64_t)sms * 8);
  MOE_LAUNCH(k_norm_fwd_long<T>, grid, 256, 0, st, (const T*)x, (const T*)res, (const T*)w, (const T*)b, (T*)y,
             (T*)sum, mean, rstd, a.rows, a.H, a.rms, a.eps);
  return cudaSuccess;
}

// Blocks of the backward: as many as fit at once or the rows need; two rows a group and fewer stay in
// one block, which needs no second kernel.
int bwd_blocks_needed(int rows, int groups) { return rows <= 2 * groups ? 1 : (int)(((int64_t)rows + groups - 1) / groups); }

template <typename T, int EPT, int G>
cudaError_t bwd_ring(const BwdArgs& a, int sms, cudaStream_t st, int* chunks) {
  constexpr int VPT = EPT * (int)sizeof(T) / 16, stage = 3 * VPT * 512 * 16, groups = 512 / G;
  constexpr int stages = 196608 / stage < 4 ? 196608 / stage : 4;
  static_assert(stages >= 2 && stages * stage >= (int)sizeof(float) * 2 * G * EPT, "ring too small");
  static std::atomic<int> cache{0};
  auto kern = k_norm_bwd_ring<T, VPT, G, stages>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, stages * stage);
  if (e != cudaSuccess) return e;
  *chunks = resident_blocks(kern, &cache, 512, stages * stage, bwd_blocks_needed(a.rows, groups), sms, kMaxParts);
  MOE_LAUNCH(kern, *chunks, 512, stages * stage, st, a);
  return cudaSuccess;
}

template <typename T, int VPT, int G>
cudaError_t bwd_odd(const BwdArgs& a, int sms, cudaStream_t st, int* chunks) {
  constexpr int threads = odd_threads<G>, groups = threads / G;
  constexpr size_t smem = groups > 1 ? sizeof(float) * 2 * G * VPT : 0;
  static std::atomic<int> cache{0};
  auto kern = k_norm_bwd_odd<T, VPT, G>;
  *chunks = resident_blocks(kern, &cache, threads, smem, bwd_blocks_needed(a.rows, groups), sms, kMaxParts);
  MOE_LAUNCH(kern, *chunks, threads, smem, st, a);
  return cudaSuccess;
}

// The smallest group that covers the row with the columns a thread can keep sums for: 32 elements
// in bf16, 16 in fp32 and in rows without 16-byte alignment. chunks stays 0 for longer rows.
template <typename T>
cudaError_t bwd_regs(const BwdArgs& a, int sms, cudaStream_t st, int* chunks) {
  const int h = a.H;
  *chunks = 0;
  if (h % (16 / (int)sizeof(T))) {
    if (h <= 256) return bwd_odd<T, 8, 32>(a, sms, st, chunks);
    if (h <= 1024) return bwd_odd<T, 8, 128>(a, sms, st, chunks);
    if (h <= 2048) return bwd_odd<T, 16, 128>(a, sms, st, chunks);
    if (h <= 4096) return bwd_odd<T, 8, 512>(a, sms, st, chunks);
    if (h <= 8192) return bwd_odd<T, 16, 512>(a, sms, st, chunks);
    return cudaSuccess;
  }
  if (h <= 256) return bwd_ring<T, 8, 32>(a, sms, st, chunks);
  if (h <= 512) return bwd_ring<T, 16, 32>(a, sms, st, chunks);
  if constexpr (sizeof(T) == 2) {
    if (h <= 1024) return bwd_ring<T, 32, 32>(a, sms, st, chunks);
    if (h <= 2048) return bwd_ring<T, 16, 128>(a, sms, st, chunks);
    if (h <= 4096) return bwd_ring<T, 32, 128>(a, sms, st, chunks);
    if (h <= 8192) return bwd_ring<T, 32, 256>(a, sms, st, chunks);
    if (h <= 16384) return bwd_ring<T, 32, 512>(a, sms, st, chunks);
  } else {
    if (h <= 2048) return bwd_ring<T, 16, 128>(a, sms, st, chunks);
    if (h <= 4096) return bwd_ring<T, 16, 256>(a, sms, st, chunks);
    if (h <= 8192) return bwd_ring<T, 16, 512>(a, sms, st, chunks);
  }
  return cudaSuccess;
}

template <typename T>
cudaError_t bwd(const moe_norm_dims& d, void* ws, const void* dy, const void* dsum, const void* x, const void* w,
                const float* mean, const float* rstd, void* dx, void* dw, void* db, int sms, cudaStream_t st,
                int* launches) {
  float* part = static_cast<float*>(ws);
  const int rows = (int)d.T, H = (int)d.H;
  const BwdArgs a = {dy, dsum, x, w, mean, rstd, dx, dw, db, part, rows, H};
  int chunks;
  cudaError_t e = bwd_regs<T>(a, sms, st, &chunks);
  if (e != cudaSuccess) return e;
  const int cb = (H + 31) / 32;
  if (chunks == 1) {
    *launches += 1;
    return cudaSuccess;
  }
  if (chunks) {
    *launches += 2;
    MOE_LAUNCH(k_norm_dw_sum<T>, cb, 1024, 0, st, (const float*)part, chunks, H, (T*)dw, (T*)db);
    return cudaSuccess;
  }
  const int per = (rows + kNormChunks - 1) / kNormChunks;
  chunks = (rows + per - 1) / per;
  *launches += 3;  // the weight gradients before dx, which may be written over dy
  MOE_LAUNCH(k_norm_dw_long<T>, dim3((H + 255) / 256, chunks), 256, 0, st, (const T*)dy, (const T*)x, mean, rstd, part,
             rows, H, per);
  MOE_LAUNCH(k_norm_dw_sum<T>, cb, 1024, 0, st, (const float*)part, chunks, H, (T*)dw, (T*)db);
  const int grid = (int)std::min<int64_t>(d.T, (int64_t)sms * 8);
  MOE_LAUNCH(k_norm_dx_long<T>, grid, 256, 0, st, (const T*)dy, (const T*)dsum, (const T*)x, (const T*)w, mean, rstd,
             (T*)dx, rows, H);
  return cudaSuccess;
}

}  // namespace

size_t norm_workspace_bytes(const moe_norm_dims& d) {
  // rows of partial sums: one a block (at least one row each), or the row chunks of the long rows
  const int64_t parts = std::min<int64_t>(d.T, kMaxParts);
  return (size_t)(parts * 2 * d.H) * sizeof(float) + 256;
}

cudaError_t launch_norm_fwd(const moe_norm_dims& d, const void* x, const void* residual, const void* weight,
                            const void* bias, void* y, void* sum, float* mean, float* rstd, int sms, cudaStream_t st,
                            int* launches) {
  return d.dtype == MOE_BF16
             ? fwd<__nv_bfloat16>(d, x, residual, weight, bias, y, sum, mean, rstd, sms, st, launches)
             : fwd<float>(d, x, residual, weight, bias, y, sum, mean, rstd, sms, st, launches);
}

cudaError_t launch_norm_bwd(const moe_norm_dims& d, void* ws, const void* dy, const void* dsum, const void* x,
                            const void* weight, const float* mean, const float* rstd, void* dx, void* dweight,
                            void* dbias, int sms, cudaStream_t st, int* launches) {
  return d.dtype == MOE_BF16 ? bwd<__nv_bfloat16>(d, ws, dy, dsum, x, weight, mean, rstd, dx, dweight, dbias, sms, st,
                                                  launches)
                             : bwd<float>(d, ws, dy, dsum, x, weight, mean, rstd, dx, dweight, dbias, sms, st,
                                          launches);
}

}  // namespace moe
