// optim.cu -- gradient norm and AdamW step over many tensors, states in 32 or in 8 bits.
//
//   norm = grad_scale sqrt(sum g^2);   g' = g grad_scale min(1, max_norm / norm)
//   m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2;  p -= lr (m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps) + wd p)
//
// Bound by HBM: every value is read once and written once. The tensors' descriptions travel as kernel arguments, so
// that a launch needs no table on the device and a captured one keeps its own. The values of all tensors are cut into
// chunks that never cross a tensor; persistent blocks walk them.
//
// 8 bits: m and r = sqrt(v) are held as e4m3 (3 bits of mantissa, 17 powers of two) over a float for each 256 values,
// their largest magnitude / 448. The root halves the span of exponents that v has. An r above zero never becomes zero:
// it would divide m by eps alone. Weights use the new m and r before they are rounded. A value that is not finite is
// stored as NaN and left out of its block's largest, so that it stays alone.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "block.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kBlock = 256;     // values that share a scale; a warp's step
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSteps = 2;       // a warp's steps in a chunk
constexpr int kChunk = kWarps * kSteps * kBlock;

struct Entry {
  void* p;
  const void* g;
  float* master;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t n;
  uint32_t first;   // its first chunk
  uint32_t types;   // bit 0: p is bf16, bit 1: g is bf16
  float lr_scale, wd;
};

template <int N>
struct Table {
  uint32_t count, chunks;
  Entry e[N];
};

// The tensor of a chunk, from the one that an earlier chunk was in.
template <int N>
__device__ __forceinline__ uint32_t tensor_of(const Table<N>& t, uint32_t chunk, uint32_t at) {
  uint32_t lo = at, hi = t.count;
  if (at + 1 == hi || t.e[at + 1].first > chunk) return at;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) >> 1;
    if (t.e[mid].first <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Four values from element i of an array of n (bf16 or float), zeros past its end.
__device__ __forceinline__ void load4(const void* a, bool bf, int64_t i, int64_t n, float (&f)[4]) {
  if (bf) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a) + i;
    if (i + 4 <= n) {
      const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
      f[0] = __uint_as_float(u.x << 16);
      f[1] = __uint_as_float(u.x & 0xffff0000u);
      f[2] = __uint_as_float(u.y << 16);
      f[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = i + j < n ? __bfloat162float(p[j]) : 0.0f;
    }
  } else {
    const float* p = static_cast<const float*>(a) + i;
    if (i + 4 <= n) {
      const float4 u = __ldcs(reinterpret_cast<const float4*>(p));
      f[0] = u.x;
      f[1] = u.y;
      f[2] = u.z;
      f[3] = u.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = i + j < n ? p[j] : 0.0f;
    }
  }
}
__device__ __forceinline__ void store4(void* a, bool bf, int64_t i, int64_t n, const float (&f)[4]) {
  if (bf) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a) + i;
    if (i + 4 <= n) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(f[0], f[1]), y = __floats2bfloat162_rn(f[2], f[3]);
      __stcs(reinterpret_cast<uint2*>(p),
             make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y)));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) p[j] = __float2bfloat16_rn(f[j]);
    }
  } else {
    float* p = static_cast<float*>(a) + i;
    if (i + 4 <= n) {
      __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) p[j] = f[j];
    }
  }
}

// Four e4m3 codes and their values.
__device__ __forceinline__ uint32_t load_codes(const void* a, int64_t i, int64_t n) {
  const uint8_t* p = static_cast<const uint8_t*>(a) + i;
  if (i + 4 <= n) return __ldcs(reinterpret_cast<const uint32_t*>(p));
  uint32_t u = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (i + j < n) u |= (uint32_t)p[j] << (8 * j);
  return u;
}
__device__ __forceinline__ void store_codes(void* a, int64_t i, int64_t n, uint32_t u) {
  uint8_t* p = static_cast<uint8_t*>(a) + i;
  if (i + 4 <= n) {
    __stcs(reinterpret_cast<uint32_t*>(p), u);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (i + j < n) p[j] = (uint8_t)(u >> (8 * j));
}
__device__ __forceinline__ void decode4(uint32_t u, float scale, float (&f)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> (16 * h)), __NV_E4M3);
    const float2 t = __half22float2(__half2(r));
    f[2 * h] = t.x * scale;
    f[2 * h + 1] = t.y * scale;
  }
}
__device__ __forceinline__ uint32_t encode4(const float (&f)[4]) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}

// The scale of a block's values: the warp's largest finite magnitude / 448, at least the smallest normal float.
// A value that is not finite becomes NaN.
__device__ __forceinline__ float block_scale(float (&x)[2][4]) {
  uint32_t big = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) big = max(big, __float_as_uint(x[h][j]) & 0x7fffffffu);
  big = __reduce_max_sync(0xffffffffu, big);
  if (big >= 0x7f800000u) {
    big = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t u = __float_as_uint(x[h][j]) & 0x7fffffffu;
        if (u >= 0x7f800000u) x[h][j] = __uint_as_float(0x7fffffffu);
        else big = max(big, u);
      }
    big = __reduce_max_sync(0xffffffffu, big);
  }
  return fmaxf(__uint_as_float(big) * (1.0f / 448.0f), 1.17549435e-38f);
}

__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct AdamWArgs {
  float lr, b1, b2, c1, c2;   // c = 1 - b
  float eps, wide, bc1, bc2;  // wide: grad_scale; bc1 = 1 / (1 - b1^t), bc2 = 1 / sqrt(1 - b2^t)
  float max_norm, ln_b1, ln_b2;
  const float* norm;
  const float* lr_at;
  const int* step_at;
};

template <int BITS, int N>
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ Table<N> tab, const AdamWArgs a) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  float gs = a.wide, lr = a.lr, bc1 = a.bc1, bc2 = a.bc2;
  if (a.norm) {
    const float n = *a.norm;
    if (!(fabsf(n) < INFINITY)) return;  // a step on such gradients would destroy the weights: none is made
    if (a.max_norm > 0.0f) gs *= a.max_norm / fmaxf(n, a.max_norm);
  }
  if (a.lr_at) lr = *a.lr_at;
  if (a.step_at) {
    const float t = (float)*a.step_at;
    bc1 = -1.0f / expm1f(t * a.ln_b1);
    bc2 = rsqrtf(-expm1f(t * a.ln_b2));
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t at = 0;
  for (uint32_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
    at = tensor_of(tab, chunk, at);
    const Entry& e = tab.e[at];
    const bool pb = e.types & 1, gb = e.types & 2;
    const float elr = lr * e.lr_scale, wd = e.wd;
#pragma unroll
    for (int step = 0; step < kSteps; ++step) {
      const int64_t blk = (int64_t)(chunk - e.first) * (kWarps * kSteps) + step * kWarps + warp;
      const int64_t i0 = blk * kBlock + lane * 4, n = e.n;
      if (blk * kBlock >= n) break;
      float p[2][4], g[2][4], m[2][4], v[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t i = i0 + h * 128;
        load4(e.g, gb, i, n, g[h]);
        if (e.master) load4(e.master, false, i, n, p[h]);
        else load4(e.p, pb, i, n, p[h]);
        if constexpr (BITS == 32) {
          load4(e.m, false, i, n, m[h]);
          load4(e.v, false, i, n, v[h]);
        } else {
          decode4(load_codes(e.m, i, n), e.ms[blk], m[h]);
          decode4(load_codes(e.v, i, n), e.vs[blk], v[h]);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float gg = g[h][j] * gs;
          const float vo = BITS == 8 ? v[h][j] * v[h][j] : v[h][j];
          m[h][j] = a.b1 * m[h][j] + a.c1 * gg;
          const float vn = a.b2 * vo + a.c2 * (gg * gg);
          const float r = sqrt_approx(vn);
          v[h][j] = BITS == 8 ? r : vn;
          p[h][j] -= elr * (__fdividef(m[h][j] * bc1, r * bc2 + a.eps) + wd * p[h][j]);
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t i = i0 + h * 128;
        if (e.master) store4(e.master, false, i, n, p[h]);
        store4(e.p, pb, i, n, p[h]);
        if constexpr (BITS == 32) {
          store4(e.m, false, i, n, m[h]);
          store4(e.v, false, i, n, v[h]);
        }
      }
      if constexpr (BITS == 8) {
        const float ms = block_scale(m), vs = block_scale(v), mi = 1.0f / ms, vi = 1.0f / vs;
        if (lane == 0) {
          e.ms[blk] = ms;
          e.vs[blk] = vs;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[4], y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[j] = m[h][j] * mi;
            y[j] = v[h][j] * vi;
            if (v[h][j] > 0.0f && y[j] < 0.001953125f) y[j] = 0.001953125f;  // 2^-9, the smallest e4m3
          }
          store_codes(e.m, i0 + h * 128, n, encode4(x));
          store_codes(e.v, i0 + h * 128, n, encode4(y));
        }
      }
    }
  }
}

// ---------------------------------------------------------------- norm
constexpr int kNormChunk = kThreads * 32;  // values: four 16-byte loads a thread in bf16

// A block's sum of squares over its chunks; the last block of the last launch adds the blocks' in order.
template <int N>
__global__ void __launch_bounds__(kThreads) k_grad_norm(const __grid_constant__ Table<N> tab, float* part, int part0,
                                                        int parts, unsigned* done, float scale, float* norm) {
  __shared__ float red[kWarps];
  __shared__ double wide[kWarps];
  __shared__ bool last;
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t at = 0;
  float sum = 0.0f;
  for (uint32_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
    at = tensor_of(tab, chunk, at);
    const Entry& e = tab.e[at];
    const bool gb = e.types & 2;
    const int64_t i0 = (int64_t)(chunk - e.first) * kNormChunk + threadIdx.x * 4;
    float f[8][4];
#pragma unroll
    for (int u = 0; u < 8; ++u) load4(e.g, gb, i0 + u * kThreads * 4, e.n, f[u]);
#pragma unroll
    for (int u = 0; u < 8; ++u) sum += (f[u][0] * f[u][0] + f[u][1] * f[u][1]) + (f[u][2] * f[u][2] + f[u][3] * f[u][3]);
  }
  sum = warp_sum(sum);
  if (lane == 0) red[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kWarps; ++w) sum += red[w];
    part[part0 + blockIdx.x] = sum;
    __threadfence();
    last = norm && atomicAdd(done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double d = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) d += (double)__ldcg(part + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (lane == 0) wide[warp] = d;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kWarps; ++w) d += wide[w];
    *norm = (float)(sqrt(d) * (double)fabsf(scale));
    *done = 0;
  }
}

// ---------------------------------------------------------------- host side
constexpr int kMany = 384, kFew = 24;  // 80 bytes a tensor: kernel arguments hold 32764
static_assert(sizeof(Table<kMany>) + sizeof(AdamWArgs) <= 32764, "kernel arguments");
constexpr int kBlocksPerSm = 8;  // of kThreads
constexpr int kNormBlocks = 2048;  // at most, whatever the device

// Fills a table with tensors [from, ...) as far as it goes; returns how many of the list it took.
template <int N>
int64_t fill(Table<N>* t, const moe_adamw_tensor* list, int64_t count, int64_t chunk) {
  t->count = 0;
  uint64_t chunks = 0;
  int64_t i = 0;
  for (; i < count && t->count < N; ++i) {
    const moe_adamw_tensor& s = list[i];
    if (s.n == 0) continue;
    const uint64_t c = (uint64_t)((s.n + chunk - 1) / chunk);
    if (chunks + c >= (1ull << 31)) break;  // the rest in another launch
    Entry& e = t->e[t->count++];
    e = {s.param, s.grad, s.master, s.m, s.v, s.m_scale, s.v_scale, s.n, (uint32_t)chunks,
         (uint32_t)(s.dtype == MOE_BF16) | (uint32_t)(s.grad_dtype == MOE_BF16) << 1, s.lr_scale, s.weight_decay};
    chunks += c;
  }
  t->chunks = (uint32_t)chunks;
  return i;
}

int grid_of(uint32_t chunks, int sms) { return (int)std::min<int64_t>(chunks, (int64_t)sms * kBlocksPerSm); }

template <int N>
cudaError_t adamw_launches(int bits, const AdamWArgs& a, const moe_adamw_tensor* list, int64_t count, int sms,
                           cudaStream_t st, int* launches) {
  Table<N> t;
  while (count > 0) {
    const int64_t took = fill(&t, list, count, kChunk);
    list += took;
    count -= took;
    if (!t.count) continue;
    *launches += 1;
    if (bits == 8) MOE_LAUNCH((k_adamw<8, N>), grid_of(t.chunks, sms), kThreads, 0, st, t, a);
    else MOE_LAUNCH((k_adamw<32, N>), grid_of(t.chunks, sms), kThreads, 0, st, t, a);
  }
  return cudaSuccess;
}

template <int N>
cudaError_t norm_launches(char* ws, const moe_adamw_tensor* list, int64_t count, float scale, float* norm, int sms,
                          cudaStream_t st, int* launches) {
  Table<N> t;
  float* part = reinterpret_cast<float*>(ws + kNormHeader);
  unsigned* done = reinterpret_cast<unsigned*>(ws + 64);
  int part0 = 0;
  do {
    const int64_t took = fill(&t, list, count, kNormChunk);
    list += took;
    count -= took;
    while (count > 0 && list->n == 0) ++list, --count;  // the launch with the last values is the one that finishes
    const int grid = std::max(1, std::min(kNormBlocks, grid_of(t.chunks, sms)));  // no value at all: one block writes a norm of zero
    *launches += 1;
    MOE_LAUNCH((k_grad_norm<N>), grid, kThreads, 0, st, t, part, part0, part0 + grid, done, scale,
               count > 0 ? nullptr : norm);
    part0 += grid;
  } while (count > 0);
  return cudaSuccess;
}

}  // namespace

// Every launch leaves a sum for each of its blocks.
size_t grad_norm_workspace_bytes(const moe_adamw_tensor* list, int64_t count) {
  uint64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i) chunks += (uint64_t)((list[i].n + kNormChunk - 1) / kNormChunk);
  const uint64_t launches = (uint64_t)(count + kMany - 1) / kMany + (chunks >> 30) + 1;
  return kNormHeader + (size_t)((launches * kNormBlocks * 4 + 255) / 256 * 256);
}

cudaError_t launch_grad_norm(void* ws, const moe_adamw_tensor* list, int64_t count, float scale, float* norm, int sms,
                             cudaStream_t st, int* launches) {
  // arguments are copied with every launch: a short list takes a short table
  return count <= kFew ? norm_launches<kFew>(static_cast<char*>(ws), list, count, scale, norm, sms, st, launches)
                       : norm_launches<kMany>(static_cast<char*>(ws), list, count, scale, norm, sms, st, launches);
}

cudaError_t launch_adamw(const moe_adamw_dims& d, const moe_adamw_tensor* list, int64_t count, const float* norm,
                         const float* lr, const int* step, int sms, cudaStream_t st, int* launches) {
  AdamWArgs a = {};
  a.lr = d.lr;
  a.b1 = (float)d.beta1;
  a.b2 = (float)d.beta2;
  a.c1 = (float)(1.0 - d.beta1);
  a.c2 = (float)(1.0 - d.beta2);
  a.eps = d.eps;
  a.wide = d.grad_scale;
  a.bc1 = (float)(1.0 / (1.0 - std::pow(d.beta1, (double)d.step)));
  a.bc2 = (float)(1.0 / std::sqrt(1.0 - std::pow(d.beta2, (double)d.step)));
  a.ln_b1 = d.beta1 > 0.0 ? (float)std::log(d.beta1) : -INFINITY;
  a.ln_b2 = d.beta2 > 0.0 ? (float)std::log(d.beta2) : -INFINITY;
  a.max_norm = d.max_norm;
  a.norm = norm;
  a.lr_at = lr;
  a.step_at = step;
  return count <= kFew ? adamw_launches<kFew>(d.state_bits, a, list, count, sms, st, launches)
                       : adamw_launches<kMany>(d.state_bits, a, list, count, sms, st, launches);
}

}  // namespace moe
