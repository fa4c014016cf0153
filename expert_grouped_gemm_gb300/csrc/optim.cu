// optim.cu -- gradient norm and AdamW step over many tensors, states in 32 or in 8 bits.
//
//   norm = grad_scale sqrt(sum g^2);   g' = g grad_scale min(1, max_norm / norm)
//   m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2;  p -= lr (m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps) + wd p)
//
// Bound by HBM: every value is read once and written once. The tensors' descriptions travel as kernel arguments, so
// that a launch needs no table on the device and a captured one keeps its own. The values of all tensors are cut into
// chunks that never cross a tensor. With 32 bits a block takes one chunk (604M values in 2.40 ms, 7.1 TB/s; resident
// blocks that walk 2.68); with 8 bits, where instructions count beside bytes (37 a value), resident blocks walk them
// (1.08 ms, 5.6 TB/s; a block each 6% more). The norm of 604M bf16 values takes 175 us (7.0 TB/s).
//
// 8 bits: m and r = sqrt(v) are held as e4m3 (3 bits of mantissa, 17 powers of two) over a float for each 256 values,
// their largest magnitude / 448. The root halves the span of exponents that v has. An r above zero never becomes zero:
// it would divide m by eps alone. Weights use the new m and r before they are rounded. A value that is not finite is
// stored as NaN and left out of its block's largest, so that it stays alone.
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "block.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int kBlock = 256;     // values that share a scale; a warp's step
constexpr int kThreads = 256, kWarps = kThreads / 32;
// A warp's blocks in a chunk: their loads are in flight together. Two where the states have 8 bits and a block is 1.5 KB;
// with 32 bits one has 3.6 KB, and more of them cost registers that more warps use better.
template <int BITS>
constexpr int steps_of = BITS == 8 ? 2 : 1;
template <int BITS>
constexpr int chunk_of = kWarps * steps_of<BITS> * kBlock;

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

// The same for the norm.
struct Grad {
  const void* g;
  int64_t n;
  uint32_t first;
  uint32_t types;
};

constexpr int kMap = 1024;
template <typename E, int N>
struct Table {
  uint32_t count, chunks;
  uint16_t map[kMap];  // a chunk's tensor, where there are no more chunks: a search would wait for every step
  E e[N];
};

// The tensor of a chunk, from the one that an earlier chunk was in.
template <typename E, int N>
__device__ __forceinline__ uint32_t tensor_of(const Table<E, N>& t, uint32_t chunk, uint32_t at) {
  if (t.chunks <= kMap) return t.map[chunk];
  uint32_t lo = at, hi = t.count;
  if (at + 1 == hi || t.e[at + 1].first > chunk) return at;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) >> 1;
    if (t.e[mid].first <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Four neighbouring values: as they lie in memory, and as floats.
template <bool BF>
struct Four;
template <>
struct Four<true> {
  uint2 u;
  __device__ __forceinline__ void load(const void* a, int64_t i) {
    u = __ldcg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a) + i));
  }
  __device__ __forceinline__ void get(float (&f)[4]) const {
    f[0] = __uint_as_float(u.x << 16);
    f[1] = __uint_as_float(u.x & 0xffff0000u);
    f[2] = __uint_as_float(u.y << 16);
    f[3] = __uint_as_float(u.y & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(void* a, int64_t i, const float (&f)[4]) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(f[0], f[1]), y = __floats2bfloat162_rn(f[2], f[3]);
    __stcg(reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a) + i),
           make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y)));
  }
};
template <>
struct Four<false> {
  float4 u;
  __device__ __forceinline__ void load(const void* a, int64_t i) {
    u = __ldcg(reinterpret_cast<const float4*>(static_cast<const float*>(a) + i));
  }
  __device__ __forceinline__ void get(float (&f)[4]) const {
    f[0] = u.x;
    f[1] = u.y;
    f[2] = u.z;
    f[3] = u.w;
  }
  static __device__ __forceinline__ void store(void* a, int64_t i, const float (&f)[4]) {
    __stcg(reinterpret_cast<float4*>(static_cast<float*>(a) + i), make_float4(f[0], f[1], f[2], f[3]));
  }
};

// The same at the end of an array of n, value by value; zeros past it.
__device__ __forceinline__ void load_tail(const void* a, bool bf, int64_t i, int64_t n, float (&f)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    f[j] = i + j >= n ? 0.0f : bf ? __bfloat162float(static_cast<const __nv_bfloat16*>(a)[i + j]) : static_cast<const float*>(a)[i + j];
}
__device__ __forceinline__ void store_tail(void* a, bool bf, int64_t i, int64_t n, const float (&f)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (i + j >= n) break;
    if (bf) static_cast<__nv_bfloat16*>(a)[i + j] = __float2bfloat16_rn(f[j]);
    else static_cast<float*>(a)[i + j] = f[j];
  }
}

// Four e4m3 codes: their values, and the codes of four values.
__device__ __forceinline__ void decode4(uint32_t u, float (&f)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u >> (16 * h)), __NV_E4M3);
    const float2 t = __half22float2(__half2(r));
    f[2 * h] = t.x;
    f[2 * h + 1] = t.y;
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
  float big = 0.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) big = fmaxf(big, fabsf(x[h][j]));  // passes over NaN
  uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
  if (most == 0x7f800000u) {
    big = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (fabsf(x[h][j]) < INFINITY) big = fmaxf(big, fabsf(x[h][j]));
        else x[h][j] = __uint_as_float(0x7fffffffu);
      }
    most = __reduce_max_sync(0xffffffffu, __float_as_uint(big));
  }
  return fmaxf(__uint_as_float(most) * (1.0f / 448.0f), 1.17549435e-38f);
}

struct AdamWArgs {
  float lr, b1, b2, c1, c2;   // c = 1 - b
  float eps, wide, bc1, bc2;  // wide: grad_scale; bc1 = 1 / (1 - b1^t), bc2 = 1 / sqrt(1 - b2^t)
  float max_norm, ln_b1, ln_b2;
  const float* norm;
  const float* lr_at;
  const int* step_at;
};

// What the values of a tensor share in a step.
struct Factors {
  float gs, b1, c1, b2, c2, bc2, eps;  // gs: the gradients' factor
  // w = w + (-decay w - move m / (r bc2 + eps)). The decay joins the change, not a factor 1 - decay: a float next to one
  // is off by up to 2^-25, the same way for every value and step (lr 1e-5 with a decay of 0.01: 1.19 times it).
  float decay, move;
};

// Two floats in one 64-bit operand: the same roundings in half the instructions.
typedef uint64_t f2;
__device__ __forceinline__ f2 two(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void apart(f2 x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 both(float a) { return two(a, a); }

// An infinite weight is an entry that a program has masked. It keeps its value: what decays is the largest float, since
// inf against inf, or 0 inf, is NaN.
__device__ __forceinline__ float finite(float a) {
  asm("min.xorsign.abs.f32 %0, %0, %1;" : "+f"(a) : "f"(3.40282347e38f));
  return a;
}

// The root's correction needs a residual that is a float: below 2^-100 its last bits pass the smallest one, 2^-149.
// Smaller v, zero and what is not finite take the library's root.
constexpr uint32_t kRootMin = 0x0d800000u;  // 2^-100

// The step of four values of a block; with 8 bits m and v hold codes' values, sm and sv what they are multiples of, and
// v receives r = sqrt(v). Roundings are those of m = c1 g + (b1 m), v = c2 (g g) + (b2 v) with fused last steps, whatever
// the compiler would join otherwise: in 8 bits a last bit can decide between two codes. For the same reason r is the
// rounded root: an approximate one and one correction by the residual v - r^2 (P. Markstein, IBM J. Res. Develop. 34, 1990).
// That it is the rounded one rests on how far the approximation is off: compared with __fsqrt_rn, all mantissas of every
// pair of exponents from 2^-100 to 2^126 are equal.
template <int BITS>
__device__ __forceinline__ void update4(const Factors& k, float sm, float sv, const float (&g)[4], float (&p)[4],
                                        float (&m)[4], float (&v)[4]) {
  float r[4];
  uint32_t far = 0;
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const f2 gg = mul2(two(g[j], g[j + 1]), both(k.gs));
    f2 mo = two(m[j], m[j + 1]), vo = two(v[j], v[j + 1]);
    if constexpr (BITS == 8) {
      mo = mul2(mo, both(sm));
      const f2 ro = mul2(vo, both(sv));
      vo = mul2(ro, ro);
    }
    const f2 mn = fma2(both(k.c1), gg, mul2(both(k.b1), mo));
    const f2 vn = fma2(both(k.c2), mul2(gg, gg), mul2(both(k.b2), vo));
    apart(mn, m[j], m[j + 1]);
    apart(vn, v[j], v[j + 1]);
    if constexpr (BITS == 8) {
      float y[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y[i]) : "f"(v[j + i]));
        far = max(far, __float_as_uint(v[j + i]) - kRootMin);
      }
      const f2 y2 = two(y[0], y[1]), r0 = mul2(vn, y2), half = mul2(y2, both(0.5f));
      apart(fma2(fma2(mul2(r0, both(-1.0f)), r0, vn), half, r0), r[j], r[j + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) asm("sqrt.approx.f32 %0, %1;" : "=f"(r[j + i]) : "f"(v[j + i]));
    }
  }
  if constexpr (BITS == 8) {
    if (far >= 0x7f800000u - kRootMin) {
#pragma unroll
      for (int j = 0; j < 4; ++j) r[j] = __fsqrt_rn(v[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    float den[2], inv[2];
    apart(fma2(two(r[j], r[j + 1]), both(k.bc2), both(k.eps)), den[0], den[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv[i]) : "f"(den[i]));
    const f2 move = mul2(mul2(two(m[j], m[j + 1]), both(-k.move)), two(inv[0], inv[1]));
    const f2 w = two(finite(p[j]), finite(p[j + 1]));
    apart(add2(two(p[j], p[j + 1]), fma2(both(-k.decay), w, move)), p[j], p[j + 1]);
    if constexpr (BITS == 8) {
      v[j] = r[j];
      v[j + 1] = r[j + 1];
    }
  }
}

// m and r of a block as codes over new scales. x / scale is the rounded quotient, or nearly always: with the rounded
// reciprocal, one correction of the product by its residual (the same paper). Of 6e10 quotients of x from 2^-101 on, all
// mantissas over 4096 scales among them, none differs from the division; below, the residual passes the smallest float and
// one in 2e6 is off by its last bit.
__device__ __forceinline__ void codes4(const float (&x)[4], float scale, float inv, bool root, uint32_t& code) {
  float q[4];
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const f2 a = two(x[j], x[j + 1]), q0 = mul2(a, both(inv));
    apart(fma2(fma2(q0, both(-scale), a), both(inv), q0), q[j], q[j + 1]);
  }
  if (root) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (x[j] > 0.0f) q[j] = fmaxf(q[j], 0.001953125f);  // 2^-9, the smallest e4m3
  }
  code = encode4(q);
}
__device__ __forceinline__ void pack_block(const Entry& e, int64_t blk, int lane, float (&m)[2][4], float (&r)[2][4],
                                           uint32_t (&mc)[2], uint32_t (&rc)[2]) {
  const float ms = block_scale(m), rs = block_scale(r), mi = 1.0f / ms, ri = 1.0f / rs;
  if (lane == 0) {
    e.ms[blk] = ms;
    e.vs[blk] = rs;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    codes4(m[h], ms, mi, false, mc[h]);
    codes4(r[h], rs, ri, true, rc[h]);
  }
}

// Whole blocks blk, blk + kWarps, ... (`steps` of them) of a tensor: every load is sent for before the first is used.
template <int BITS, int kSteps, bool PB, bool GB, bool MASTER>
__device__ __forceinline__ void whole_blocks(const Entry& e, const Factors& k, int64_t blk, int lane) {
  Four<GB> g[kSteps][2];
  Four<MASTER ? false : PB> p[kSteps][2];
  Four<false> m[BITS == 32 ? kSteps : 1][2], v[BITS == 32 ? kSteps : 1][2];
  uint32_t mc[BITS == 8 ? kSteps : 1][2], vc[BITS == 8 ? kSteps : 1][2];
  float sm[kSteps], sv[kSteps];
  const void* w = MASTER ? e.master : e.p;
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int64_t b = blk + s * kWarps, i = b * kBlock + lane * 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      g[s][h].load(e.g, i + h * 128);
      p[s][h].load(w, i + h * 128);
      if constexpr (BITS == 32) {
        m[s][h].load(e.m, i + h * 128);
        v[s][h].load(e.v, i + h * 128);
      } else {
        mc[s][h] = __ldcg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(e.m) + i + h * 128));
        vc[s][h] = __ldcg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(e.v) + i + h * 128));
      }
    }
    sm[s] = BITS == 8 ? e.ms[b] : 1.0f;
    sv[s] = BITS == 8 ? e.vs[b] : 1.0f;
  }
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int64_t b = blk + s * kWarps, i = b * kBlock + lane * 4;
    float mf[2][4], vf[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float gf[4], pf[4];
      g[s][h].get(gf);
      p[s][h].get(pf);
      if constexpr (BITS == 32) {
        m[s][h].get(mf[h]);
        v[s][h].get(vf[h]);
      } else {
        decode4(mc[s][h], mf[h]);
        decode4(vc[s][h], vf[h]);
      }
      update4<BITS>(k, sm[s], sv[s], gf, pf, mf[h], vf[h]);
      if constexpr (MASTER) Four<false>::store(e.master, i + h * 128, pf);
      Four<PB>::store(e.p, i + h * 128, pf);
      if constexpr (BITS == 32) {
        Four<false>::store(e.m, i + h * 128, mf[h]);
        Four<false>::store(e.v, i + h * 128, vf[h]);
      }
    }
    if constexpr (BITS == 8) {
      uint32_t mo[2], vo[2];
      pack_block(e, b, lane, mf, vf, mo, vo);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        __stcg(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(e.m) + i + h * 128), mo[h]);
        __stcg(reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(e.v) + i + h * 128), vo[h]);
      }
    }
  }
}

template <int BITS, int kSteps>
__device__ __forceinline__ void whole_blocks(const Entry& e, const Factors& k, int64_t blk, int lane) {
  if (e.master) {
    if (e.types & 2) whole_blocks<BITS, kSteps, true, true, true>(e, k, blk, lane);
    else whole_blocks<BITS, kSteps, true, false, true>(e, k, blk, lane);
  } else if (e.types & 1) {
    if (e.types & 2) whole_blocks<BITS, kSteps, true, true, false>(e, k, blk, lane);
    else whole_blocks<BITS, kSteps, true, false, false>(e, k, blk, lane);
  } else {
    if (e.types & 2) whole_blocks<BITS, kSteps, false, true, false>(e, k, blk, lane);
    else whole_blocks<BITS, kSteps, false, false, false>(e, k, blk, lane);
  }
}

// The block that a tensor ends in.
template <int BITS>
__device__ __forceinline__ void last_block(const Entry& e, const Factors& k, int64_t blk, int lane) {
  const bool pb = e.types & 1, gb = e.types & 2;
  const int64_t i = blk * kBlock + lane * 4, n = e.n;
  float gf[2][4], pf[2][4], mf[2][4], vf[2][4], sm = 1.0f, sv = 1.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t at = i + h * 128;
    load_tail(e.g, gb, at, n, gf[h]);
    load_tail(e.master ? e.master : e.p, e.master ? false : pb, at, n, pf[h]);
    if constexpr (BITS == 32) {
      load_tail(e.m, false, at, n, mf[h]);
      load_tail(e.v, false, at, n, vf[h]);
    } else {
      uint32_t mc = 0, vc = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (at + j < n) {
          mc |= (uint32_t)static_cast<const uint8_t*>(e.m)[at + j] << (8 * j);
          vc |= (uint32_t)static_cast<const uint8_t*>(e.v)[at + j] << (8 * j);
        }
      decode4(mc, mf[h]);
      decode4(vc, vf[h]);
    }
  }
  if constexpr (BITS == 8) {
    sm = e.ms[blk];
    sv = e.vs[blk];
    __syncwarp();  // every lane has read the block's scales before one is written
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t at = i + h * 128;
    update4<BITS>(k, sm, sv, gf[h], pf[h], mf[h], vf[h]);
    if (e.master) store_tail(e.master, false, at, n, pf[h]);
    store_tail(e.p, pb, at, n, pf[h]);
    if constexpr (BITS == 32) {
      store_tail(e.m, false, at, n, mf[h]);
      store_tail(e.v, false, at, n, vf[h]);
    }
  }
  if constexpr (BITS == 8) {
    uint32_t mo[2], vo[2];
    pack_block(e, blk, lane, mf, vf, mo, vo);
    for (int h = 0; h < 2; ++h)
      for (int j = 0; j < 4; ++j)
        if (i + h * 128 + j < n) {
          static_cast<uint8_t*>(e.m)[i + h * 128 + j] = (uint8_t)(mo[h] >> (8 * j));
          static_cast<uint8_t*>(e.v)[i + h * 128 + j] = (uint8_t)(vo[h] >> (8 * j));
        }
  }
}

template <int BITS, int N>
__global__ void __launch_bounds__(kThreads, 4) k_adamw(const __grid_constant__ Table<Entry, N> tab, const AdamWArgs a) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  float gs = a.wide, lr = a.lr, bc1 = a.bc1, bc2 = a.bc2;
  if (a.norm) {
    const float n = *a.norm;
    if (!(fabsf(n) < INFINITY)) return;  // a step on such gradients would destroy the weights: none is made
    if (a.max_norm > 0.0f && n > a.max_norm) gs *= a.max_norm / n;  // no quotient of two infinities
  }
  if (a.lr_at) lr = *a.lr_at;
  if (a.step_at) {
    const float t = fmaxf((float)*a.step_at, 1.0f);
    bc1 = -1.0f / expm1f(t * a.ln_b1);
    bc2 = rsqrtf(-expm1f(t * a.ln_b2));
  }
  Factors k = {gs, a.b1, a.c1, a.b2, a.c2, bc2, a.eps, 0.0f, 0.0f};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t at = 0;
  for (uint32_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
    at = tensor_of(tab, chunk, at);
    const Entry& e = tab.e[at];
    const float elr = lr * e.lr_scale;
    k.decay = elr * e.wd;
    k.move = elr * bc1;
    constexpr int kSteps = steps_of<BITS>;
    const int64_t blk0 = (int64_t)(chunk - e.first) * (kWarps * kSteps), blk = blk0 + warp;
    if (kSteps > 1 && (blk0 + kWarps * kSteps) * kBlock <= e.n) {
      whole_blocks<BITS, kSteps>(e, k, blk, lane);
    } else {
      for (int s = 0; s < kSteps; ++s) {
        const int64_t b = blk + s * kWarps;
        if ((b + 1) * kBlock <= e.n) whole_blocks<BITS, 1>(e, k, b, lane);
        else if (b * kBlock < e.n) last_block<BITS>(e, k, b, lane);
      }
    }
  }
}

// ---------------------------------------------------------------- norm
constexpr int kNormChunk = kThreads * 32;  // values: four 16-byte loads a thread in bf16, in flight together

// This thread's squares of the n values of a chunk, four 16-byte loads in flight.
template <bool BF>
__device__ __forceinline__ float squares(const void* g, int n) {
  constexpr int V = BF ? 8 : 4;
  const uint4* p = static_cast<const uint4*>(g);
  const int vecs = n / V;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kNormChunk / V; i += 4 * kThreads) {
    uint4 u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = i + j * kThreads + threadIdx.x;
      u[j] = at < vecs ? __ldcg(p + at) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[V];
      if constexpr (BF) {
        bf16x8_to_f(u[j], f);
      } else {
        f[0] = __uint_as_float(u[j].x);
        f[1] = __uint_as_float(u[j].y);
        f[2] = __uint_as_float(u[j].z);
        f[3] = __uint_as_float(u[j].w);
      }
      float s = (f[0] * f[0] + f[1] * f[1]) + (f[2] * f[2] + f[3] * f[3]);
      if constexpr (BF) s += (f[4] * f[4] + f[5] * f[5]) + (f[6] * f[6] + f[7] * f[7]);
      sum += s;
    }
  }
  const int at = vecs * V + threadIdx.x;
  if (at < n) {
    const float f = BF ? __bfloat162float(static_cast<const __nv_bfloat16*>(g)[at]) : static_cast<const float*>(g)[at];
    sum += f * f;
  }
  return sum;
}

// A block's sum of squares over its chunks; the last block of the last launch adds the blocks' in order.
template <int N>
__global__ void __launch_bounds__(kThreads) k_grad_norm(const __grid_constant__ Table<Grad, N> tab, float* part, int part0,
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
    const Grad& e = tab.e[at];
    const bool gb = e.types & 2;
    const int64_t i0 = (int64_t)(chunk - e.first) * kNormChunk;
    const int n = (int)min((int64_t)kNormChunk, e.n - i0);
    const char* g = static_cast<const char*>(e.g) + i0 * (gb ? 2 : 4);
    sum += gb ? squares<true>(g, n) : squares<false>(g, n);
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
// Lengths of tables: kernel arguments hold 32764 bytes, and every launch copies its own, so a short list takes a short
// one.
constexpr int kMany = 376, kSome = 176, kFew = 48;      // 80 bytes a tensor
constexpr int kGradMany = 1200, kGradFew = 176;         // 24 bytes
static_assert(sizeof(Table<Entry, kMany>) + sizeof(AdamWArgs) <= 32764 && sizeof(Table<Grad, kGradMany>) + 64 <= 32764,
              "kernel arguments");
constexpr int kNormBlocks = 2048;  // at most, whatever the device

void set(Entry& e, const moe_adamw_tensor& s, uint32_t first, uint32_t types) {
  e = {s.param, s.grad, s.master, s.m, s.v, s.m_scale, s.v_scale, s.n, first, types, s.lr_scale, s.weight_decay};
}
void set(Grad& e, const moe_adamw_tensor& s, uint32_t first, uint32_t types) { e = {s.grad, s.n, first, types}; }

// Fills a table with the list's first tensors, as many as fit; returns how many of the list it took.
template <typename E, int N>
int64_t fill(Table<E, N>* t, const moe_adamw_tensor* list, int64_t count, int64_t chunk) {
  t->count = 0;
  uint64_t chunks = 0;
  int64_t i = 0;
  for (; i < count && t->count < N; ++i) {
    const moe_adamw_tensor& s = list[i];
    if (s.n == 0) continue;
    const uint64_t c = (uint64_t)((s.n + chunk - 1) / chunk);
    if (chunks + c >= (1ull << 31)) break;  // the rest in another launch
    set(t->e[t->count++], s, (uint32_t)chunks, (uint32_t)(s.dtype == MOE_BF16) | (uint32_t)(s.grad_dtype == MOE_BF16) << 1);
    chunks += c;
  }
  t->chunks = (uint32_t)chunks;
  if (chunks <= kMap)
    for (uint32_t j = 0; j < t->count; ++j)
      for (uint32_t c = t->e[j].first, end = j + 1 < t->count ? t->e[j + 1].first : t->chunks; c < end; ++c) t->map[c] = (uint16_t)j;
  return i;
}

// As many blocks as are resident at once, for kernels whose blocks walk many chunks: one more round of blocks would
// double their time.
template <typename K>
int grid_of(K kernel, std::atomic<int>& per, uint32_t chunks, int sms) {
  int n = per.load(std::memory_order_relaxed);  // asked once: every GPU that runs this code has the same SMs
  if (n < 1) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, 0) != cudaSuccess || n < 1) n = 1;
    per.store(n, std::memory_order_relaxed);
  }
  return (int)std::min<int64_t>(chunks, (int64_t)sms * n);
}

template <int N>
cudaError_t adamw_launches(int bits, const AdamWArgs& a, const moe_adamw_tensor* list, int64_t count, int sms,
                           cudaStream_t st, int* launches) {
  static std::atomic<int> resident{0};
  Table<Entry, N> t;
  while (count > 0) {
    const int64_t took = fill(&t, list, count, bits == 8 ? chunk_of<8> : chunk_of<32>);
    list += took;
    count -= took;
    if (!t.count) continue;
    *launches += 1;
    if (bits == 8) MOE_LAUNCH((k_adamw<8, N>), grid_of(k_adamw<8, N>, resident, t.chunks, sms), kThreads, 0, st, t, a);
    else MOE_LAUNCH((k_adamw<32, N>), t.chunks, kThreads, 0, st, t, a);
  }
  return cudaSuccess;
}

template <int N>
cudaError_t norm_launches(char* ws, const moe_adamw_tensor* list, int64_t count, float scale, float* norm, int sms,
                          cudaStream_t st, int* launches) {
  static std::atomic<int> resident{0};
  Table<Grad, N> t;
  float* part = reinterpret_cast<float*>(ws + kNormHeader);
  unsigned* done = reinterpret_cast<unsigned*>(ws + 64);
  int part0 = 0;
  do {
    const int64_t took = fill(&t, list, count, kNormChunk);
    list += took;
    count -= took;
    while (count > 0 && list->n == 0) ++list, --count;  // the launch with the last values is the one that finishes
    const int grid = std::max(1, std::min(kNormBlocks, grid_of(k_grad_norm<N>, resident, t.chunks, sms)));  // no value at all: one block writes a norm of zero
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
  const uint64_t launches = (uint64_t)(count + kGradFew - 1) / kGradFew + (chunks >> 30) + 1;
  return kNormHeader + (size_t)((launches * kNormBlocks * 4 + 255) / 256 * 256);
}

cudaError_t launch_grad_norm(void* ws, const moe_adamw_tensor* list, int64_t count, float scale, float* norm, int sms,
                             cudaStream_t st, int* launches) {
  return count <= kGradFew ? norm_launches<kGradFew>(static_cast<char*>(ws), list, count, scale, norm, sms, st, launches)
                           : norm_launches<kGradMany>(static_cast<char*>(ws), list, count, scale, norm, sms, st, launches);
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
  return count <= kFew    ? adamw_launches<kFew>(d.state_bits, a, list, count, sms, st, launches)
         : count <= kSome ? adamw_launches<kSome>(d.state_bits, a, list, count, sms, st, launches)
                          : adamw_launches<kMany>(d.state_bits, a, list, count, sms, st, launches);
}

}  // namespace moe
