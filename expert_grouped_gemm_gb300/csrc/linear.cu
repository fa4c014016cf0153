// linear.cu -- y = act(x w + bias) + residual and its gradients.
//
//   dz = dy act'(pre), dx = dz w^T, dw = x^T dz, dbias = column sums of dz.
#include <algorithm>

#include "act.cuh"
#include "block.h"
#include "common.cuh"
#include "linear_f32.h"
#include "linear_tc.h"

namespace moe {
namespace {

// ---------------------------------------------------------------- fp32 products
// fp32 operands need fp32 products (tf32 keeps 10 bits of a factor), so these run on the CUDA
// cores: a 64 x 64 tile per block of 128 threads, 8 x 4 outputs a thread (three 16-byte shared
// loads for 32 FMAs), k in slabs of 16, the next slab's global loads in registers while this one is
// multiplied. Bound by FMA issue (2000 x 2000 x 2000 357 us, 45 of 80 TFLOP/s: half of the
// instructions are shared loads, packs and copies). As six bf16 products of exact three-way splits on the tensor cores
// they would lose accuracy: those truncate as they accumulate, and products of positive operands over k = 4096 came out
// 1.4e-5 low, where fp32 sums are within 1e-6. Where the tiles alone leave SMs idle, S blocks of a
// cluster share a tile, each with a part of K, and add the parts in rank order. A launch does one product
// or two (dx and dw), each with its own S: a cluster of the larger S holds several tiles of the other.
// Together they fill the SMs that either leaves idle: 300 x 768 x 1000 with dz 41.8 -> 33.9 us, 17 x 256 x 700
// 16.6 -> 10.7, 2000 x 2000 x 2000 740 -> 708.
constexpr int kSB = kF32Tile, kSK = kF32Slab, kSThreads = 128;

// A thread's eight elements of the 64 x 16 slab of an operand X[r, k] (r: the 64 rows of A or columns
// of B): two 16-byte loads along the contiguous index where the rows allow, else eight loads with
// neighbouring threads on the contiguous index.
struct Slab {
  const float* p;      // element of the first load in slab 0
  int64_t dr, dslab;   // from one load to the next, from one slab to the next
  int r, k, rstep, kstep, R, K;
  bool vec, kc;        // 16-byte loads; k is the contiguous index
  float v[8];
  __device__ __forceinline__ void init(const float* X, int64_t sr, int64_t sk, int r0, int R_, int K_, int tid) {
    R = R_;
    K = K_;
    kc = sk == 1;
    vec = (kc ? sr % 4 == 0 && K % 4 == 0 : sk % 4 == 0 && R % 4 == 0);
    if (vec) {
      r = kc ? tid >> 2 : (tid & 15) * 4;
      k = kc ? (tid & 3) * 4 : tid >> 4;
      rstep = kc ? 32 : 0;
      kstep = kc ? 0 : 8;
    } else {
      r = kc ? tid >> 4 : tid & 63;
      k = kc ? tid & 15 : tid >> 6;
      rstep = kc ? 8 : 0;
      kstep = kc ? 0 : 2;
    }
    p = X + (int64_t)(r0 + r) * sr + (int64_t)k * sk;
    dr = rstep * sr + kstep * sk;
    dslab = kSK * sk;
    R -= r0;
  }
  __device__ __forceinline__ void fetch(int s) {
    const float* q = p + s * dslab;
    const int ks = s * kSK + k;
    if (vec) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r + i * rstep < R && ks + i * kstep < K) t = *reinterpret_cast<const float4*>(q + i * dr);
        v[4 * i] = t.x;
        v[4 * i + 1] = t.y;
        v[4 * i + 2] = t.z;
        v[4 * i + 3] = t.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = r + i * rstep < R && ks + i * kstep < K ? q[i * dr] : 0.0f;
    }
  }
  __device__ __forceinline__ void stash(float (*t)[kSB + 4]) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (kc) {
#pragma unroll
          for (int j = 0; j < 4; ++j) t[k + j][r + i * rstep] = v[4 * i + j];
        } else {
          *reinterpret_cast<float4*>(&t[k + i * kstep][r]) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) t[k + i * kstep][r + i * rstep] = v[i];
    }
  }
};

struct SimtWork {
  SimtGemm g[2];
  int S[2];       // parts of a tile
  int tiles[2];
  int blocks0;    // blocks of the first product
  int cluster;    // blocks of a cluster, a multiple of both S
};

// This block's share of a tile's rows, four columns a thread: the parts' sums (rank0: the tile's first block in its
// cluster) and the epilogue.
template <bool XENT>
__device__ __forceinline__ void finish_rows(const SimtGemm& g, float (*sums)[kSB], int m0, int n0, int S, int part, int rank0,
                                            float* out) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const bool vec = (XENT && g.ldo ? g.ldo : g.N) % 4 == 0;
  const int n = n0 + tx * 4;
  for (int r = kSB * part / S + ty; r < kSB * (part + 1) / S; r += kSThreads / 16) {
    const int m = m0 + r;
    if (m >= g.M || n >= g.N) break;
    float z[4] = {0, 0, 0, 0}, y[4];
    for (int p = 0; p < S; ++p) {
      float4 v;
      const uint32_t at = smem_u32(&sums[r][tx * 4]);
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                   : "r"(S > 1 ? mapa_shared(at, rank0 + p) : at));
      z[0] += v.x;
      z[1] += v.y;
      z[2] += v.z;
      z[3] += v.w;
    }
    const int64_t o = (int64_t)m * g.N + n, oy = XENT && g.ldo ? (int64_t)m * g.ldo + n : o;
    if (g.bias)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < g.N) z[j] += g.bias[n + j];
    act_fwd<false, 4>(g.act, z, y);
    if (g.residual)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < g.N) y[j] += g.residual[o + j];
    if (vec && (!XENT || n + 4 <= g.N)) {
      if (g.pre) *reinterpret_cast<float4*>(g.pre + o) = make_float4(z[0], z[1], z[2], z[3]);
      *reinterpret_cast<float4*>(out + oy) = make_float4(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < g.N) {
          if (g.pre) g.pre[o + j] = z[j];
          out[oy + j] = y[j];
        }
    }
  }
}

// XENT: a product of the cross entropy, whose matrices have rows of their own lengths and whose K may have parts
// (SimtGemm); the linear operator's kernel does not look for either.
template <bool XENT>
__global__ void __launch_bounds__(kSThreads, 4) k_linear_f32(const SimtWork work) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  __shared__ __align__(16) float sa[2][kSK][kSB + 4];
  __shared__ __align__(16) float sb[2][kSK][kSB + 4];
  __shared__ __align__(16) float sums[kSB][kSB];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int second = (int)blockIdx.x >= work.blocks0;
  const SimtGemm& g = work.g[second];
  const int S = work.S[second];
  const int block = (int)blockIdx.x - (second ? work.blocks0 : 0);
  const int part = block % S;
  int tile = block / S;
  const int rank0 = (int)(blockIdx.x % work.cluster) - part;  // the tile's first block in the cluster
  if (tile >= work.tiles[second]) {  // fills up the last cluster: nobody reads its sums
    if (work.cluster > 1) {
      cluster_sync_all();
      cluster_sync_all();
    }
    return;
  }
  const int nt = (g.N + kSB - 1) / kSB;
  const int slabs = (g.K + kSK - 1) / kSK;
  int first = part, all = S;  // this block's part of K, of so many
  float* out = g.out;
  if (XENT && g.parts > 1) {
    const int per = (g.M + kSB - 1) / kSB * nt, q = tile / per;
    tile -= q * per;
    first += q * S;
    all *= g.parts;
    out += (int64_t)q * g.M * g.N;
  }
  const int s0 = (int)((int64_t)slabs * first / all), s1 = (int)((int64_t)slabs * (first + 1) / all);
  const int m0 = tile / nt * kSB, n0 = tile % nt * kSB;
  Slab A, B;
  A.init(g.A, g.sam, g.sak, m0, XENT ? g.ma : g.M, XENT ? g.ka : g.K, tid);
  B.init(g.B, g.sbn, g.sbk, n0, XENT ? g.nb : g.N, g.K, tid);
  auto fetch = [&](int s) {
    A.fetch(s);
    B.fetch(s);
  };
  auto stash = [&](int buf) {
    A.stash(sa[buf]);
    B.stash(sb[buf]);
  };
  // two rows of an output column share one packed FMA (fma.rn.f32x2: the same roundings, half the
  // instructions)
  uint64_t acc[4][4] = {};
  fetch(s0);
  stash(0);
  __syncthreads();
  int buf = 0;
  for (int s = s0; s < s1; ++s) {
    if (s + 1 < s1) fetch(s + 1);
#pragma unroll
    for (int k = 0; k < kSK; ++k) {
      const ulonglong2 a0 = *reinterpret_cast<const ulonglong2*>(&sa[buf][k][ty * 8]);
      const ulonglong2 a1 = *reinterpret_cast<const ulonglong2*>(&sa[buf][k][ty * 8 + 4]);
      const float4 b = *reinterpret_cast<const float4*>(&sb[buf][k][tx * 4]);
      const uint64_t av[4] = {a0.x, a0.y, a1.x, a1.y};
      const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint64_t bb;
        asm("mov.b64 %0, {%1, %1};" : "=l"(bb) : "f"(bv[j]));
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[i][j]) : "l"(av[i]), "l"(bb));
      }
    }
    if (s + 1 < s1) stash(buf ^ 1);
    __syncthreads();
    buf ^= 1;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) asm("mov.b64 {%0, %1}, %2;" : "=f"(lo[j]), "=f"(hi[j]) : "l"(acc[i][j]));
    *reinterpret_cast<float4*>(&sums[ty * 8 + 2 * i][tx * 4]) = make_float4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<float4*>(&sums[ty * 8 + 2 * i + 1][tx * 4]) = make_float4(hi[0], hi[1], hi[2], hi[3]);
  }
  if (work.cluster > 1) cluster_sync_all();
  else __syncthreads();
  finish_rows<XENT>(g, sums, m0, n0, S, part, rank0, out);
  if (work.cluster > 1) cluster_sync_all();  // no block leaves while another still reads its sums
}

// ---------------------------------------------------------------- dz and the bias gradient
// dz = dy act'(pre), row stride ldz (stored when dz is given), and the column sums of dz (when
// part is given). Bound by HBM: dy and pre are read once, dz written once (8192 x 4096 bf16 38 us,
// 5.3 TB/s). A block of 64 x 4
// threads owns 64 vectors of VEC columns and a chunk of rows, four rows of it at a time, with
// the loads of four steps in flight; it adds its columns in registers, then over its four
// row lanes in order.
constexpr int kDzCols = 64, kDzRows = 4;
constexpr int kDzSlots = 1216;  // blocks to aim for: 8 for each of 152 SMs

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
  T v[VEC];
};

//
// The last block of a group of `wide` column blocks to finish (a counter in the workspace's header,
// left at zero) adds the chunks' sums into the bias gradient: a few lanes a column, each in chunk
// order, then the lanes, so the result does not depend on which block that was. With db null the
// sums stay in part.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) k_linear_dz(const T* dy, const T* pre, T* dz, float* part, unsigned* done,
                                                   T* db, int M, int N, int64_t ldz, int act, int per, int wide) {
  using V = Vec<T, VEC>;
  pdl_wait();  // the previous kernel has completed and its writes are visible
  __shared__ __align__(16) float red[kDzRows][kDzCols * VEC];
  const int cx = threadIdx.x % kDzCols, ry = threadIdx.x / kDzCols;
  const int n = (blockIdx.x * kDzCols + cx) * VEC;
  const int m1 = min(M, ((int)blockIdx.y + 1) * per);
  float sum[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) sum[i] = 0.0f;
  if (n < N) {
    constexpr int U = 4;  // rows in flight
    for (int m = blockIdx.y * per + ry; m < m1; m += U * kDzRows) {
      V d[U], z[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (m + u * kDzRows < m1) {
          const int64_t o = (int64_t)(m + u * kDzRows) * N + n;
          d[u] = *reinterpret_cast<const V*>(dy + o);
          if (pre) z[u] = *reinterpret_cast<const V*>(pre + o);
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (m + u * kDzRows < m1) {
          float f[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) f[i] = io<T>::to_f(d[u].v[i]);
          if (pre) {
            float zf[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) zf[i] = io<T>::to_f(z[u].v[i]);
            act_grad_mul<sizeof(T) == 2, VEC>(act, zf, f);
          }
          if (dz) {
            V out;
#pragma unroll
            for (int i = 0; i < VEC; ++i) out.v[i] = io<T>::cvt(f[i]);
            *reinterpret_cast<V*>(dz + (int64_t)(m + u * kDzRows) * ldz + n) = out;
          }
#pragma unroll
          for (int i = 0; i < VEC; ++i) sum[i] += f[i];
        }
    }
  }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < VEC; ++i) red[ry][cx * VEC + i] = sum[i];
  __syncthreads();
  for (int c = threadIdx.x; c < kDzCols * VEC; c += blockDim.x) {
    const int col = blockIdx.x * kDzCols * VEC + c;
    if (col >= N) break;
    float s = red[0][c];
#pragma unroll
    for (int r = 1; r < kDzRows; ++r) s += red[r][c];
    part[(int64_t)blockIdx.y * N + col] = s;
  }
  if (!db) return;
  __shared__ bool last;
  const int first = blockIdx.x / wide * wide, blocks = min(wide, (int)gridDim.x - first);
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned* count = done + blockIdx.x / wide;
    last = atomicAdd(count, 1u) == gridDim.y * blocks - 1;
    if (last) *count = 0;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  constexpr int W = VEC >= 4 ? 4 : 1;               // columns a thread adds, in one load
  constexpr int TC = kDzCols * VEC / W;             // threads across a block's columns
  constexpr int LANES = 256 / TC;
  using F = Vec<float, W>;
  F* lanes = reinterpret_cast<F*>(&red[0][0]);      // [LANES][TC]
  const int chunks = (int)gridDim.y, tc = threadIdx.x % TC, lr = threadIdx.x / TC;
  for (int blk = first; blk < first + blocks; ++blk) {
    const int col = blk * kDzCols * VEC + tc * W;
    F s = {};
    if (col < N) {
#pragma unroll 16
      for (int c = lr; c < chunks; c += LANES) {
        F v;
        if constexpr (W == 4) {
          const float4 u = __ldcg(reinterpret_cast<const float4*>(part + (int64_t)c * N + col));
          v = {u.x, u.y, u.z, u.w};
        } else {
          v = {__ldcg(part + (int64_t)c * N + col)};
        }
#pragma unroll
        for (int i = 0; i < W; ++i) s.v[i] += v.v[i];
      }
    }
    __syncthreads();
    lanes[lr * TC + tc] = s;
    __syncthreads();
    if (lr == 0 && col < N) {
#pragma unroll
      for (int r = 1; r < LANES; ++r)
#pragma unroll
        for (int i = 0; i < W; ++i) s.v[i] += lanes[r * TC + tc].v[i];
#pragma unroll
      for (int i = 0; i < W; ++i) db[col + i] = io<T>::cvt(s.v[i]);
    }
  }
}

// The chunks' column sums added: 32 chunk lanes a column, each in chunk order, then the lanes in order.
template <typename T>
__global__ void __launch_bounds__(1024) k_linear_dbias(const float* part, int chunks, int N, T* db) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  __shared__ float red[32][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int n = blockIdx.x * 32 + cx;
  float s = 0.0f;
  if (n < N) {
#pragma unroll 5
    for (int c = ry; c < chunks; c += 32) s += part[(int64_t)c * N + n];
  }
  red[ry][cx] = s;
  __syncthreads();
  if (ry == 0 && n < N) {
#pragma unroll
    for (int r = 1; r < 32; ++r) s += red[r][cx];
    db[n] = io<T>::cvt(s);
  }
}

// Row chunks of the column sums: enough blocks for two rounds on every SM, at least 16 rows each.
int dz_chunks(int64_t M, int64_t N, int vec) {
  const int64_t cb = (N + kDzCols * vec - 1) / (kDzCols * vec);
  const int64_t want = std::max<int64_t>(1, (int64_t)kDzSlots / cb);
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, (M + 15) / 16));
}

// Matrices with odd rows copied to rows of a multiple of 16 bytes, for the tensor-core products
// (TMA reads rows at 16-byte strides). The columns past C of dst are never read. Up to two matrices
// a launch: blocks [0, split) take the first.
//
// A thread stores 16 bytes of a row and loads the two aligned pieces of 16 that they lie in (one of
// them its neighbour's, from L1): bound by HBM, 4096 x 50257 in 139 us, 5.9 TB/s (value by value 247).
struct PackArgs {
  const __nv_bfloat16* src[2];  // 16-byte aligned, as dst
  __nv_bfloat16* dst[2];
  int64_t n[2], ld[2];  // elements, row stride of dst (a multiple of 8)
  int C[2];
  int split;
};

// U: stores of a thread's step, their loads in flight together.
template <int U>
__global__ void __launch_bounds__(256, 4) k_pack_rows(const __grid_constant__ PackArgs a) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const int w = (int)blockIdx.x >= a.split;
  const int b = (int)blockIdx.x - (w ? a.split : 0), blocks = w ? (int)gridDim.x - a.split : a.split;
  const __nv_bfloat16* src = a.src[w];
  __nv_bfloat16* dst = a.dst[w];
  const int64_t n = a.n[w], ld = a.ld[w];
  const int C = a.C[w], row = (C + 7) / 8;  // stores of a row
  const int64_t stores = n / C * row;
  for (int64_t base = (int64_t)b * (256 * U) + threadIdx.x; base < stores; base += (int64_t)blocks * (256 * U)) {
    int64_t r = base / row, from[U], to[U];
    int c = (int)(base - r * row);
    ulonglong2 lo[U], hi[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = base + u * 256 < stores;
      from[u] = in ? r * C + c * 8 : n;
      to[u] = r * ld + c * 8;
      const int64_t f = from[u] & ~7ll;
      if (f + 16 <= n) {
        const ulonglong2* p = reinterpret_cast<const ulonglong2*>(src + f);
        lo[u] = p[0];
        hi[u] = p[1];
      }
      c += 256;
      if (row >= 256) {
        if (c >= row) {
          c -= row;
          ++r;
        }
      } else {
        r += c / row;
        c %= row;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t f = from[u] & ~7ll;
      if (f + 16 <= n) {
        const bool far = from[u] & 4;
        const int bits = (int)(from[u] & 3) * 16;
        const uint64_t x = far ? lo[u].y : lo[u].x, y = far ? hi[u].x : lo[u].y, z = far ? hi[u].y : hi[u].x;
        const auto joined = [&](uint64_t l, uint64_t h) { return l >> bits | h << 1 << (63 - bits); };
        *reinterpret_cast<ulonglong2*>(dst + to[u]) = make_ulonglong2(joined(x, y), joined(y, z));
      } else {  // where the matrix ends
        for (int i = 0; i < 8 && from[u] + i < n; ++i) dst[to[u] + i] = src[from[u] + i];
      }
    }
  }
}

}  // namespace

// One product or two (count) in one launch.
cudaError_t launch_linear_f32(const SimtGemm* g, int count, bool xent, int sms, cudaStream_t st, int* launches) {
  SimtWork w;
  int64_t tiles[2] = {0, 0};
  int slabs[2] = {0, 0};
  for (int i = 0; i < 2; ++i) {
    w.g[i] = g[i < count ? i : 0];
    if (!w.g[i].ma) w.g[i].ma = w.g[i].M;
    if (!w.g[i].nb) w.g[i].nb = w.g[i].N;
    if (!w.g[i].ka) w.g[i].ka = w.g[i].K;
    w.S[i] = 1;
    if (i >= count) continue;
    tiles[i] = (((int64_t)g[i].M + kSB - 1) / kSB) * ((g[i].N + kSB - 1) / kSB);
    slabs[i] = (g[i].K + kSK - 1) / kSK / g[i].parts;  // of a part, if K has parts
    tiles[i] *= g[i].parts;
  }
  // four blocks fit an SM; the product with the longer parts is split while its blocks still fit beside
  // the other's, or (xent) while a part of it would outlast the GPU's even share of all slabs; a part keeps at least
  // four slabs
  const int64_t slots = (int64_t)sms * 4, share = (tiles[0] * slabs[0] + tiles[1] * slabs[1]) / slots;
  while (true) {
    const int i = count > 1 && (int64_t)slabs[1] * w.S[0] > (int64_t)slabs[0] * w.S[1];
    if (w.S[i] == kF32Cluster || slabs[i] < 8 * w.S[i]) break;
    if (tiles[0] * w.S[0] + tiles[1] * w.S[1] + tiles[i] * w.S[i] > slots && !(xent && slabs[i] / w.S[i] > share)) break;
    w.S[i] *= 2;
  }
  w.cluster = std::max(w.S[0], w.S[1]);
  const auto blocks = [&](int i) { return (tiles[i] * w.S[i] + w.cluster - 1) / w.cluster * w.cluster; };
  if (blocks(0) + blocks(1) >= (1ll << 31)) return cudaErrorInvalidValue;
  for (int i = 0; i < 2; ++i) w.tiles[i] = (int)tiles[i];
  w.blocks0 = (int)blocks(0);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  if (MOE_PDL) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (w.cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = (unsigned)w.cluster;
    at[n].val.clusterDim.y = 1;
    at[n++].val.clusterDim.z = 1;
  }
  cfg.gridDim = dim3((unsigned)(blocks(0) + blocks(1)));
  cfg.blockDim = dim3(kSThreads);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = n;
  *launches += 1;
  return xent ? cudaLaunchKernelEx(&cfg, k_linear_f32<true>, w) : cudaLaunchKernelEx(&cfg, k_linear_f32<false>, w);
}

namespace {

int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace: header, column sums, dz, and copies of x and w with rows of a multiple of 16 bytes
// where the caller's are not.
struct LinearWs {
  size_t part, dz, xp, wp, total;
};
LinearWs layout(const moe_linear_dims& d) {
  const bool bf = d.dtype == MOE_BF16;
  const size_t es = bf ? 2 : 4;
  LinearWs L;
  size_t o = kLinearHeader;
  L.part = o;
  o += up256((size_t)dz_chunks(d.M, d.N, d.N % (16 / (int64_t)es) ? 1 : 16 / (int)es) * d.N * sizeof(float));
  L.dz = o;
  o += up256((size_t)d.M * (bf ? up8(d.N) : d.N) * es);
  L.xp = o;
  if (bf && d.K % 8) o += up256((size_t)d.M * up8(d.K) * es);
  L.wp = o;
  if (bf && d.N % 8) o += up256((size_t)d.K * up8(d.N) * es);
  L.total = o;
  return L;
}

// Each matrix given (p, R rows of C) is replaced by a packed copy where its rows are no multiple of
// 16 bytes; one launch for both.
struct Packed {
  PackArgs a = {};
  int count = 0;
  void add(const void** p, void* copy, int64_t R, int64_t C) {
    if (C % 8) add(p, copy, R, C, up8(C));
  }
  void add(const void** p, void* copy, int64_t R, int64_t C, int64_t ld) {
    a.src[count] = static_cast<const __nv_bfloat16*>(*p);
    a.dst[count] = static_cast<__nv_bfloat16*>(copy);
    a.n[count] = R * C;
    a.ld[count] = ld;
    a.C[count++] = (int)C;
    *p = copy;
  }
  cudaError_t run(int sms, cudaStream_t st, int* launches) {
    if (!count) return cudaSuccess;
    const int64_t most = (int64_t)sms * 8;
    int64_t steps[2] = {0, 0};  // of blocks that store 16 bytes a thread
    for (int i = 0; i < count; ++i) steps[i] = (a.n[i] / a.C[i] * ((a.C[i] + 7) / 8) + 255) / 256;
    *launches += 1;
    if (steps[0] <= most && steps[1] <= most) {
      a.split = (int)steps[0];
      MOE_LAUNCH(k_pack_rows<1>, a.split + (int)steps[1], 256, 0, st, a);
    } else {
      a.split = (int)std::min<int64_t>((steps[0] + 1) / 2, most);
      MOE_LAUNCH(k_pack_rows<2>, a.split + (int)std::min<int64_t>((steps[1] + 1) / 2, most), 256, 0, st, a);
    }
    return cudaSuccess;
  }
};

}  // namespace

cudaError_t launch_pack_rows(const void** p, void* copy, int64_t R, int64_t C, int64_t ld, int sms, cudaStream_t st,
                             int* launches) {
  Packed pk;
  if (ld != C) pk.add(p, copy, R, C, ld);
  return pk.run(sms, st, launches);
}

namespace {

template <typename T>
cudaError_t run_dz(const moe_linear_dims& d, char* ws, float* part, const void* dy, const void* pre, void* dz,
                   int64_t ldz, void* db, cudaStream_t st, int* launches) {
  constexpr int V = 16 / sizeof(T);
  const int M = (int)d.M, N = (int)d.N;
  const int vec = N % V ? 1 : V;
  const int cb = (N + kDzCols * vec - 1) / (kDzCols * vec);
  const int want = dz_chunks(M, N, vec), per = (M + want - 1) / want, chunks = (M + per - 1) / per;
  unsigned* done = reinterpret_cast<unsigned*>(ws + kLinearCounters);
  const int wide = (cb + kLinearMaxCounters - 1) / kLinearMaxCounters;
  if (!db) part = nullptr;
  // Few chunks are added by the last block (a launch and 3 us saved at M = 300); many would keep it
  // for longer than a kernel over all columns takes (152 chunks of 4096 columns: 51 us with dz, 43
  // in two kernels).
  void* later = chunks > 32 ? db : nullptr;
  if (later) db = nullptr;
  *launches += 1;
  if (vec == V)
    MOE_LAUNCH((k_linear_dz<T, V>), dim3(cb, chunks), 256, 0, st, (const T*)dy, (const T*)pre, (T*)dz, part, done,
               (T*)db, M, N, ldz, d.act, per, wide);
  else
    MOE_LAUNCH((k_linear_dz<T, 1>), dim3(cb, chunks), 256, 0, st, (const T*)dy, (const T*)pre, (T*)dz, part, done,
               (T*)db, M, N, ldz, d.act, per, wide);
  if (later) {
    *launches += 1;
    MOE_LAUNCH(k_linear_dbias<T>, (N + 31) / 32, 1024, 0, st, (const float*)part, chunks, N, (T*)later);
  }
  return cudaSuccess;
}

cudaError_t fwd_bf16(const moe_linear_dims& d, char* ws, const void* x, const void* w, const void* bias,
                     const void* residual, void* y, void* pre, int sms, cudaStream_t st, int* launches) {
  const LinearWs L = layout(d);
  cudaError_t e;
  Packed pk;
  pk.add(&x, ws + L.xp, d.M, d.K);
  pk.add(&w, ws + L.wp, d.K, d.N);
  if ((e = pk.run(sms, st, launches)) != cudaSuccess) return e;
  LinearGemm g = {(int)d.M, (int)d.N, (int)d.K, x,   w,     up8(d.K),  up8(d.N), 0, 1, bias, residual,
                  y,        pre,      d.act,    d.out_f32, reinterpret_cast<int*>(ws)};
  *launches += 1;
  return launch_linear_tc(g, sms, st);
}

cudaError_t bwd_bf16(const moe_linear_dims& d, char* ws, const void* dy, const void* x, const void* w, const void* pre,
                     const void* dx_add, void* dx, void* dw, void* dbias, int sms, cudaStream_t st, int* launches) {
  const LinearWs L = layout(d);
  const int M = (int)d.M, K = (int)d.K, N = (int)d.N;
  float* part = reinterpret_cast<float*>(ws + L.part);
  int* status = reinterpret_cast<int*>(ws);
  // dz is dy itself without an activation, unless the products need it with wider rows. It is rounded to bf16 because
  // both products read it as a tensor-core operand, which has the type of the other (the error against 64 bits is 0.0023
  // of the gradients' size for 0.0017 of their own rounding alone; two more products of what the rounding drops
  // would double the time). The bias gradient sums the unrounded values.
  const bool store = (dx || dw) && (d.act != MOE_ACT_NONE || N % 8);
  const void* dz = store ? ws + L.dz : dy;
  cudaError_t e = cudaSuccess;
  if (store || dbias)
    e = run_dz<__nv_bfloat16>(d, ws, part, dy, pre, store ? ws + L.dz : nullptr, up8(N), dbias, st, launches);
  if (e == cudaSuccess) {
    Packed pk;
    if (dx) pk.add(&w, ws + L.wp, K, N);
    if (dw) pk.add(&x, ws + L.xp, M, K);
    e = pk.run(sms, st, launches);
  }
  if (e != cudaSuccess || !(dx || dw)) return e;
  const LinearGemm gx = {M, K, N, dz, w, up8(N), up8(N), 0, 0, nullptr, dx_add, dx, nullptr, MOE_ACT_NONE, 0, status};
  const LinearGemm gw = {K, N, M, x, dz, up8(K), up8(N), 1, 1, nullptr, nullptr, dw, nullptr, MOE_ACT_NONE, 0, status};
  if (dx && dw) return launch_linear_tc2(gx, gw, sms, st, launches);
  *launches += 1;
  return launch_linear_tc(dx ? gx : gw, sms, st);
}

const float* f(const void* p) { return static_cast<const float*>(p); }

cudaError_t bwd_f32(const moe_linear_dims& d, char* ws, const void* dy, const void* x, const void* w, const void* pre,
                    const void* dx_add, void* dx, void* dw, void* dbias, int sms, cudaStream_t st, int* launches) {
  const LinearWs L = layout(d);
  const int M = (int)d.M, K = (int)d.K, N = (int)d.N;
  float* part = reinterpret_cast<float*>(ws + L.part);
  const bool store = (dx || dw) && d.act != MOE_ACT_NONE;
  const void* dz = store ? ws + L.dz : dy;
  cudaError_t e = cudaSuccess;
  if (store || dbias) e = run_dz<float>(d, ws, part, dy, pre, store ? ws + L.dz : nullptr, N, dbias, st, launches);
  if (e != cudaSuccess || !(dx || dw)) return e;
  SimtGemm g[2];
  int n = 0;
  if (dx) g[n++] = {f(dz), f(w), N, 1, 1, N, M, N, K, nullptr, f(dx_add), (float*)dx, nullptr, MOE_ACT_NONE};
  if (dw) g[n++] = {f(x), f(dz), 1, K, N, 1, K, M, N, nullptr, nullptr, (float*)dw, nullptr, MOE_ACT_NONE};
  return launch_linear_f32(g, n, false, sms, st, launches);
}

}  // namespace

size_t linear_workspace_bytes(const moe_linear_dims& d) { return layout(d).total; }

cudaError_t launch_linear_fwd(const moe_linear_dims& d, void* ws, const void* x, const void* w, const void* bias,
                              const void* residual, void* y, void* pre, int sms, cudaStream_t st, int* launches) {
  if (d.dtype == MOE_BF16)
    return fwd_bf16(d, static_cast<char*>(ws), x, w, bias, residual, y, pre, sms, st, launches);
  SimtGemm g = {f(x), f(w), d.K, 1, d.N, 1, (int)d.M, (int)d.K, (int)d.N, f(bias), f(residual), (float*)y, (float*)pre,
                d.act};
  return launch_linear_f32(&g, 1, false, sms, st, launches);
}

cudaError_t launch_linear_bwd(const moe_linear_dims& d, void* ws, const void* dy, const void* x, const void* w,
                              const void* pre, const void* dx_add, void* dx, void* dw, void* dbias, int sms,
                              cudaStream_t st, int* launches) {
  return d.dtype == MOE_BF16 ? bwd_bf16(d, static_cast<char*>(ws), dy, x, w, pre, dx_add, dx, dw, dbias, sms, st, launches)
                             : bwd_f32(d, static_cast<char*>(ws), dy, x, w, pre, dx_add, dx, dw, dbias, sms, st, launches);
}

}  // namespace moe
