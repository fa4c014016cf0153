// linear.cu -- y = act(x w + bias) + residual and its gradients.
//
//   dz = dy act'(pre), dx = dz w^T, dw = x^T dz, dbias = column sums of dz.
#include <algorithm>

#include "act.cuh"
#include "block.h"
#include "common.cuh"
#include "linear_tc.h"

namespace moe {
namespace {

// One product C = op(A) op(B) with element strides, and the epilogue of the forward.
struct SimtGemm {
  const void* A;
  const void* B;
  int64_t sam, sak, sbk, sbn;  // element strides of A[m, k] and B[k, n]
  int M, K, N;
  const void* bias;
  const void* residual;
  void* out;
  void* pre;
  int act, out_f32;
};

constexpr int kSBM = 64, kSBN = 64, kSBK = 16;

// 64 x 64 tile per block of 256 threads, 4 x 4 outputs a thread, fp32 FMAs in ascending k.
template <typename T>
__global__ void __launch_bounds__(256) k_linear_simt(const SimtGemm g) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  __shared__ float sa[kSBK][kSBM + 4];
  __shared__ float sb[kSBK][kSBN + 4];
  const T* A = reinterpret_cast<const T*>(g.A);
  const T* B = reinterpret_cast<const T*>(g.B);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int nt = (g.N + kSBN - 1) / kSBN;
  const int m0 = (blockIdx.x / nt) * kSBM, n0 = (blockIdx.x % nt) * kSBN;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < g.K; k0 += kSBK) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = tid + 256 * r;  // neighbouring threads on the contiguous index
      int m, k;
      if (g.sak == 1) {
        k = i & 15;
        m = i >> 4;
      } else {
        m = i & 63;
        k = i >> 6;
      }
      sa[k][m] = m0 + m < g.M && k0 + k < g.K ? io<T>::to_f(A[(int64_t)(m0 + m) * g.sam + (int64_t)(k0 + k) * g.sak]) : 0.0f;
      int n, kb;
      if (g.sbk == 1) {
        kb = i & 15;
        n = i >> 4;
      } else {
        n = i & 63;
        kb = i >> 6;
      }
      sb[kb][n] = n0 + n < g.N && k0 + kb < g.K ? io<T>::to_f(B[(int64_t)(k0 + kb) * g.sbk + (int64_t)(n0 + n) * g.sbn]) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSBK; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = sa[k][ty * 4 + i];
        b[i] = sb[k][tx * 4 + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= g.M || n >= g.N) continue;
      const int64_t o = (int64_t)m * g.N + n;
      const float z = acc[i][j] + (g.bias ? io<T>::to_f(reinterpret_cast<const T*>(g.bias)[n]) : 0.0f);
      const float zz[1] = {z};
      float yy[1];
      act_fwd<sizeof(T) == 2, 1>(g.act, zz, yy);
      float y = yy[0];
      if (g.residual) y += io<T>::to_f(reinterpret_cast<const T*>(g.residual)[o]);
      if (g.pre) reinterpret_cast<T*>(g.pre)[o] = io<T>::cvt(z);
      if (g.out_f32) reinterpret_cast<float*>(g.out)[o] = y;
      else reinterpret_cast<T*>(g.out)[o] = io<T>::cvt(y);
    }
}

// ---------------------------------------------------------------- dz and the bias gradient
// dz = dy act'(pre), row stride ldz (stored when dz is given), and the column sums of dz (when
// part is given). Bound by HBM: dy and pre are read once, dz written once. A block of 64 x 4
// threads owns 64 vectors of VEC columns and a chunk of rows, four rows of it at a time, with
// the loads of eight steps in flight; it adds its columns in registers, then over its four
// row lanes in order.
constexpr int kDzCols = 64, kDzRows = 4;
constexpr int kDzSlots = 1216;  // blocks to aim for: 8 for each of 152 SMs

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[VEC]) {
  struct alignas(sizeof(T) * VEC) A {
    T v[VEC];
  };
  const A a = *reinterpret_cast<const A*>(p);
#pragma unroll
  for (int i = 0; i < VEC; ++i) f[i] = io<T>::to_f(a.v[i]);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[VEC]) {
  struct alignas(sizeof(T) * VEC) A {
    T v[VEC];
  };
  A a;
#pragma unroll
  for (int i = 0; i < VEC; ++i) a.v[i] = io<T>::cvt(f[i]);
  *reinterpret_cast<A*>(p) = a;
}

template <typename T, int VEC>
__global__ void __launch_bounds__(256) k_linear_dz(const T* dy, const T* pre, T* dz, float* part, int M, int N,
                                                   int64_t ldz, int act, int per) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  __shared__ float red[kDzRows][kDzCols * VEC];
  const int cx = threadIdx.x % kDzCols, ry = threadIdx.x / kDzCols;
  const int n = (blockIdx.x * kDzCols + cx) * VEC;
  const int m1 = min(M, ((int)blockIdx.y + 1) * per);
  float sum[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) sum[i] = 0.0f;
  if (n < N) {
    constexpr int U = 4;  // rows in flight
    for (int m = blockIdx.y * per + ry; m < m1; m += U * kDzRows) {
      float d[U][VEC], z[U][VEC];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (m + u * kDzRows < m1) {
          const int64_t o = (int64_t)(m + u * kDzRows) * N + n;
          load_vec<T, VEC>(dy + o, d[u]);
          if (pre) load_vec<T, VEC>(pre + o, z[u]);
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (m + u * kDzRows < m1) {
          if (pre) act_grad_mul<sizeof(T) == 2, VEC>(act, z[u], d[u]);
          if (dz) store_vec<T, VEC>(dz + (int64_t)(m + u * kDzRows) * ldz + n, d[u]);
#pragma unroll
          for (int i = 0; i < VEC; ++i) sum[i] += d[u][i];
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
}

// The chunks' column sums added: eight lanes of chunks per column, then those in order.
template <typename T>
__global__ void __launch_bounds__(256) k_linear_dbias(const float* part, int chunks, int N, T* db) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  __shared__ float red[8][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int n = blockIdx.x * 32 + cx;
  float s = 0.0f;
  if (n < N) {
#pragma unroll 8
    for (int c = ry; c < chunks; c += 8) s += part[(int64_t)c * N + n];
  }
  red[ry][cx] = s;
  __syncthreads();
  if (ry == 0 && n < N) {
#pragma unroll
    for (int r = 1; r < 8; ++r) s += red[r][cx];
    db[n] = io<T>::cvt(s);
  }
}

// Row chunks of the column sums: enough blocks for two rounds on every SM, at least 16 rows each.
int dz_chunks(int64_t M, int64_t N, int vec) {
  const int64_t cb = (N + kDzCols * vec - 1) / (kDzCols * vec);
  const int64_t want = std::max<int64_t>(1, (int64_t)kDzSlots / cb);
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, (M + 15) / 16));
}

// A matrix with odd rows copied to rows of a multiple of 16 bytes, for the tensor-core products
// (TMA reads rows at 16-byte strides). The columns past C of dst are never read.
__global__ void __launch_bounds__(256) k_pack_rows(const __nv_bfloat16* src, __nv_bfloat16* dst, int64_t R, int C,
                                                   int64_t ld) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  constexpr int U = 8;
  const int64_t total = R * C;
  for (int64_t base = (int64_t)blockIdx.x * 256 * U + threadIdx.x; base < total; base += (int64_t)gridDim.x * 256 * U) {
    __nv_bfloat16 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (base + u * 256 < total) v[u] = src[base + u * 256];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = base + u * 256;
      if (i < total) {
        const int64_t r = i / C;
        dst[r * ld + (i - r * C)] = v[u];
      }
    }
  }
}

template <typename T>
cudaError_t run_simt(const SimtGemm& g, cudaStream_t st, int* launches) {
  const int64_t tiles = (((int64_t)g.M + kSBM - 1) / kSBM) * ((g.N + kSBN - 1) / kSBN);
  if (tiles >= (1ll << 31)) return cudaErrorInvalidValue;
  *launches += 1;
  MOE_LAUNCH(k_linear_simt<T>, (unsigned)tiles, 256, 0, st, g);
  return cudaSuccess;
}

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

// p itself when its rows are multiples of 16 bytes, else a packed copy at `copy`
cudaError_t packed(const void** p, void* copy, int64_t R, int64_t C, int sms, cudaStream_t st, int* launches) {
  if (C % 8 == 0) return cudaSuccess;
  const int64_t blocks = (R * C + 2047) / 2048;
  *launches += 1;
  MOE_LAUNCH(k_pack_rows, (unsigned)std::min<int64_t>(blocks, (int64_t)sms * 8), 256, 0, st,
             static_cast<const __nv_bfloat16*>(*p), static_cast<__nv_bfloat16*>(copy), R, (int)C, up8(C));
  *p = copy;
  return cudaSuccess;
}

template <typename T>
cudaError_t run_dz(const moe_linear_dims& d, const void* dy, const void* pre, void* dz, int64_t ldz, float* part,
                   cudaStream_t st, int* launches) {
  constexpr int V = 16 / sizeof(T);
  const int M = (int)d.M, N = (int)d.N;
  const int vec = N % V ? 1 : V;
  const int cb = (N + kDzCols * vec - 1) / (kDzCols * vec);
  const int want = dz_chunks(M, N, vec), per = (M + want - 1) / want, chunks = (M + per - 1) / per;
  *launches += 1;
  if (vec == V)
    MOE_LAUNCH((k_linear_dz<T, V>), dim3(cb, chunks), 256, 0, st, (const T*)dy, (const T*)pre, (T*)dz, part, M, N, ldz,
               d.act, per);
  else
    MOE_LAUNCH((k_linear_dz<T, 1>), dim3(cb, chunks), 256, 0, st, (const T*)dy, (const T*)pre, (T*)dz, part, M, N, ldz,
               d.act, per);
  return cudaSuccess;
}

template <typename T>
cudaError_t run_dbias(const moe_linear_dims& d, const float* part, void* db, cudaStream_t st, int* launches) {
  constexpr int V = 16 / sizeof(T);
  const int M = (int)d.M, N = (int)d.N;
  const int want = dz_chunks(M, N, N % V ? 1 : V), per = (M + want - 1) / want, chunks = (M + per - 1) / per;
  *launches += 1;
  MOE_LAUNCH(k_linear_dbias<T>, (N + 31) / 32, 256, 0, st, part, chunks, N, (T*)db);
  return cudaSuccess;
}

cudaError_t fwd_bf16(const moe_linear_dims& d, char* ws, const void* x, const void* w, const void* bias,
                     const void* residual, void* y, void* pre, int sms, cudaStream_t st, int* launches) {
  const LinearWs L = layout(d);
  cudaError_t e;
  if ((e = packed(&x, ws + L.xp, d.M, d.K, sms, st, launches)) != cudaSuccess) return e;
  if ((e = packed(&w, ws + L.wp, d.K, d.N, sms, st, launches)) != cudaSuccess) return e;
  LinearGemm g = {(int)d.M, (int)d.N, (int)d.K, x,   w,     up8(d.K),  up8(d.N), 0, 1, bias, residual,
                  y,        pre,      d.act,    d.out_f32, reinterpret_cast<int*>(ws)};
  *launches += 1;
  return launch_linear_tc(g, sms, st);
}

cudaError_t bwd_bf16(const moe_linear_dims& d, char* ws, const void* dy, const void* x, const void* w, const void* pre,
                     void* dx, void* dw, void* dbias, int sms, cudaStream_t st, int* launches) {
  const LinearWs L = layout(d);
  const int M = (int)d.M, K = (int)d.K, N = (int)d.N;
  float* part = reinterpret_cast<float*>(ws + L.part);
  int* status = reinterpret_cast<int*>(ws);
  // dz is dy itself without an activation, unless the products need it with wider rows
  const bool store = (dx || dw) && (d.act != MOE_ACT_NONE || N % 8);
  const void* dz = store ? ws + L.dz : dy;
  cudaError_t e = cudaSuccess;
  if (store || dbias)
    e = run_dz<__nv_bfloat16>(d, dy, pre, store ? ws + L.dz : nullptr, up8(N), dbias ? part : nullptr, st, launches);
  if (e == cudaSuccess && dbias) e = run_dbias<__nv_bfloat16>(d, part, dbias, st, launches);
  if (e == cudaSuccess && dx) {
    if ((e = packed(&w, ws + L.wp, K, N, sms, st, launches)) != cudaSuccess) return e;
    LinearGemm g = {M, K, N, dz, w, up8(N), up8(N), 0, 0, nullptr, nullptr, dx, nullptr, MOE_ACT_NONE, 0, status};
    *launches += 1;
    e = launch_linear_tc(g, sms, st);
  }
  if (e == cudaSuccess && dw) {
    if ((e = packed(&x, ws + L.xp, M, K, sms, st, launches)) != cudaSuccess) return e;
    LinearGemm g = {K, N, M, x, dz, up8(K), up8(N), 1, 1, nullptr, nullptr, dw, nullptr, MOE_ACT_NONE, 0, status};
    *launches += 1;
    e = launch_linear_tc(g, sms, st);
  }
  return e;
}

cudaError_t bwd_f32(const moe_linear_dims& d, char* ws, const void* dy, const void* x, const void* w, const void* pre,
                    void* dx, void* dw, void* dbias, cudaStream_t st, int* launches) {
  const LinearWs L = layout(d);
  const int M = (int)d.M, K = (int)d.K, N = (int)d.N;
  float* part = reinterpret_cast<float*>(ws + L.part);
  const bool store = (dx || dw) && d.act != MOE_ACT_NONE;
  const void* dz = store ? ws + L.dz : dy;
  cudaError_t e = cudaSuccess;
  if (store || dbias) e = run_dz<float>(d, dy, pre, store ? ws + L.dz : nullptr, N, dbias ? part : nullptr, st, launches);
  if (e == cudaSuccess && dbias) e = run_dbias<float>(d, part, dbias, st, launches);
  if (e == cudaSuccess && dx) {
    SimtGemm g = {dz, w, N, 1, 1, N, M, N, K, nullptr, nullptr, dx, nullptr, MOE_ACT_NONE, 0};
    e = run_simt<float>(g, st, launches);
  }
  if (e == cudaSuccess && dw) {
    SimtGemm g = {x, dz, 1, K, N, 1, K, M, N, nullptr, nullptr, dw, nullptr, MOE_ACT_NONE, 0};
    e = run_simt<float>(g, st, launches);
  }
  return e;
}

}  // namespace

size_t linear_workspace_bytes(const moe_linear_dims& d) { return layout(d).total; }

cudaError_t launch_linear_fwd(const moe_linear_dims& d, void* ws, const void* x, const void* w, const void* bias,
                              const void* residual, void* y, void* pre, int sms, cudaStream_t st, int* launches) {
  if (d.dtype == MOE_BF16)
    return fwd_bf16(d, static_cast<char*>(ws), x, w, bias, residual, y, pre, sms, st, launches);
  SimtGemm g = {x, w, d.K, 1, d.N, 1, (int)d.M, (int)d.K, (int)d.N, bias, residual, y, pre, d.act, d.out_f32};
  return run_simt<float>(g, st, launches);
}

cudaError_t launch_linear_bwd(const moe_linear_dims& d, void* ws, const void* dy, const void* x, const void* w,
                              const void* pre, void* dx, void* dw, void* dbias, int sms, cudaStream_t st,
                              int* launches) {
  return d.dtype == MOE_BF16 ? bwd_bf16(d, static_cast<char*>(ws), dy, x, w, pre, dx, dw, dbias, sms, st, launches)
                             : bwd_f32(d, static_cast<char*>(ws), dy, x, w, pre, dx, dw, dbias, st, launches);
}

}  // namespace moe
