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

constexpr int kColChunks = 64;  // row chunks of the bias gradient's partial sums

// dz = dy act'(pre) (stored when dz is given) and, when part is given, the column sums of one
// chunk of rows.
template <typename T>
__global__ void __launch_bounds__(256) k_linear_dz(const T* dy, const T* pre, T* dz, float* part, int M, int N, int act,
                                                   int per) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const int n = blockIdx.x * blockDim.x + threadIdx.x;
  if (n >= N) return;
  const int m0 = blockIdx.y * per, m1 = min(M, m0 + per);
  float s = 0.0f;
  for (int m = m0; m < m1; ++m) {
    const int64_t o = (int64_t)m * N + n;
    float v = io<T>::to_f(dy[o]);
    if (pre) {
      const float z[1] = {io<T>::to_f(pre[o])};
      float d[1] = {v};
      act_grad_mul<sizeof(T) == 2, 1>(act, z, d);
      v = d[0];
    }
    if (dz) dz[o] = io<T>::cvt(v);
    s += v;
  }
  if (part) part[(int64_t)blockIdx.y * N + n] = s;
}

template <typename T>
__global__ void __launch_bounds__(256) k_linear_dbias(const float* part, int chunks, int N, T* db) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const int n = blockIdx.x * blockDim.x + threadIdx.x;
  if (n >= N) return;
  float s = 0.0f;
  for (int c = 0; c < chunks; ++c) s += part[(int64_t)c * N + n];
  db[n] = io<T>::cvt(s);
}

template <typename T>
cudaError_t run_simt(const SimtGemm& g, cudaStream_t st, int* launches) {
  const int64_t tiles = (((int64_t)g.M + kSBM - 1) / kSBM) * ((g.N + kSBN - 1) / kSBN);
  if (tiles >= (1ll << 31)) return cudaErrorInvalidValue;
  *launches += 1;
  MOE_LAUNCH(k_linear_simt<T>, (unsigned)tiles, 256, 0, st, g);
  return cudaSuccess;
}

// The tensor-core kernel needs bf16 rows of a multiple of 16 bytes.
bool tc_shape(const moe_linear_dims& d) { return d.dtype == MOE_BF16 && d.K % 8 == 0 && d.N % 8 == 0; }

template <typename T>
cudaError_t fwd(const moe_linear_dims& d, void* ws, const void* x, const void* w, const void* bias,
                const void* residual, void* y, void* pre, int sms, cudaStream_t st, int* launches) {
  if (tc_shape(d)) {
    LinearGemm g = {(int)d.M, (int)d.N, (int)d.K, x, w, d.K, d.N, 0, 1, bias, residual, y, pre, d.act, d.out_f32,
                    static_cast<int*>(ws)};
    *launches += 1;
    return launch_linear_tc(g, sms, st);
  }
  SimtGemm g = {x, w, d.K, 1, d.N, 1, (int)d.M, (int)d.K, (int)d.N, bias, residual, y, pre, d.act, d.out_f32};
  return run_simt<T>(g, st, launches);
}

template <typename T>
cudaError_t bwd(const moe_linear_dims& d, void* ws, const void* dy, const void* x, const void* w, const void* pre,
                void* dx, void* dw, void* dbias, int sms, cudaStream_t st, int* launches) {
  const int M = (int)d.M, K = (int)d.K, N = (int)d.N;
  const bool has_act = d.act != MOE_ACT_NONE;
  float* part = reinterpret_cast<float*>(static_cast<char*>(ws) + kLinearHeader);
  T* dzb = reinterpret_cast<T*>(static_cast<char*>(ws) + kLinearHeader +
                                ((size_t)kColChunks * N * sizeof(float) + 255) / 256 * 256);
  const void* dz = has_act ? dzb : dy;
  if (has_act || dbias) {
    const int per = (M + kColChunks - 1) / kColChunks, chunks = (M + per - 1) / per;
    *launches += 1;
    MOE_LAUNCH(k_linear_dz<T>, dim3((N + 255) / 256, chunks), 256, 0, st, (const T*)dy, (const T*)pre,
               has_act ? dzb : nullptr, dbias ? part : nullptr, M, N, d.act, per);
    if (dbias) {
      *launches += 1;
      MOE_LAUNCH(k_linear_dbias<T>, (N + 255) / 256, 256, 0, st, (const float*)part, chunks, N, (T*)dbias);
    }
  }
  cudaError_t e = cudaSuccess;
  if (tc_shape(d)) {
    int* status = static_cast<int*>(ws);
    if (dx) {
      LinearGemm g = {M, K, N, dz, w, N, N, 0, 0, nullptr, nullptr, dx, nullptr, MOE_ACT_NONE, 0, status};
      *launches += 1;
      if ((e = launch_linear_tc(g, sms, st)) != cudaSuccess) return e;
    }
    if (dw) {
      LinearGemm g = {K, N, M, x, dz, K, N, 1, 1, nullptr, nullptr, dw, nullptr, MOE_ACT_NONE, 0, status};
      *launches += 1;
      e = launch_linear_tc(g, sms, st);
    }
    return e;
  }
  if (dx) {
    SimtGemm g = {dz, w, N, 1, 1, N, M, N, K, nullptr, nullptr, dx, nullptr, MOE_ACT_NONE, 0};
    if ((e = run_simt<T>(g, st, launches)) != cudaSuccess) return e;
  }
  if (dw) {
    SimtGemm g = {x, dz, 1, K, N, 1, K, M, N, nullptr, nullptr, dw, nullptr, MOE_ACT_NONE, 0};
    e = run_simt<T>(g, st, launches);
  }
  return e;
}

}  // namespace

size_t linear_workspace_bytes(const moe_linear_dims& d) {
  const size_t es = d.dtype == MOE_BF16 ? 2 : 4;
  return kLinearHeader + ((size_t)kColChunks * d.N * sizeof(float) + 255) / 256 * 256 +
         ((size_t)d.M * d.N * es + 255) / 256 * 256;
}

cudaError_t launch_linear_fwd(const moe_linear_dims& d, void* ws, const void* x, const void* w, const void* bias,
                              const void* residual, void* y, void* pre, int sms, cudaStream_t st, int* launches) {
  return d.dtype == MOE_BF16 ? fwd<__nv_bfloat16>(d, ws, x, w, bias, residual, y, pre, sms, st, launches)
                             : fwd<float>(d, ws, x, w, bias, residual, y, pre, sms, st, launches);
}

cudaError_t launch_linear_bwd(const moe_linear_dims& d, void* ws, const void* dy, const void* x, const void* w,
                              const void* pre, void* dx, void* dw, void* dbias, int sms, cudaStream_t st,
                              int* launches) {
  return d.dtype == MOE_BF16 ? bwd<__nv_bfloat16>(d, ws, dy, x, w, pre, dx, dw, dbias, sms, st, launches)
                             : bwd<float>(d, ws, dy, x, w, pre, dx, dw, dbias, sms, st, launches);
}

}  // namespace moe
