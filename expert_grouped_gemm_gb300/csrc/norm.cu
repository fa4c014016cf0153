// norm.cu -- layer norm and RMS norm of rows, forward and backward.
//
// h = x + residual, y = (h - mean) rstd w + b. Sums are fp32 throughout; the variance is
// the mean of the squared deviations, taken in a second pass over the row (the one-pass
// form sum(h^2) - mean^2 loses every digit when the mean is large against the spread).
// Both directions are bound by HBM: each tensor is read or written once.
#include "block.h"
#include "common.cuh"

namespace moe {
namespace {

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

// Block per row, three passes over it.
template <typename T>
__global__ void __launch_bounds__(256) k_norm_fwd(const T* x, const T* res, const T* w, const T* b, T* y, T* sum,
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

// dx, block per row.
template <typename T>
__global__ void __launch_bounds__(256) k_norm_dx(const T* dy, const T* dsum, const T* x, const T* w, const float* mean,
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
__global__ void __launch_bounds__(256) k_norm_dw(const T* dy, const T* x, const float* mean, const float* rstd,
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

// The chunks' partial sums added in chunk order.
template <typename T>
__global__ void __launch_bounds__(256) k_norm_dw_sum(const float* part, int chunks, int H, T* dw, T* db) {
  pdl_wait();  // the previous kernel has completed and its writes are visible
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= H) return;
  float aw = 0.0f, ab = 0.0f;
  for (int c = 0; c < chunks; ++c) {
    aw += part[((int64_t)c * 2) * H + i];
    ab += part[((int64_t)c * 2 + 1) * H + i];
  }
  dw[i] = io<T>::cvt(aw);
  if (db) db[i] = io<T>::cvt(ab);
}

template <typename T>
cudaError_t fwd(const moe_norm_dims& d, const void* x, const void* res, const void* w, const void* b, void* y,
                void* sum, float* mean, float* rstd, int sms, cudaStream_t st, int* launches) {
  const int grid = (int)(d.T < (int64_t)sms * 8 ? d.T : (int64_t)sms * 8);
  *launches += 1;
  MOE_LAUNCH(k_norm_fwd<T>, grid, 256, 0, st, (const T*)x, (const T*)res, (const T*)w, (const T*)b, (T*)y, (T*)sum,
             mean, rstd, (int)d.T, (int)d.H, d.kind == MOE_NORM_RMS ? 1 : 0, d.eps);
  return cudaSuccess;
}

template <typename T>
cudaError_t bwd(const moe_norm_dims& d, void* ws, const void* dy, const void* dsum, const void* x, const void* w,
                const float* mean, const float* rstd, void* dx, void* dw, void* db, int sms, cudaStream_t st,
                int* launches) {
  float* part = static_cast<float*>(ws);
  const int rows = (int)d.T, H = (int)d.H;
  const int per = (rows + kNormChunks - 1) / kNormChunks;
  const int chunks = (rows + per - 1) / per;
  const int cb = (H + 255) / 256;
  *launches += 1;  // before dx, which may be written over dy
  MOE_LAUNCH(k_norm_dw<T>, dim3(cb, chunks), 256, 0, st, (const T*)dy, (const T*)x, mean, rstd, part, rows, H, per);
  *launches += 1;
  MOE_LAUNCH(k_norm_dw_sum<T>, cb, 256, 0, st, (const float*)part, chunks, H, (T*)dw, (T*)db);
  *launches += 1;
  const int grid = (int)(d.T < (int64_t)sms * 8 ? d.T : (int64_t)sms * 8);
  MOE_LAUNCH(k_norm_dx<T>, grid, 256, 0, st, (const T*)dy, (const T*)dsum, (const T*)x, (const T*)w, mean, rstd,
             (T*)dx, rows, H);
  return cudaSuccess;
}

}  // namespace

size_t norm_workspace_bytes(const moe_norm_dims& d) { return (size_t)kNormChunks * 2 * d.H * sizeof(float); }

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
