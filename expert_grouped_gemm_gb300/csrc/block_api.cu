// block_api.cu -- the C ABI of the operators around the experts: argument checks, then the
// launchers of norm.cu, gate.cu and linear.cu. Nothing is enqueued when a check fails.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "block.h"

namespace moe {
namespace {

int bad(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return internal_fail(code, buf);
}

int check_ptr(const void* p, const char* name, bool required, unsigned align = 16) {
  if (!p) return required ? bad(MOE_ERR_INVALID_ARG, "%s is null", name) : MOE_OK;
  if (reinterpret_cast<uintptr_t>(p) % align) return bad(MOE_ERR_INVALID_ARG, "%s not %u-byte aligned", name, align);
  return MOE_OK;
}

int check_dtype(int32_t t, const char* name) {
  return t == MOE_BF16 || t == MOE_F32 ? MOE_OK : bad(MOE_ERR_INVALID_ARG, "unknown %s %d", name, t);
}

int check_workspace(void* ws, size_t have, size_t need) {
  if (!ws) return bad(MOE_ERR_WORKSPACE, "workspace is null");
  if (reinterpret_cast<uintptr_t>(ws) & 255) return bad(MOE_ERR_WORKSPACE, "workspace not 256-byte aligned");
  if (have < need) return bad(MOE_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", have, need);
  return MOE_OK;
}

int finish(cudaError_t e, const char* what, int launches) {
  internal_count_launches(launches);
  return e == cudaSuccess ? MOE_OK : bad(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// SMs of the current device (looked up once per device)
int sm_count() {
  constexpr int kMaxDev = 64;
  static std::mutex mu;
  static int cache[kMaxDev];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 148;
  std::lock_guard<std::mutex> lk(mu);
  if (cache[dev]) return cache[dev];
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  return cache[dev] = n;
}

// Row indices are 32-bit and run ahead of the last row by a few grid strides.
constexpr int64_t kMaxRows = (1ll << 31) - (1 << 20);

int check_norm(const moe_norm_dims* d) {
  if (!d) return bad(MOE_ERR_INVALID_ARG, "dims is null");
  if (d->T < 1 || d->H < 1) return bad(MOE_ERR_INVALID_ARG, "T and H must be >= 1");
  if (d->T > kMaxRows) return bad(MOE_ERR_UNSUPPORTED, "T > 2^31 - 2^20");
  if (d->H > 65536) return bad(MOE_ERR_UNSUPPORTED, "H (%lld) > 65536", (long long)d->H);
  if (d->kind != MOE_NORM_LAYER && d->kind != MOE_NORM_RMS)
    return bad(MOE_ERR_INVALID_ARG, "unknown norm kind %d", d->kind);
  if (!std::isfinite(d->eps) || d->eps < 0.0f) return bad(MOE_ERR_INVALID_ARG, "eps must be finite and >= 0");
  return check_dtype(d->dtype, "dtype");
}

int check_gate(const moe_gate_dims* d) {
  if (!d) return bad(MOE_ERR_INVALID_ARG, "dims is null");
  if (d->T < 1 || d->E < 1 || d->k < 1 || d->n_group < 1)
    return bad(MOE_ERR_INVALID_ARG, "T, E, k, n_group must be >= 1");
  if (d->T >= (1ll << 31) / 32) return bad(MOE_ERR_UNSUPPORTED, "T >= 2^26");
  if (d->E > 1024) return bad(MOE_ERR_UNSUPPORTED, "E > 1024");
  if (d->n_group > 32) return bad(MOE_ERR_UNSUPPORTED, "n_group > 32");
  if (d->E % d->n_group) return bad(MOE_ERR_INVALID_ARG, "n_group must divide E");
  if (d->topk_group < 1 || d->topk_group > d->n_group)
    return bad(MOE_ERR_INVALID_ARG, "need 1 <= topk_group <= n_group");
  if (d->k > d->topk_group * (d->E / d->n_group))
    return bad(MOE_ERR_INVALID_ARG, "k (%lld) exceeds the experts of the kept groups", (long long)d->k);
  if (d->k > 32) return bad(MOE_ERR_UNSUPPORTED, "k > 32");
  if (d->group_take != 1 && d->group_take != 2) return bad(MOE_ERR_INVALID_ARG, "group_take must be 1 or 2");
  if (d->score != MOE_SCORE_SOFTMAX && d->score != MOE_SCORE_SIGMOID)
    return bad(MOE_ERR_INVALID_ARG, "unknown score %d", d->score);
  if (!std::isfinite(d->scale)) return bad(MOE_ERR_INVALID_ARG, "scale must be finite");
  int rc = check_dtype(d->dtype, "dtype");
  return rc ? rc : check_dtype(d->grad_dtype, "grad_dtype");
}

int check_linear(const moe_linear_dims* d) {
  if (!d) return bad(MOE_ERR_INVALID_ARG, "dims is null");
  if (d->M < 1 || d->K < 1 || d->N < 1) return bad(MOE_ERR_INVALID_ARG, "M, K, N must be >= 1");
  if (d->M > kMaxRows || d->K >= (1 << 24) || d->N >= (1 << 24))
    return bad(MOE_ERR_UNSUPPORTED, "needs M <= 2^31 - 2^20 and K, N < 2^24");
  if (d->act < MOE_ACT_NONE || d->act > MOE_ACT_SILU) return bad(MOE_ERR_INVALID_ARG, "unknown act %d", d->act);
  if (d->out_f32 != 0 && d->out_f32 != 1) return bad(MOE_ERR_INVALID_ARG, "out_f32 must be 0 or 1");
  return check_dtype(d->dtype, "dtype");
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_norm_workspace_size(const moe_norm_dims* dims, size_t* bytes) {
  if (int rc = check_norm(dims)) return rc;
  if (!bytes) return bad(MOE_ERR_INVALID_ARG, "bytes is null");
  *bytes = norm_workspace_bytes(*dims);
  return MOE_OK;
}

int moe_norm_fwd(const moe_norm_dims* dims, void* stream, const void* x, const void* residual, const void* weight,
                 const void* bias, void* y, void* sum, float* mean, float* rstd) {
  int rc;
  if ((rc = check_norm(dims)) || (rc = check_ptr(x, "x", true)) || (rc = check_ptr(residual, "residual", false)) ||
      (rc = check_ptr(weight, "weight", true)) || (rc = check_ptr(bias, "bias", false)) ||
      (rc = check_ptr(y, "y", true)) || (rc = check_ptr(sum, "sum", false)) ||
      (rc = check_ptr(mean, "mean", false, 4)) || (rc = check_ptr(rstd, "rstd", false, 4)))
    return rc;
  if (sum && !residual) return bad(MOE_ERR_INVALID_ARG, "sum given without residual");
  if (sum == y) return bad(MOE_ERR_INVALID_ARG, "sum and y must be different buffers");
  if (mean && dims->kind == MOE_NORM_RMS) return bad(MOE_ERR_INVALID_ARG, "mean must be null for MOE_NORM_RMS");
  int n = 0;
  const cudaError_t e = launch_norm_fwd(*dims, x, residual, weight, bias, y, sum, mean, rstd, sm_count(),
                                        static_cast<cudaStream_t>(stream), &n);
  return finish(e, "moe_norm_fwd", n);
}

int moe_norm_bwd(const moe_norm_dims* dims, void* ws, size_t ws_bytes, void* stream, const void* dy, const void* dsum,
                 const void* x, const void* weight, const float* mean, const float* rstd, void* dx, void* dweight,
                 void* dbias) {
  int rc;
  if ((rc = check_norm(dims)) || (rc = check_workspace(ws, ws_bytes, norm_workspace_bytes(*dims))) ||
      (rc = check_ptr(dy, "dy", true)) || (rc = check_ptr(dsum, "dsum", false)) || (rc = check_ptr(x, "x", true)) ||
      (rc = check_ptr(weight, "weight", true)) || (rc = check_ptr(mean, "mean", dims->kind == MOE_NORM_LAYER, 4)) ||
      (rc = check_ptr(rstd, "rstd", true, 4)) || (rc = check_ptr(dx, "dx", true)) ||
      (rc = check_ptr(dweight, "dweight", true)) || (rc = check_ptr(dbias, "dbias", false)))
    return rc;
  if (mean && dims->kind == MOE_NORM_RMS) return bad(MOE_ERR_INVALID_ARG, "mean must be null for MOE_NORM_RMS");
  int n = 0;
  const cudaError_t e = launch_norm_bwd(*dims, ws, dy, dsum, x, weight, mean, rstd, dx, dweight, dbias, sm_count(),
                                        static_cast<cudaStream_t>(stream), &n);
  return finish(e, "moe_norm_bwd", n);
}

int moe_gate_fwd(const moe_gate_dims* dims, void* stream, const void* logits, const float* bias, int32_t* topk_idx,
                 float* topk_w, int32_t* expert_count) {
  int rc;
  if ((rc = check_gate(dims)) || (rc = check_ptr(logits, "logits", true)) ||
      (rc = check_ptr(bias, "bias", false, 4)) || (rc = check_ptr(topk_idx, "topk_idx", true, 4)) ||
      (rc = check_ptr(topk_w, "topk_w", true, 4)) || (rc = check_ptr(expert_count, "expert_count", false, 4)))
    return rc;
  int n = 0;
  const cudaError_t e = launch_gate_fwd(*dims, logits, bias, topk_idx, topk_w, expert_count, sm_count(),
                                        static_cast<cudaStream_t>(stream), &n);
  return finish(e, "moe_gate_fwd", n);
}

int moe_gate_bwd(const moe_gate_dims* dims, void* stream, const void* logits, const int32_t* topk_idx,
                 const float* dtopk_w, void* dlogits) {
  int rc;
  if ((rc = check_gate(dims)) || (rc = check_ptr(logits, "logits", true)) ||
      (rc = check_ptr(topk_idx, "topk_idx", true, 4)) || (rc = check_ptr(dtopk_w, "dtopk_w", true, 4)) ||
      (rc = check_ptr(dlogits, "dlogits", true)))
    return rc;
  int n = 0;
  const cudaError_t e = launch_gate_bwd(*dims, logits, topk_idx, dtopk_w, dlogits, sm_count(),
                                        static_cast<cudaStream_t>(stream), &n);
  return finish(e, "moe_gate_bwd", n);
}

int moe_linear_workspace_size(const moe_linear_dims* dims, size_t* bytes) {
  if (int rc = check_linear(dims)) return rc;
  if (!bytes) return bad(MOE_ERR_INVALID_ARG, "bytes is null");
  *bytes = linear_workspace_bytes(*dims);
  return MOE_OK;
}

int moe_linear_fwd(const moe_linear_dims* dims, void* ws, size_t ws_bytes, void* stream, const void* x, const void* w,
                   const void* bias, const void* residual, void* y, void* pre) {
  int rc;
  if ((rc = check_linear(dims)) || (rc = check_workspace(ws, ws_bytes, linear_workspace_bytes(*dims))) ||
      (rc = check_ptr(x, "x", true)) || (rc = check_ptr(w, "w", true)) || (rc = check_ptr(bias, "bias", false)) ||
      (rc = check_ptr(residual, "residual", false)) || (rc = check_ptr(y, "y", true)) ||
      (rc = check_ptr(pre, "pre", false)))
    return rc;
  if (pre == y) return bad(MOE_ERR_INVALID_ARG, "pre and y must be different buffers");
  if (dims->out_f32 && dims->dtype == MOE_BF16 && y == residual)
    return bad(MOE_ERR_INVALID_ARG, "y and residual have different types and cannot share a buffer");
  int n = 0;
  const cudaError_t e = launch_linear_fwd(*dims, ws, x, w, bias, residual, y, pre, sm_count(),
                                          static_cast<cudaStream_t>(stream), &n);
  return finish(e, "moe_linear_fwd", n);
}

int moe_linear_bwd(const moe_linear_dims* dims, void* ws, size_t ws_bytes, void* stream, const void* dy, const void* x,
                   const void* w, const void* pre, const void* dx_add, void* dx, void* dw, void* dbias) {
  int rc;
  if ((rc = check_linear(dims)) || (rc = check_workspace(ws, ws_bytes, linear_workspace_bytes(*dims))) ||
      (rc = check_ptr(dy, "dy", true)) || (rc = check_ptr(x, "x", dw != nullptr)) ||
      (rc = check_ptr(w, "w", dx != nullptr)) || (rc = check_ptr(pre, "pre", dims->act != MOE_ACT_NONE)) ||
      (rc = check_ptr(dx_add, "dx_add", false)) || (rc = check_ptr(dx, "dx", false)) ||
      (rc = check_ptr(dw, "dw", false)) ||
      (rc = check_ptr(dbias, "dbias", false)))
    return rc;
  if (dx_add && !dx) return bad(MOE_ERR_INVALID_ARG, "dx_add given without dx");
  if (dims->act == MOE_ACT_NONE && pre) return bad(MOE_ERR_INVALID_ARG, "pre must be null for MOE_ACT_NONE");
  int n = 0;
  const cudaError_t e = launch_linear_bwd(*dims, ws, dy, x, w, pre, dx_add, dx, dw, dbias, sm_count(),
                                          static_cast<cudaStream_t>(stream), &n);
  return finish(e, "moe_linear_bwd", n);
}

}  // extern "C"
