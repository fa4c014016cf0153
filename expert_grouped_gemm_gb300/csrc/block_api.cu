// block_api.cu -- the C ABI of the operators around the experts: argument checks, then the
// launchers of norm.cu, gate.cu, linear.cu, balance.cu, xent.cu and optim.cu. Nothing is enqueued when a check fails.
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

int check_balance(const moe_balance_dims* d) {
  if (!d) return bad(MOE_ERR_INVALID_ARG, "dims is null");
  if (d->T < 1 || d->E < 1 || d->k < 1 || d->S < 0)
    return bad(MOE_ERR_INVALID_ARG, "T, E, k must be >= 1 and S >= 0");
  if (d->T >= (1ll << 31) / 32) return bad(MOE_ERR_UNSUPPORTED, "T >= 2^26");
  if (d->E > 1024) return bad(MOE_ERR_UNSUPPORTED, "E > 1024");
  if (d->k > 32) return bad(MOE_ERR_UNSUPPORTED, "k > 32");
  if (d->S > (1 << 20)) return bad(MOE_ERR_UNSUPPORTED, "S > 2^20");
  if (d->score != MOE_SCORE_SOFTMAX && d->score != MOE_SCORE_SIGMOID)
    return bad(MOE_ERR_INVALID_ARG, "unknown score %d", d->score);
  if (!std::isfinite(d->alpha) || !std::isfinite(d->z_coef))
    return bad(MOE_ERR_INVALID_ARG, "alpha and z_coef must be finite");
  if (d->z_coef != 0.0f && d->score == MOE_SCORE_SIGMOID)
    return bad(MOE_ERR_INVALID_ARG, "the z loss belongs to softmax scores: z_coef must be 0 with sigmoid");
  int rc = check_dtype(d->dtype, "dtype");
  return rc ? rc : check_dtype(d->grad_dtype, "grad_dtype");
}

int check_seq(const moe_balance_dims* d, const int32_t* seq_start) {
  if ((d->S > 0) != (seq_start != nullptr)) return bad(MOE_ERR_INVALID_ARG, "seq_start is given iff S > 0");
  return check_ptr(seq_start, "seq_start", false, 4);
}

int check_xent(const moe_xent_dims* d) {
  if (!d) return bad(MOE_ERR_INVALID_ARG, "dims is null");
  if (d->M < 1 || d->H < 1 || d->V < 1) return bad(MOE_ERR_INVALID_ARG, "M, H, V must be >= 1");
  if (d->M > kMaxRows || d->H >= (1 << 24) || d->V >= (1 << 24))
    return bad(MOE_ERR_UNSUPPORTED, "needs M <= 2^31 - 2^20 and H, V < 2^24");
  if (d->tied != 0 && d->tied != 1) return bad(MOE_ERR_INVALID_ARG, "tied must be 0 or 1");
  if (!std::isfinite(d->z_coef)) return bad(MOE_ERR_INVALID_ARG, "z_coef must be finite");
  return check_dtype(d->dtype, "dtype");
}

// The list of an optimiser call; all: every pointer that a step with this many state bits needs, else the gradients.
int check_tensors(const moe_adamw_tensor* list, int64_t count, bool all, int bits) {
  if (count < 0 || count > (1 << 24)) return bad(MOE_ERR_INVALID_ARG, "count must be in [0, 2^24]");
  if (count && !list) return bad(MOE_ERR_INVALID_ARG, "tensors is null");
  for (int64_t i = 0; i < count; ++i) {
    const moe_adamw_tensor& t = list[i];
    const auto need = [&](const void* p, const char* name, bool required, unsigned align) -> int {
      if (p ? reinterpret_cast<uintptr_t>(p) % align == 0 : !required) return MOE_OK;
      return bad(MOE_ERR_INVALID_ARG, "tensor %lld: %s %s", (long long)i, name, p ? "misaligned" : "is null");
    };
    if (t.n < 0 || t.n > (1ll << 40)) return bad(MOE_ERR_INVALID_ARG, "tensor %lld: n out of range", (long long)i);
    if (t.grad_dtype != MOE_BF16 && t.grad_dtype != MOE_F32)
      return bad(MOE_ERR_INVALID_ARG, "tensor %lld: unknown grad_dtype %d", (long long)i, t.grad_dtype);
    int rc = need(t.grad, "grad", t.n > 0, 16);
    if (rc) return rc;
    if (!all) continue;
    if (t.dtype != MOE_BF16 && t.dtype != MOE_F32)
      return bad(MOE_ERR_INVALID_ARG, "tensor %lld: unknown dtype %d", (long long)i, t.dtype);
    if (!std::isfinite(t.lr_scale) || !std::isfinite(t.weight_decay))
      return bad(MOE_ERR_INVALID_ARG, "tensor %lld: lr_scale and weight_decay must be finite", (long long)i);
    if ((rc = need(t.param, "param", t.n > 0, 16)) || (rc = need(t.master, "master", false, 16)) ||
        (rc = need(t.m, "m", t.n > 0, 16)) || (rc = need(t.v, "v", t.n > 0, 16)) ||
        (rc = need(t.m_scale, "m_scale", bits == 8 && t.n > 0, 4)) ||
        (rc = need(t.v_scale, "v_scale", bits == 8 && t.n > 0, 4)))
      return rc;
    if (t.master && t.dtype != MOE_BF16)
      return bad(MOE_ERR_INVALID_ARG, "tensor %lld: master is for bf16 weights", (long long)i);
    if (bits == 32 && (t.m_scale || t.v_scale))
      return bad(MOE_ERR_INVALID_ARG, "tensor %lld: scales are for states of 8 bits", (long long)i);
  }
  return MOE_OK;
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

int moe_balance_workspace_size(const moe_balance_dims* dims, size_t* bytes) {
  if (int rc = check_balance(dims)) return rc;
  if (!bytes) return bad(MOE_ERR_INVALID_ARG, "bytes is null");
  *bytes = balance_workspace_bytes(*dims);
  return MOE_OK;
}

int moe_balance_fwd(const moe_balance_dims* dims, void* ws, size_t ws_bytes, void* stream, const void* logits,
                    const int32_t* topk_idx, const int32_t* seq_start, float* loss, int32_t* count, float* prob) {
  int rc;
  if ((rc = check_balance(dims)) || (rc = check_workspace(ws, ws_bytes, balance_workspace_bytes(*dims))) ||
      (rc = check_ptr(logits, "logits", true)) || (rc = check_ptr(topk_idx, "topk_idx", true, 4)) ||
      (rc = check_seq(dims, seq_start)) || (rc = check_ptr(loss, "loss", true, 4)) ||
      (rc = check_ptr(count, "count", true, 4)) || (rc = check_ptr(prob, "prob", false, 4)))
    return rc;
  int n = 0;
  const cudaError_t e = launch_balance_fwd(*dims, ws, logits, topk_idx, seq_start, loss, count, prob,
                                           static_cast<cudaStream_t>(stream), &n);
  return finish(e, "moe_balance_fwd", n);
}

int moe_balance_bwd(const moe_balance_dims* dims, void* stream, const void* logits, const int32_t* count,
                    const int32_t* seq_start, const float* dloss, const void* dlogits_add, void* dlogits) {
  int rc;
  if ((rc = check_balance(dims)) || (rc = check_ptr(logits, "logits", true)) ||
      (rc = check_ptr(count, "count", true, 4)) || (rc = check_seq(dims, seq_start)) ||
      (rc = check_ptr(dloss, "dloss", false, 4)) || (rc = check_ptr(dlogits_add, "dlogits_add", false)) ||
      (rc = check_ptr(dlogits, "dlogits", true)))
    return rc;
  int n = 0;
  const cudaError_t e = launch_balance_bwd(*dims, logits, count, seq_start, dloss, dlogits_add, dlogits,
                                           static_cast<cudaStream_t>(stream), &n);
  return finish(e, "moe_balance_bwd", n);
}

int moe_xent_workspace_size(const moe_xent_dims* dims, int backward, size_t* bytes) {
  if (int rc = check_xent(dims)) return rc;
  if (!bytes) return bad(MOE_ERR_INVALID_ARG, "bytes is null");
  *bytes = xent_workspace_bytes(*dims, backward != 0);
  return MOE_OK;
}

int moe_xent_fwd(const moe_xent_dims* dims, void* ws, size_t ws_bytes, void* stream, const void* x, const void* w,
                 const int32_t* target, float* loss, float* lse, float* total) {
  int rc;
  if ((rc = check_xent(dims)) || (rc = check_workspace(ws, ws_bytes, xent_workspace_bytes(*dims, false))) ||
      (rc = check_ptr(x, "x", true)) || (rc = check_ptr(w, "w", true)) ||
      (rc = check_ptr(target, "target", true, 4)) || (rc = check_ptr(loss, "loss", true, 4)) ||
      (rc = check_ptr(lse, "lse", true, 4)) || (rc = check_ptr(total, "total", false, 4)))
    return rc;
  if (loss == lse || (total && (total == loss || total == lse)))
    return bad(MOE_ERR_INVALID_ARG, "loss, lse and total must be different buffers");
  int n = 0;
  const cudaError_t e = launch_xent_fwd(*dims, ws, x, w, target, loss, lse, total, sm_count(),
                                        static_cast<cudaStream_t>(stream), &n);
  return finish(e, "moe_xent_fwd", n);
}

int moe_xent_bwd(const moe_xent_dims* dims, void* ws, size_t ws_bytes, void* stream, const void* x, const void* w,
                 const int32_t* target, const float* lse, const float* dloss, const float* total, void* dx, void* dw) {
  int rc;
  if ((rc = check_xent(dims)) || (rc = check_workspace(ws, ws_bytes, xent_workspace_bytes(*dims, true))) ||
      (rc = check_ptr(x, "x", true)) || (rc = check_ptr(w, "w", true)) ||
      (rc = check_ptr(target, "target", true, 4)) || (rc = check_ptr(lse, "lse", true, 4)) ||
      (rc = check_ptr(dloss, "dloss", false, 4)) || (rc = check_ptr(total, "total", !dloss, 4)) ||
      (rc = check_ptr(dx, "dx", false)) || (rc = check_ptr(dw, "dw", false)))
    return rc;
  if (dloss && total) return bad(MOE_ERR_INVALID_ARG, "give dloss or total, not both");
  if (!dx && !dw) return bad(MOE_ERR_INVALID_ARG, "dx and dw are both null");
  if ((dx && (dx == x || dx == w || dx == dw)) || (dw && (dw == x || dw == w)))
    return bad(MOE_ERR_INVALID_ARG, "dx and dw must be buffers of their own");
  int n = 0;
  const cudaError_t e = launch_xent_bwd(*dims, ws, x, w, target, lse, dloss, total, dx, dw, sm_count(),
                                        static_cast<cudaStream_t>(stream), &n);
  return finish(e, "moe_xent_bwd", n);
}

int moe_grad_norm_workspace_size(const moe_adamw_tensor* tensors, int64_t count, size_t* bytes) {
  if (int rc = check_tensors(tensors, count, false, 32)) return rc;
  if (!bytes) return bad(MOE_ERR_INVALID_ARG, "bytes is null");
  *bytes = grad_norm_workspace_bytes(tensors, count);
  return MOE_OK;
}

int moe_grad_norm(const moe_adamw_tensor* tensors, int64_t count, void* ws, size_t ws_bytes, void* stream,
                  float grad_scale, float* norm) {
  int rc;
  if ((rc = check_tensors(tensors, count, false, 32)) ||
      (rc = check_workspace(ws, ws_bytes, grad_norm_workspace_bytes(tensors, count))) ||
      (rc = check_ptr(norm, "norm", true, 4)))
    return rc;
  if (!std::isfinite(grad_scale)) return bad(MOE_ERR_INVALID_ARG, "grad_scale must be finite");
  int n = 0;
  const cudaError_t e = launch_grad_norm(ws, tensors, count, grad_scale, norm, sm_count(),
                                         static_cast<cudaStream_t>(stream), &n);
  return finish(e, "moe_grad_norm", n);
}

int moe_adamw_step(const moe_adamw_dims* dims, const moe_adamw_tensor* tensors, int64_t count, void* stream,
                   const float* norm, const float* lr, const int32_t* step) {
  if (!dims) return bad(MOE_ERR_INVALID_ARG, "dims is null");
  if (!(dims->beta1 >= 0.0 && dims->beta1 < 1.0 && dims->beta2 >= 0.0 && dims->beta2 < 1.0))
    return bad(MOE_ERR_INVALID_ARG, "beta1 and beta2 must be in [0, 1)");
  if (dims->step < 1) return bad(MOE_ERR_INVALID_ARG, "step must be >= 1");
  if (!std::isfinite(dims->lr) || !std::isfinite(dims->grad_scale) || std::isnan(dims->max_norm))
    return bad(MOE_ERR_INVALID_ARG, "lr and grad_scale must be finite, max_norm no NaN");
  if (!std::isfinite(dims->eps) || dims->eps < 1.17549435e-38f)
    return bad(MOE_ERR_INVALID_ARG, "eps must be finite and at least 2^-126");
  if (dims->state_bits != 32 && dims->state_bits != 8) return bad(MOE_ERR_INVALID_ARG, "state_bits must be 32 or 8");
  int rc;
  if ((rc = check_tensors(tensors, count, true, dims->state_bits)) || (rc = check_ptr(norm, "norm", false, 4)) ||
      (rc = check_ptr(lr, "lr", false, 4)) || (rc = check_ptr(step, "step", false, 4)))
    return rc;
  int n = 0;
  const cudaError_t e = launch_adamw(*dims, tensors, count, norm, lr, step, sm_count(),
                                     static_cast<cudaStream_t>(stream), &n);
  return finish(e, "moe_adamw_step", n);
}

}  // extern "C"
