// block.h -- host launchers of the norm, gate and linear operators.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// Hooks of moe_api.cu for the other translation units of the C ABI.
int internal_fail(int code, const char* msg);
void internal_count_launches(int n);

// ---------------------------------------------------------------- norm.cu
size_t norm_workspace_bytes(const moe_norm_dims& d);
cudaError_t launch_norm_fwd(const moe_norm_dims& d, const void* x, const void* residual, const void* weight,
                            const void* bias, void* y, void* sum, float* mean, float* rstd, int sms, cudaStream_t st,
                            int* launches);
cudaError_t launch_norm_bwd(const moe_norm_dims& d, void* ws, const void* dy, const void* dsum, const void* x,
                            const void* weight, const float* mean, const float* rstd, void* dx, void* dweight,
                            void* dbias, int sms, cudaStream_t st, int* launches);

// ---------------------------------------------------------------- gate.cu
cudaError_t launch_gate_fwd(const moe_gate_dims& d, const void* logits, const float* bias, int* topk_idx, float* topk_w,
                            int* count, int sms, cudaStream_t st, int* launches);
cudaError_t launch_gate_bwd(const moe_gate_dims& d, const void* logits, const int* topk_idx, const float* dw,
                            void* dlogits, int sms, cudaStream_t st, int* launches);

// ---------------------------------------------------------------- linear.cu
constexpr size_t kLinearHeader = 4096;   // status word; counters, zero between calls
constexpr size_t kLinearCounters = 64;   // where they begin
constexpr int kLinearMaxCounters = (int)(kLinearHeader - kLinearCounters) / 4;
size_t linear_workspace_bytes(const moe_linear_dims& d);
cudaError_t launch_linear_fwd(const moe_linear_dims& d, void* ws, const void* x, const void* w, const void* bias,
                              const void* residual, void* y, void* pre, int sms, cudaStream_t st, int* launches);
cudaError_t launch_linear_bwd(const moe_linear_dims& d, void* ws, const void* dy, const void* x, const void* w,
                              const void* pre, const void* dx_add, void* dx, void* dw, void* dbias, int sms,
                              cudaStream_t st, int* launches);

}  // namespace moe
