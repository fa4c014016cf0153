// linear_f32.h -- one description for the fp32 products of the linear operator.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// One product C = op(A) op(B) with element strides, and the epilogue of the forward.
struct SimtGemm {
  const float* A;
  const float* B;
  int64_t sam, sak, sbk, sbn;  // element strides of A[m, k] and B[k, n]
  int M, K, N;
  const float* bias;
  const float* residual;  // [M, N]; may be out
  float* out;
  float* pre;
  int act;
  int64_t ldo = 0;  // row stride of out, 0: N
};

// One product or two (count) in one launch.
cudaError_t launch_linear_f32(const SimtGemm* g, int count, int sms, cudaStream_t st, int* launches);

}  // namespace moe
