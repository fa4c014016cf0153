// linear_tc.h -- one description for the tensor-core products of the linear operator.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// D[M, N] = A B with A[m, k] at A + m * lda + k (a_mn = 0) or A + k * lda + m (a_mn = 1), and
// B[k, n] at B + n * ldb + k (b_mn = 0) or B + k * ldb + n (b_mn = 1); bf16, lda and ldb multiples
// of 8 elements. The epilogue is the forward's: z = D + bias, y = act(z) + residual.
struct LinearGemm {
  int M, N, K;
  const void* A;
  const void* B;
  int64_t lda, ldb;
  int a_mn, b_mn;
  const void* bias;      // [N] or null
  const void* residual;  // [M, N] or null
  void* y;               // [M, N] bf16, or float with out_f32
  void* pre;             // [M, N] bf16 or null
  int act, out_f32;
  int* status;           // receives MOE_ERR_TIMEOUT when a wait runs out
};

cudaError_t launch_linear_tc(const LinearGemm& g, int sms, cudaStream_t st);
// Two independent products (neither reads what the other writes), in one launch where both are large.
cudaError_t launch_linear_tc2(const LinearGemm& g0, const LinearGemm& g1, int sms, cudaStream_t st, int* launches);

}  // namespace moe
