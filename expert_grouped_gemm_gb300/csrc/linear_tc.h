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

// The same for the cross entropy, which asks for more; a type of its own, so that the linear operator's kernels neither
// receive nor test it.
struct XentGemm : LinearGemm {
  int64_t ldy = 0;       // row stride of y, 0: N
  int add = 0;           // with out_f32: added to what y holds
  const float* div = nullptr;  // the product is divided by *div (0: becomes 0)
  int parts = 1;         // with out_f32, launch_xent_parts: K in so many parts, whose sums go to y + part * M * ldy
};

// What the epilogues of the cross entropy read and write beside a product l[M, N] of logits, columns v0 .. v0 + N - 1 of
// a vocabulary of V.
struct XentEpi {
  float2* part;         // statistics: [slots][M]
  float* at;            // statistics: [M], receives the logit of a target among these columns
  const int* target;
  const float* lse;
  const float* dloss;   // null: gradient of the sum of the losses
  const float* own;     // gradient: [M], that of each row's target
  float z;
  int v0, V;
};
// The rows' statistics, one slot for *width columns; nothing else is written.
cudaError_t launch_xent_stats(const XentGemm& g, const XentEpi& x, int sms, cudaStream_t st, int* width);
// y[M, N] (bf16, rows of a multiple of 8) = gradient of the loss to the logits.
cudaError_t launch_xent_grad(const XentGemm& g, const XentEpi& x, int sms, cudaStream_t st);
// A product of that gradient, without bias, residual, pre and activation.
cudaError_t launch_xent_product(const XentGemm& g, int sms, cudaStream_t st);
// One of few tiles and a long K on CTA pairs, K in g.parts parts (out_f32).
cudaError_t launch_xent_parts(const XentGemm& g, int sms, cudaStream_t st);

cudaError_t launch_linear_tc(const LinearGemm& g, int sms, cudaStream_t st);
// Two independent products (neither reads what the other writes), in one launch where both are large.
cudaError_t launch_linear_tc2(const LinearGemm& g0, const LinearGemm& g1, int sms, cudaStream_t st, int* launches);

}  // namespace moe
