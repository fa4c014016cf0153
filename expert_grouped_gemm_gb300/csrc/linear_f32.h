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
  // the cross entropy's alone:
  int64_t ldo = 0;  // row stride of out, 0: N
  // Where rows are longer in memory: how many of A's rows and B's columns may be read (what lies past M and N is not
  // used), and how many k of A (zeros past K). 0: M, N, K. Multiples of 4 are read 16 bytes at a time.
  int ma = 0, nb = 0, ka = 0;
  // K in so many parts, whose sums lie one after the other, [parts][M, N] in out (no epilogue, no ldo), for the caller
  // to add: for a product of few tiles whose K is long for the eight parts that a cluster adds.
  int parts = 1;
};

constexpr int kF32Tile = 64, kF32Slab = 16, kF32Cluster = 8;  // rows and columns of a tile, k of a step, parts of a tile

// One product or two (count) in one launch. xent: ldo, ma, nb, ka and parts are taken, and a product of few tiles and a
// long K is split although the other one fills the GPU.
cudaError_t launch_linear_f32(const SimtGemm* g, int count, bool xent, int sms, cudaStream_t st, int* launches);

}  // namespace moe
