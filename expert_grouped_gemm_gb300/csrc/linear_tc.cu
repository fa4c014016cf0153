// linear_tc.cu -- the linear operator's launches of the tensor-core products.
#include "linear_tc.cuh"

namespace moe {
namespace {

// Two products in one launch of CTA pairs, the longer k axis first (Walk).
cudaError_t launch_two(const LinearGemm& g0, const LinearGemm& g1, int sms, cudaStream_t st) {
  const LinearGemm &l = g0.K >= g1.K ? g0 : g1, &s = g0.K >= g1.K ? g1 : g0;
  TcWork<2, kEpiLinear> w;
  if (!fill<2, 256, true, false, 2, kEpiLinear>(&w, 0, l) || !fill<2, 256, true, false, 2, kEpiLinear>(&w, 1, s)) return cudaErrorInvalidValue;
  const int64_t units = sms / 2;
  w.rem = (int)(w.p[0].items % units);
  // a unit without a tile of the last round has time for `fit` tiles of the second product
  const int64_t fit = (2 * (int64_t)w.p[0].kblocks + w.p[1].kblocks) / (2 * (int64_t)w.p[1].kblocks);
  w.extra = w.rem ? (int)std::min<int64_t>((units - w.rem) * fit, w.p[1].items) : 0;
  halve(&w.p[1], w.p[1].items - w.extra, units);
  return launch_work<2, 256, true, false, 2, kEpiLinear>(w, units, st);
}

}  // namespace

cudaError_t launch_linear_tc(const LinearGemm& g, int sms, cudaStream_t st) { return launch_out<kEpiLinear>(g, sms, st); }

cudaError_t launch_linear_tc2(const LinearGemm& g0, const LinearGemm& g1, int sms, cudaStream_t st, int* launches) {
  const LinearChoice c0 = choose_linear(g0.M, g0.N, g0.K, g0.a_mn, sms);
  const LinearChoice c1 = choose_linear(g1.M, g1.N, g1.K, g1.a_mn, sms);
  const auto pair = [](const LinearChoice& c) { return c.nb == 0 && c.S == 2; };
  // k-blocks a unit walks through in both products. Together, in us (dx and dw, separate / in one launch):
  //   44: 2080 x 1096 x 2312 37.4 / 32.4;  54: 2048 x 2048 x 2048 32.9 / 31.1;
  //   88: 1500 x 2880 x 2880 43.2 / 42.3;  108: 1024 x 4096 x 4096 55.9 / 50.6, 4096 x 2048 x 2048 53.4 / 53.5;
  //   216: 8192 x 1024 x 4096 91.8 / 101, 8192 x 2048 x 2048 92.9 / 90.2;  862: 8192 x 4096 x 4096 328 / 341.
  // After the first product's ragged round the units no longer walk k in step, and what one reads is less
  // often in L2 for the others: longer walks lose more by that than a launch costs.
  const auto kblocks = [](const LinearGemm& g) {
    return (double)((g.M + 255) / 256) * ((g.N + 255) / 256) * ((g.K + kBK - 1) / kBK);
  };
  const double walk = (kblocks(g0) + kblocks(g1)) / (sms / 2);
  if (pair(c0) && pair(c1) && g0.N % 8 == 0 && g1.N % 8 == 0 && walk <= 128.0) {
    *launches += 1;
    return launch_two(g0, g1, sms, st);
  }
  *launches += 2;
  const cudaError_t e = launch_linear_tc(g0, sms, st);
  return e != cudaSuccess ? e : launch_linear_tc(g1, sms, st);
}

}  // namespace moe
