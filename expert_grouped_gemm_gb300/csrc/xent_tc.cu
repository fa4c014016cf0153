// xent_tc.cu -- the cross entropy's launches of the tensor-core products: logits that leave the epilogue as a row's
// statistics, or as its gradient, and the products of that gradient.
#include "linear_tc.cuh"

namespace moe {
namespace {

template <int CTAS, int BN, int EPI>
cudaError_t launch_tile(const XentGemm& g, const XentEpi& x, int sms, cudaStream_t st) {
  TcWork<1, EPI> w;
  if (!fill<CTAS, BN, true, false, 1, EPI>(&w, 0, g)) return cudaErrorInvalidValue;
  w.p[0].x = x;
  const int64_t units = sms / CTAS;
  if (CTAS == 2 && EPI == kEpiGrad) halve(&w.p[0], w.p[0].items, units);  // statistics have one slot for a tile's half
  w.rem = w.extra = 0;
  return launch_work<CTAS, BN, true, false, 1, EPI>(w, std::min<int64_t>(w.p[0].items, units), st);
}

template <int NB, int EPI>
cudaError_t launch_split(const XentGemm& g, const XentEpi& x, int S, cudaStream_t st) {
  switch (S) {
    case 1: return launch_split_as<NB, 1, true, EPI>(g, st, x);
    case 2: return launch_split_as<NB, 2, true, EPI>(g, st, x);
    case 4: return launch_split_as<NB, 4, true, EPI>(g, st, x);
    default: return launch_split_as<NB, 8, true, EPI>(g, st, x);
  }
}

template <int EPI>
cudaError_t launch(const XentGemm& g, const XentEpi& x, int sms, cudaStream_t st, int* width) {
  const LinearChoice c = choose_linear(g.M, g.N, g.K, g.a_mn, sms);
  *width = c.nb || c.S == 2 ? 128 : 64;
  if (c.nb == 16) return launch_split<16, EPI>(g, x, c.S, st);
  if (c.nb == 32) return launch_split<32, EPI>(g, x, c.S, st);
  if (c.nb == 64) return launch_split<64, EPI>(g, x, c.S, st);
  return c.S == 2 ? launch_tile<2, 256, EPI>(g, x, sms, st) : launch_tile<1, 128, EPI>(g, x, sms, st);
}

}  // namespace

cudaError_t launch_xent_stats(const XentGemm& g, const XentEpi& x, int sms, cudaStream_t st, int* width) {
  return launch<kEpiStats>(g, x, sms, st, width);
}

cudaError_t launch_xent_grad(const XentGemm& g, const XentEpi& x, int sms, cudaStream_t st) {
  int width;
  return launch<kEpiGrad>(g, x, sms, st, &width);
}

cudaError_t launch_xent_product(const XentGemm& g, int sms, cudaStream_t st) { return launch_out<kEpiProduct>(g, sms, st); }

cudaError_t launch_xent_parts(const XentGemm& g, int sms, cudaStream_t st) {
  return launch_tile_out<2, 256, kEpiProduct>(g, sms, st);
}

}  // namespace moe
