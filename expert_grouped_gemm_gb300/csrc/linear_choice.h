// linear_choice.h -- which kernel a bf16 product of the linear operator runs on. Host code alone.
#pragma once
#include <stdint.h>

namespace moe {

// Estimated time (us) of each variant, from its rounds over the GPU and its k-blocks per round. The
// constants are a least-squares fit to 114 products (forward, dx and dw for M = 1 .. 8192 and
// weights 256x256 .. 4096x4096 and 1024x8192, every variant timed on each, caches cold); the
// variant with the least estimate is 1.6% slower than the best of all on average; at worst 34%, in the dx of
// 64 x 2048 x 768 (6.3 us on 64 tokens and 8 CTAs, 4.7 on 32 and 4), then 19% (dx of 200 x 512 x 512). Odd N, an
// activation and a kept z cost a tile more than this knows.
// Measured examples (us), pair / single / split with its best cluster:
//   M = 16,   K = 4096, N = 4096:   23.4 / 21.9 / 9.4 (16 tokens, 4 CTAs)
//   M = 512,  K = 512,  N = 512:     7.2 /  6.0 / 4.9 (64 tokens, 4 CTAs)
//   M = 4096, K = 2048, N = 128:    14.9 / 13.5 / 9.3 (64 tokens, 4 CTAs)
//   M = 2048, K = 4096, N = 4096:   46.3 / 78.3 / 92.7
// A k-block costs 0.3 us in a tile (its load's latency over the ring) and 0.26 us in a split part;
// a round of tiles costs its epilogue; a split part costs its share of the tokens, and more where
// two CTAs share an SM.
struct LinearChoice {
  int nb, S;  // nb 0: tiles, of 128 x 128 (S = 1) or 256 x 256 on CTA pairs (S = 2)
};

inline double linear_tile_estimate(int64_t M, int64_t N, int b, int64_t units, int kb, double c0, double ck, double cr) {
  const int64_t t = ((M + b - 1) / b) * ((N + b - 1) / b), last = t % units;
  const double rounds = (double)(t / units) + (last == 0 ? 0.0 : b == 256 && t > units && 2 * last <= units ? 0.5 : 1.0);
  return c0 + rounds * (ck * kb + cr);
}

inline LinearChoice choose_linear(int64_t M, int64_t N, int64_t K, bool a_mn, int sms) {
  const int kb = (int)((K + 63) / 64);  // k-blocks of 64
  LinearChoice best = {0, 1};
  double t = linear_tile_estimate(M, N, 128, sms, kb, 1.56, 0.302, 1.25);
  const double pair = linear_tile_estimate(M, N, 256, sms / 2, kb, 2.23, 0.300, 3.05);
  if (pair < t) {
    t = pair;
    best = {0, 2};
  }
  // an MN-major token matrix is read in chunks of 64 tokens
  for (int nb = a_mn ? 64 : 16; nb <= 64 && (nb < 2 * M || nb == 16 || a_mn); nb *= 2) {
    const int64_t tiles = ((M + nb - 1) / nb) * ((N + 127) / 128);
    for (int S = 1; S <= 8 && S <= kb; S *= 2) {
      const double rounds = (double)((tiles * S + 2 * sms - 1) / (2 * sms));
      const double kbs = (double)((kb + S - 1) / S), shared = tiles * S > sms ? 1.0 : 0.0;
      const double e = 1.82 + (S > 1 ? 1.87 : 0.0) + rounds * (kbs * (0.26 + 0.048 * nb / 64) + 0.034 * nb / S) +
                       shared * (1.81 * rounds + 0.073 * S);
      if (e < t) {
        t = e;
        best = {nb, S};
      }
    }
  }
  return best;
}

}  // namespace moe
