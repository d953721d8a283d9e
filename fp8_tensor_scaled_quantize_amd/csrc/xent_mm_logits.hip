// The logits' products of the cross entropy: statistics, and the gradient.
#include "xent_mm.h"

namespace fp8mi {

int64_t xent_lse_tile(int64_t M, int64_t N) { return pick16(M, N, 1, false); }

template <class P> static hipError_t launch_logits(const P& p, int tile, hipStream_t st) {
  switch (tile) {
    case 256: return launch_mm16_tile<256, 256, 2, 4, 1, 0, 0>(p, st);
    case 128: return launch_mm16_tile<128, 128, 2, 2, 2, 0, 0>(p, st);
    default: return launch_mm16_tile<64, 64, 1, 4, 2, 0, 0>(p, st);
  }
}
hipError_t launch_xent_lse(const XentLseArgs& p, hipStream_t st) {
  return launch_logits(p, (int)xent_lse_tile(p.M, p.vocab), st);
}
hipError_t launch_xent_grad(const XentGradArgs& p, hipStream_t st) {
  return launch_logits(p, pick16(p.M, p.N, 1, false), st);
}

}  // namespace fp8mi
