// The logits' products of the cross entropy: statistics, and the gradient.
#include "xent_mm.h"

namespace fp8mi {

int64_t xent_lse_tile(int64_t M, int64_t N) { return pick16(M, N, 1, false); }

// 256 x 256 tiles, and 128 x 256 for a last row of tiles that is at most half full
// (they start as CUs come free): 333 x 50001 x 1536 79 -> 66 us; with more rows the
// same (1111 x 50001 x 1536, gradient 184 and 184).
template <class P>
__global__ void __launch_bounds__(512, 1) xent_band(P p, int64_t tiles_m, int64_t tiles_n) {
  using Big = TileLds<256, 256, 8, 0>;
  using Band = TileLds<128, 256, 8, 0>;
  static_assert(Big::kSmem >= Band::kSmem, "the big tile's LDS is the larger");
  __shared__ __align__(16) uint8_t pool[Big::kSmem + P::template extra_bytes<256, 256>()];
  const int64_t big = tiles_m * tiles_n;
  int64_t tm, tn;
  if ((int64_t)blockIdx.x < big) {
    tile_coords(blockIdx.x, tiles_m, tiles_n, 4, tm, tn);
    mm_tile<kOpF16, P::kOpB, 256, 256, 2, 4, -1, 0, false, 0>(p, tm * 256, tn * 256, 0, pool);
  } else {
    mm_tile<kOpF16, P::kOpB, 128, 256, 2, 4, -1, 0, false, 0>(p, tiles_m * 256, ((int64_t)blockIdx.x - big) * 256, 0, pool);
  }
}

template <class P> static hipError_t launch_logits(const P& p0, int tile, hipStream_t st) {
  P p = p0;
  const int64_t rest = p.M % 256, tiles_m = p.M / 256, tiles_n = (p.N + 255) / 256;
  if (tile == 256 && tiles_m > 0 && rest > 0 && rest <= 128) {
    p.early_loads = 1;
    hipLaunchKernelGGL(xent_band<P>, dim3((unsigned)((tiles_m + 1) * tiles_n)), dim3(512), 0, st, p, tiles_m, tiles_n);
    return hipGetLastError();
  }
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
