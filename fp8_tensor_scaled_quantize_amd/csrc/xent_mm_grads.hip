// The products of the logits' gradient with the weights and with the rows.
#include "xent_mm.h"

namespace fp8mi {

template <int LAY, class P> static hipError_t launch_grads(const P& p, hipStream_t st) {
  switch (pick16(p.M, p.N, p.batch, true)) {
    case 256: return launch_mm16_tile<256, 256, 2, 4, 1, LAY, 0>(p, st);
    case 192: return launch_mm16_tile<256, 192, 2, 4, 1, LAY, 0>(p, st);
    case 128: return launch_mm16_tile<128, 128, 2, 2, 2, LAY, 0>(p, st);
    default: return launch_mm16_tile<64, 64, 1, 4, 2, LAY, 0>(p, st);
  }
}

// Both products in one launch, 64 x 64 tiles, where neither fills the chip: the
// first workgroups take G B (the longer sums), the others G^T A (64 x 1000 x 512:
// 6.3 + 4.0 us and a launch between, together 6.0).
__global__ void __launch_bounds__(256, 2) mm16_both(AddArgs a, KmArgs b, int64_t tiles_am, int64_t tiles_an,
                                                    int64_t wgs_a, int64_t tiles_bm, int64_t tiles_bn) {
  using Lds = TileLds<64, 64, 4, 0>;
  __shared__ __align__(16) uint8_t pool[Lds::kBytes];
  int64_t tm, tn;
  if ((int64_t)blockIdx.x < wgs_a) {
    const uint32_t tiles = (uint32_t)(tiles_am * tiles_an);
    tile_coords(blockIdx.x % tiles, tiles_am, tiles_an, 4, tm, tn);
    mm_tile<kOpF16, kOpCodes, 64, 64, 1, 4, -1, 2, false, 0>(a, tm * 64, tn * 64, (int64_t)(blockIdx.x / tiles), pool);
  } else {
    tile_coords((int64_t)blockIdx.x - wgs_a, tiles_bm, tiles_bn, 4, tm, tn);
    mm_tile<kOpF16, kOpF16, 64, 64, 1, 4, -1, 3, false, 0>(b, tm * 64, tn * 64, 0, pool);
  }
}

hipError_t launch_mm16_grads(const AddArgs* add, const KmArgs* km, hipStream_t st) {
  if (add && km && pick16(add->M, add->N, add->batch, true) == 64 && pick16(km->M, km->N, 1, true) == 64) {
    const int64_t am = (add->M + 63) / 64, an = (add->N + 63) / 64, bm = (km->M + 63) / 64, bn = (km->N + 63) / 64;
    hipLaunchKernelGGL(mm16_both, dim3((unsigned)(am * an * add->batch + bm * bn)), dim3(256), 0, st, *add, *km, am, an,
                       am * an * add->batch, bm, bn);
    return hipGetLastError();
  }
  if (add) {
    const hipError_t e = launch_grads<2>(*add, st);
    if (e != hipSuccess) return e;
  }
  return km ? launch_grads<3>(*km, st) : hipSuccess;
}

}  // namespace fp8mi
