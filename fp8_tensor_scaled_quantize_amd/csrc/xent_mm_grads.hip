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

// Both products in one launch, in tiles of T x T, where neither fills the chip with
// larger ones: the first workgroups take G B, the others G^T A.  64 x 1000 x 512: 6.3 + 4.0
// us and a launch between, together 6.0; 512 x 2000 x 1024, in 128 x 128: 15.3 + 11.9,
// together 14.5.
template <int T, class KM>
__global__ void __launch_bounds__(256, 2) mm16_both(AddArgs a, KM b, int64_t tiles_am, int64_t tiles_an, int64_t wgs_a,
                                                    int64_t tiles_bm, int64_t tiles_bn) {
  constexpr int WM = T == 64 ? 1 : 2, WN = 4 / WM;
  using Lds = TileLds<T, T, 4, 0>;
  __shared__ __align__(16) uint8_t pool[Lds::kBytes];
  int64_t tm, tn;
  if ((int64_t)blockIdx.x < wgs_a) {
    const uint32_t tiles = (uint32_t)(tiles_am * tiles_an);
    tile_coords(blockIdx.x % tiles, tiles_am, tiles_an, 4, tm, tn);
    mm_tile<kOpF16, kOpCodes, T, T, WM, WN, -1, 2, false, 0>(a, tm * T, tn * T, (int64_t)(blockIdx.x / tiles), pool);
  } else {
    const uint32_t tiles = (uint32_t)(tiles_bm * tiles_bn), wg = blockIdx.x - (uint32_t)wgs_a;
    tile_coords(wg % tiles, tiles_bm, tiles_bn, 4, tm, tn);
    mm_tile<kOpF16, kOpF16, T, T, WM, WN, -1, 3, false, 0>(b, tm * T, tn * T, (int64_t)(wg / tiles), pool);
  }
}

template <int T, class KM> static hipError_t launch_both(const AddArgs& a, const KM& b, hipStream_t st) {
  const int64_t am = (a.M + T - 1) / T, an = (a.N + T - 1) / T, bm = (b.M + T - 1) / T, bn = (b.N + T - 1) / T;
  const int64_t wgs_a = am * an * a.batch;
  hipLaunchKernelGGL((mm16_both<T, KM>), dim3((unsigned)(wgs_a + bm * bn * b.batch)), dim3(256), 0, st, a, b, am, an,
                     wgs_a, bm, bn);
  return hipGetLastError();
}

template <class KM> static hipError_t launch_pair(const AddArgs* add, const KM* km, hipStream_t st) {
  if (add && km) {
    const int ta = pick16(add->M, add->N, add->batch, true);
    int tb = pick16(km->M, km->N, 1, true);
    if (KM::kTail) tb = (km->M + 63) / 64 * ((km->N + 63) / 64) < 64 ? 64 : 128;  // as splits_db goes by
    if (ta == 64 && tb == 64) return launch_both<64>(*add, *km, st);
    if (ta <= 128 && tb <= 128) return launch_both<128>(*add, *km, st);
  }
  if (add) {
    const hipError_t e = launch_grads<2>(*add, st);
    if (e != hipSuccess) return e;
  }
  if (!km) return hipSuccess;
  if constexpr (KM::kTail) {  // splits are made where tiles are few
    return launch_mm16_tile<64, 64, 1, 4, 2, 3, 0>(*km, st);
  } else {
    return launch_grads<3>(*km, st);
  }
}

hipError_t launch_mm16_grads(const AddArgs* add, const KmArgs* km, const KmSumArgs* km_sums, hipStream_t st) {
  return km_sums ? launch_pair(add, km_sums, st) : launch_pair(add, km, st);
}

}  // namespace fp8mi
