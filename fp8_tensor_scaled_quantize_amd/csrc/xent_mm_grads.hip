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
hipError_t launch_mm16_add(const AddArgs& p, hipStream_t st) { return launch_grads<2>(p, st); }
hipError_t launch_mm16_km(const Mm16Args& p, hipStream_t st) { return launch_grads<3>(p, st); }

}  // namespace fp8mi
