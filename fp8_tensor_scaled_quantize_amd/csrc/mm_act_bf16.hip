// fp8_mm_act kernels: bf16 output (mm_act_kernel.h), and the dispatch.
#include "mm_act_kernel.h"

namespace fp8mi {

hipError_t launch_mm_act_bf16(const MmActArgs& p, hipStream_t st) { return launch_act_family<-1, false>(p, st); }

hipError_t launch_mm_act(const MmActArgs& p, bool gated, hipStream_t st) {
  const bool q8 = p.out_fmt >= 0;
  // no outputs: an fp8 output still completes its scale bookkeeping
  if (p.M == 0 || p.N == 0) return q8 ? launch_mm_q8(p, kE4M3, kE4M3, st) : hipSuccess;
  if (q8 && !p.c_ring && p.c_amax_out) {
    const hipError_t e = launch_zero_word(p.c_amax_out, st);
    if (e != hipSuccess) return e;
  }
  if (q8) return gated ? launch_mm_act_q8_gated(p, st) : launch_mm_act_q8(p, st);
  return gated ? launch_mm_act_bf16_gated(p, st) : launch_mm_act_bf16(p, st);
}

}  // namespace fp8mi
