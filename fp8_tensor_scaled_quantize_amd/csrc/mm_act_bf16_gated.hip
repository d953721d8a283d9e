// fp8_mm_act kernels: bf16 output, gated activation (mm_act_kernel.h).
#include "mm_act_kernel.h"

namespace fp8mi {

hipError_t launch_mm_act_bf16_gated(const MmActArgs& p, hipStream_t st) { return launch_act_family<-1, true>(p, st); }

}  // namespace fp8mi
