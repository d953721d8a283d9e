// fp8_mm_act kernels: E4M3 output (mm_act_kernel.h).
#include "mm_act_kernel.h"

namespace fp8mi {

hipError_t launch_mm_act_q8(const MmActArgs& p, hipStream_t st) { return launch_act_family<kE4M3, false>(p, st); }

}  // namespace fp8mi
