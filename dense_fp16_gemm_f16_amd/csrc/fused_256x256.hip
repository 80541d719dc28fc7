// C = act(A B^T + bias) + residual on the 256x256 block tile (see fused.h).
#include "fused.h"

namespace gemm_f16 {

hipError_t launch_fused_256x256(const FusedParams &p, hipStream_t s) { return launch_fused_tile<Cfg<256, 256, 2, 2, 16>>(p, s); }

}  // namespace gemm_f16
