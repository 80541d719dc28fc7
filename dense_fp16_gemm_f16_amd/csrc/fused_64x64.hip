// C = act(A B^T + bias) + residual on the 64x64 block tile (see fused.h).
#include "fused.h"

namespace gemm_f16 {

hipError_t launch_fused_64x64(const FusedParams &p, hipStream_t s) { return launch_fused_tile<Cfg<64, 64, 2, 2, 16>>(p, s); }

}  // namespace gemm_f16
