// C = act(A B^T + bias) + residual on the 128x128 block tile (see fused.h).
#include "fused.h"

namespace gemm_f16 {

hipError_t launch_fused_128x128(const FusedParams &p, hipStream_t s) { return launch_fused_tile<Cfg<128, 128, 2, 2, 16>>(p, s); }

}  // namespace gemm_f16
