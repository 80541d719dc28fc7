// As fused_walk_128x256.hip, with the default policy.
#include "fused_walk.h"

namespace gemm_f16 {

hipError_t launch_fused_walk_128x256_default(const FusedParams &p, int cus, hipStream_t s) {
    return launch_walk<Cfg<128, 256, 2, 2, 16>, kStoreDefault, false>(p, cus, s);
}

}  // namespace gemm_f16
