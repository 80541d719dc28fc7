// C = act(A B^T + bias) + residual, walking the 128x256 block tiles (see fused_walk.h): device-scope
// stores.
#include "fused_walk.h"

namespace gemm_f16 {

hipError_t launch_fused_walk_128x256_stream(const FusedParams &p, int cus, hipStream_t s);  // a unit of its own

hipError_t launch_fused_walk_128x256(bool dev, const FusedParams &p, int cus, hipStream_t s) {
    return dev ? launch_walk<Cfg<128, 256, 2, 2, 16>, kStoreDevice, false>(p, cus, s)
               : launch_fused_walk_128x256_stream(p, cus, s);
}

}  // namespace gemm_f16
