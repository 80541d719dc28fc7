// C = act(A B^T + bias) + residual, walking the 256x256 block tiles (see fused_walk.h): device-scope
// stores.
#include "fused_walk.h"

namespace gemm_f16 {

// units of their own
hipError_t launch_fused_walk_256x256_stream(const FusedParams &p, int cus, hipStream_t s);
hipError_t launch_fused_walk_256x256_default(const FusedParams &p, int cus, hipStream_t s);

hipError_t launch_fused_walk_256x256(const FusedParams &p, int cus, hipStream_t s) {
    switch (p.c_store) {
        case kStoreDevice: return launch_walk<Cfg<256, 256, 2, 2, 16>, kStoreDevice, true>(p, cus, s);
        case kStoreStream: return launch_fused_walk_256x256_stream(p, cus, s);
        default: return launch_fused_walk_256x256_default(p, cus, s);
    }
}

}  // namespace gemm_f16
