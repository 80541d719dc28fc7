// C = act(A B^T + bias) + residual, walking the 256x128 block tiles (see fused_walk.h): device-scope
// stores.
#include "fused_walk.h"

namespace gemm_f16 {

// units of their own
hipError_t launch_fused_walk_256x128_stream(const FusedParams &p, int cus, hipStream_t s);
hipError_t launch_fused_walk_256x128_default(const FusedParams &p, int cus, hipStream_t s);

hipError_t launch_fused_walk_256x128(const FusedParams &p, int cus, hipStream_t s) {
    switch (p.c_store) {
        case kStoreDevice: return launch_walk<Cfg<256, 128, 2, 2, 16>, kStoreDevice, false>(p, cus, s);
        case kStoreStream: return launch_fused_walk_256x128_stream(p, cus, s);
        default: return launch_fused_walk_256x128_default(p, cus, s);
    }
}

}  // namespace gemm_f16
