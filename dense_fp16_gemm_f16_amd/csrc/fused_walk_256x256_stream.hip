// As fused_walk_256x256.hip, with streaming stores.
#include "fused_walk.h"

namespace gemm_f16 {

hipError_t launch_fused_walk_256x256_stream(const FusedParams &p, int cus, hipStream_t s) {
    return launch_walk<Cfg<256, 256, 2, 2, 16>, kStoreStream, true>(p, cus, s);
}

}  // namespace gemm_f16
