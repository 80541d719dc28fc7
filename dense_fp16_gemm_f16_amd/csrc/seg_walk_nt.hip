// The walking kernels of the segmented NT product (see segments_walk.h).
#include "segments_walk.h"

namespace gemm_f16 {

hipError_t launch_seg_walk_nt(int tile, bool f32, bool device_stores, int cus, const SegParams &p, hipStream_t s) {
    switch (tile) {
        case kSeg256x256: return launch_seg_walk<kSegNT, Cfg<256, 256, 2, 2, 16>>(p, f32, device_stores, cus, s);
        case kSeg256x128: return launch_seg_walk<kSegNT, Cfg<256, 128, 2, 2, 16>>(p, f32, device_stores, cus, s);
        case kSeg128x256: return launch_seg_walk<kSegNT, Cfg<128, 256, 2, 2, 16>>(p, f32, device_stores, cus, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace gemm_f16
