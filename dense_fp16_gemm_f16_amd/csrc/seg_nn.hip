// C = A B by segment on direct-to-LDS tiles (see segments_direct.h).
#include "segments_direct.h"

namespace gemm_f16 {

hipError_t launch_seg_nn(int tile, bool f32, const SegParams &p, hipStream_t s) {
    switch (tile) {
        case kSeg256x256: return launch_seg_tile<kSegNN, Cfg<256, 256, 2, 2, 16>>(p, f32, s);
        case kSeg256x128: return launch_seg_tile<kSegNN, Cfg<256, 128, 2, 2, 16>>(p, f32, s);
        case kSeg128x256: return launch_seg_tile<kSegNN, Cfg<128, 256, 2, 2, 16>>(p, f32, s);
        case kSeg128x128: return launch_seg_tile<kSegNN, Cfg<128, 128, 2, 2, 16>>(p, f32, s);
        case kSeg64x128: return launch_seg_tile<kSegNN, Cfg<64, 128, 2, 2, 16>>(p, f32, s);
        case kSeg32x128: return launch_seg_tile<kSegNN, Cfg<32, 128, 1, 4, 16>>(p, f32, s);
        case kSegRing: return launch_seg_ring<kSegNN, Cfg<32, 128, 1, 4, 16>, 4, 1>(p, f32, s);
        case kSegRing2: return launch_seg_ring<kSegNN, Cfg<32, 128, 1, 4, 16>, 4, 2>(p, f32, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace gemm_f16
