// Adapters on direct-to-LDS tiles (see segments_direct.h).
#include "segments_direct.h"

namespace gemm_f16 {

hipError_t launch_seg_lora(int tile, const SegParams &p, hipStream_t s) {
    switch (tile) {
        case kSeg256x256: return launch_seg_tile<kSegNT, Cfg<256, 256, 2, 2, 16>, true>(p, false, s);
        case kSeg256x128: return launch_seg_tile<kSegNT, Cfg<256, 128, 2, 2, 16>, true>(p, false, s);
        case kSeg128x256: return launch_seg_tile<kSegNT, Cfg<128, 256, 2, 2, 16>, true>(p, false, s);
        case kSeg128x128: return launch_seg_tile<kSegNT, Cfg<128, 128, 2, 2, 16>, true>(p, false, s);
        case kSeg64x128: return launch_seg_tile<kSegNT, Cfg<64, 128, 2, 2, 16>, true>(p, false, s);
        case kSeg32x128: return launch_seg_tile<kSegNT, Cfg<32, 128, 1, 4, 16>, true>(p, false, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t launch_lora_down(SegParams p, hipStream_t s) {
    // 32 x 64 tiles: with 64 rows a tile, 4096 rows fill a quarter of the CUs
    using C = Cfg<32, 64, 1, 4, 16>;
    constexpr int S = 6, KG = 2;
    p.num_n = (p.h_ld + C::BN - 1) / C::BN;
    p.num_m = (int32_t)seg_row_tiles(p.rows, p.groups, C::BM);
    const int64_t grid = (int64_t)p.num_m * p.num_n;
    return launch_seg(seg_ring_kernel<kSegNT, C, S, KG, true, true>, grid, C::kThreads * KG, s, p);
}

}  // namespace gemm_f16
