// The any-alignment kernel of the segmented products (see segments.h).
#include "segments.h"

namespace gemm_f16 {

hipError_t launch_seg_staged(int kind, bool f32, int mode, SegParams p, hipStream_t s) {
    using C = SegCfg128;
    const int cols = mode == kSegLoraDown ? p.h_ld : p.n;
    p.num_n = (cols + C::BN - 1) / C::BN;
    p.num_m = (p.k + C::BM - 1) / C::BM;
    int64_t grid;
    if (kind == kSegTN) {
        grid = (int64_t)p.groups * p.num_m * p.num_n;
    } else if (mode == kSegLoraUp) {
        grid = (int64_t)((p.rows + C::BM - 1) / C::BM) * p.num_n;
    } else {
        const int64_t m_tiles = seg_row_tiles(p.rows, p.groups, C::BM);
        p.num_m = (int32_t)m_tiles;
        grid = m_tiles * p.num_n;
    }
    if (grid >= (int64_t(1) << 31)) return hipErrorInvalidValue;
    if (mode == kSegLoraDown) return launch_seg(seg_staged_kernel<kSegNT, C, true, kSegLoraDown>, grid, C::kThreads, s, p);
    if (mode == kSegLoraUp) return launch_seg(seg_staged_kernel<kSegNT, C, false, kSegLoraUp>, grid, C::kThreads, s, p);
    switch (kind) {
        case kSegNT:
            return f32 ? launch_seg(seg_staged_kernel<kSegNT, C, true, kSegPlain>, grid, C::kThreads, s, p)
                       : launch_seg(seg_staged_kernel<kSegNT, C, false, kSegPlain>, grid, C::kThreads, s, p);
        case kSegNN:
            return f32 ? launch_seg(seg_staged_kernel<kSegNN, C, true, kSegPlain>, grid, C::kThreads, s, p)
                       : launch_seg(seg_staged_kernel<kSegNN, C, false, kSegPlain>, grid, C::kThreads, s, p);
        default:
            return f32 ? launch_seg(seg_staged_kernel<kSegTN, C, true, kSegPlain>, grid, C::kThreads, s, p)
                       : launch_seg(seg_staged_kernel<kSegTN, C, false, kSegPlain>, grid, C::kThreads, s, p);
    }
}

}  // namespace gemm_f16
