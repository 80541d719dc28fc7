// The any-alignment kernel of the segmented products (see segments.h).
#include "segments.h"

namespace gemm_f16 {

hipError_t launch_seg_staged(int kind, bool f32, bool lora, SegParams p, hipStream_t s) {
    using C = SegCfg128;
    p.num_n = (p.n + C::BN - 1) / C::BN;
    p.num_m = (p.k + C::BM - 1) / C::BM;
    int64_t grid;
    if (kind == kSegTN) {
        grid = (int64_t)p.groups * p.num_m * p.num_n;
    } else if (lora) {
        grid = (int64_t)((p.rows + C::BM - 1) / C::BM) * p.num_n;
    } else {
        const int64_t m_tiles = seg_row_tiles(p.rows, p.groups, C::BM);
        p.num_m = (int32_t)m_tiles;
        grid = m_tiles * p.num_n;
    }
    if (lora) return launch_seg(seg_staged_kernel<kSegNT, C, false, true>, grid, C::kThreads, s, p);
    switch (kind) {
        case kSegNT:
            return f32 ? launch_seg(seg_staged_kernel<kSegNT, C, true, false>, grid, C::kThreads, s, p)
                       : launch_seg(seg_staged_kernel<kSegNT, C, false, false>, grid, C::kThreads, s, p);
        case kSegNN:
            return f32 ? launch_seg(seg_staged_kernel<kSegNN, C, true, false>, grid, C::kThreads, s, p)
                       : launch_seg(seg_staged_kernel<kSegNN, C, false, false>, grid, C::kThreads, s, p);
        default:
            return f32 ? launch_seg(seg_staged_kernel<kSegTN, C, true, false>, grid, C::kThreads, s, p, p.splits)
                       : launch_seg(seg_staged_kernel<kSegTN, C, false, false>, grid, C::kThreads, s, p, p.splits);
    }
}

}  // namespace gemm_f16
