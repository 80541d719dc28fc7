// The sum of the parts of a TN product whose segments' rows were split (see
// segments.h).  Bound by the parts' bytes, most of them still in the caches
// that the products left them in.
#include "segments.h"

namespace gemm_f16 {

template <bool F32>
__global__ __launch_bounds__(256) void seg_join_kernel(const SegParams p) {
    using Out = std::conditional_t<F32, float, _Float16>;
    const int64_t count = (int64_t)p.groups * p.n * p.k;
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= count) return;
    // (part_elems is a multiple of 4: whole chunks inside each part)
    const float *src = p.h + i;
    floatx4 sum = {};
    int s = 0;
    for (; s + 4 <= p.splits; s += 4) {
        floatx4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const floatx4 *>(src + (s + q) * p.part_elems);
#pragma unroll
        for (int q = 0; q < 4; ++q) sum += v[q];
    }
    for (; s < p.splits; ++s) sum += *reinterpret_cast<const floatx4 *>(src + s * p.part_elems);
    Out out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = (Out)sum[e];  // fp16: the one rounding of C, to nearest even
    Out *dst = static_cast<Out *>(p.c) + i;
    if (i + 4 <= count && (uintptr_t)p.c % (4 * sizeof(Out)) == 0) {
        __builtin_memcpy(__builtin_assume_aligned(dst, 4 * sizeof(Out)), out, sizeof(out));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < count) dst[e] = out[e];
    }
}

hipError_t launch_seg_join(bool f32, const SegParams &p, hipStream_t s) {
    const int64_t grid = ((int64_t)p.groups * p.n * p.k + 1023) / 1024;
    return f32 ? launch_seg(seg_join_kernel<true>, grid, 256, s, p) : launch_seg(seg_join_kernel<false>, grid, 256, s, p);
}

}  // namespace gemm_f16
