// Segmented products of few rows (see segments.h): decoding, and the
// adapters' inner product there.  The time is B's bytes, so what matters is
// how many of them are in flight.
//
// A workgroup owns a segment and 16 columns.  Its waves share K evenly, in
// 32-wide steps, each taking up to kThinSteps at a time; a wave's part of B
// goes straight from memory to registers in the MFMA's layout (lane l: row
// l % 16, 8 elements at 8 (l / 16)), all of it in flight at once, and stays
// there for all of the segment's rows, 16 at a time, if that is all.  No LDS and no barrier
// until the waves' sums meet, in wave order.  Any K, N and alignment: global
// loads take 2-byte aligned addresses, and the part past K is masked.
#include <algorithm>

#include "segments.h"

namespace gemm_f16 {

constexpr int kThinSteps = 8;  // 32-wide steps of K that a wave takes at a time

struct ThinParams {
    SegParams main;       // rows against main.b
    SegParams down;       // kThinLora: the adapters' inner product
    float *sums;          // kThinLora: fp32 [rows, n]
    int32_t down_blocks;  // kThinLora: workgroups of the inner product
};

// `count` steps of a row (K >= 8), 32 elements each, from the one that ends
// a wave's part downwards; 8 elements at kl of each.  The first one, where
// `partial`, reaches past K: its chunks past K become zeros, and the chunk
// across K is loaded from the row's last 8 elements and shifted, so every
// load stays inside the row.
__device__ __forceinline__ void thin_load(half8 (&v)[kThinSteps], const _Float16 *row, int top, int count, bool partial,
                                          int kl, int k_elems) {
    const int k0 = 32 * (top - 1) + kl;
#pragma unroll
    for (int s = 0; s < kThinSteps; ++s) {
        if (s >= count) continue;
        const int k = s == 0 ? min(k0, k_elems - 8) : k0 - 32 * s;
        v[s] = __builtin_bit_cast(half8, (int4v)*reinterpret_cast<const int4u *>(row + k));
    }
    if (partial) {
        const int past = 8 - (k_elems - k0);  // elements to shift out
        unsigned __int128 w = __builtin_bit_cast(unsigned __int128, v[0]);
        if (past > 0) w = past < 8 ? w >> (16 * past) : 0;
        v[0] = __builtin_bit_cast(half8, w);
    }
}

enum ThinMode : int { kThinPlain = 0, kThinLora = 1, kThinDown = 2 };

// MODE kThinPlain: C of a grouped NT product.  kThinLora: h, each row in its
// own place, by the first down_blocks workgroups, and x W^T in fp32, one
// segment of every row, by the others.  kThinDown: h in adapter order, a
// segment's rows shared by gridDim.y workgroups.
template <bool F32, int MODE>
__global__ __launch_bounds__(1024) void seg_thin_kernel(const ThinParams tp) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the signature only
    __shared__ floatx4 red[2][16][kWave];
    const int tid = threadIdx.x, lane = tid % kWave, waves = blockDim.x / kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const bool is_down = MODE == kThinDown || (MODE == kThinLora && (int)blockIdx.x < tp.down_blocks);
    const SegParams &p = MODE == kThinLora && is_down ? tp.down : tp.main;
    const uint32_t pid = MODE == kThinLora && !is_down ? blockIdx.x - tp.down_blocks : blockIdx.x;

    const int g = (int)(pid / (uint32_t)p.num_n), n0 = (int)(pid % (uint32_t)p.num_n) * 16;
    int lo = 0, hi = p.rows;
    bool live = true;  // false: the rows behind the last segment
    if (MODE != kThinLora || is_down) {
        live = g < p.groups;
        lo = seg_bound(p.offsets, g, p.rows);
        hi = live ? seg_bound(p.offsets, g + 1, p.rows) : p.rows;
    }
    const int step = MODE == kThinDown ? 16 * (int)gridDim.y : 16;
    if (MODE == kThinDown) lo += 16 * (int)blockIdx.y;
    if (lo >= hi) return;

    using Out = std::conditional_t<F32, float, _Float16>;
    if (!live) {
        for (int r = lo + tid / 16; r < hi; r += (int)blockDim.x / 16)
            if (n0 + tid % 16 < p.n) static_cast<Out *>(p.c)[(int64_t)r * p.n + n0 + tid % 16] = (Out)0.0f;
        return;
    }
    // Lanes past the segment's rows or B's columns read the last one again:
    // their results are never stored.
    const int kl = 8 * (lane / 16);
    const _Float16 *br = p.b + ((int64_t)g * p.n + min(n0 + lane % 16, p.n - 1)) * p.k;
    // this wave's steps, [part0, part1)
    const int steps = (p.k + 31) / 32;
    const int part0 = (int)((int64_t)steps * wave / waves), part1 = (int)((int64_t)steps * (wave + 1) / waves);
    const bool one_pass = part1 - part0 <= kThinSteps;
    const float f = is_down && p.scale ? p.scale[g] : 1.0f;
    half8 bf[kThinSteps], af[kThinSteps];
    int parity = 0;
    for (int r0 = lo; r0 < hi; r0 += step, parity ^= 1) {
        floatx4 acc = {};
        bool found = true;  // an index outside A: a row of zeros
        const _Float16 *ar = nullptr;
        for (int top = part1; top > part0; top -= kThinSteps) {
            const int count = min(top - part0, kThinSteps);
            const bool partial = 32 * top > p.k;
            if (!one_pass || r0 == lo) thin_load(bf, br, top, count, partial, kl, p.k);
            if (top == part1) {  // behind B's loads
                const int r = min(r0 + lane % 16, hi - 1);
                int64_t src = r;
                if (p.index) {
                    const int v = p.index[r];
                    src = v < 0 ? -1 : v / p.fan;
                }
                found = src >= 0 && src < p.a_rows;
                ar = p.a + (found ? src : 0) * p.k;
            }
            thin_load(af, ar, top, count, partial, kl, p.k);
#pragma unroll
            for (int s = 0; s < kThinSteps; ++s)
                if (s < count) acc = Mfma<16>::run(bf[s], af[s], acc);
        }
        red[parity][wave][lane] = acc;
        lds_barrier();
        // (the waves that go on write the other half of red next)
        if (wave != 0) continue;
        // lane l holds row l % 16, columns 4 (l / 16) ..
        floatx4 sum = red[parity][0][lane];
        for (int w = 1; w < waves; ++w) sum += red[parity][w][lane];
        const int r = r0 + lane % 16, n = n0 + 4 * (lane / 16);
        if (r >= hi) continue;
        if (!found) sum = floatx4{};
        if (is_down) {
            // zeros in the columns past the rank, up to h_ld
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = n + e < p.n ? sum[e] * f : 0.0f;
            const int to = MODE == kThinDown ? r : min(max(p.index[r], 0), p.rows - 1);
            if (n < p.h_ld)
                *reinterpret_cast<floatx4 *>(static_cast<float *>(p.c) + (int64_t)to * p.h_ld + n) = sum;
        } else if (MODE == kThinLora) {
            float *c = tp.sums + (int64_t)r * p.n + n;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < p.n) c[e] = sum[e];
        } else {
            typedef Out out4 __attribute__((ext_vector_type(4)));
            Out *c = static_cast<Out *>(p.c) + (int64_t)r * p.n + n;
            if (n + 3 < p.n && ((uintptr_t)c % sizeof(out4)) == 0) {
                out4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = (Out)sum[e];
                *reinterpret_cast<out4 *>(c) = v;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < p.n) c[e] = (Out)sum[e];
            }
        }
    }
#endif
}

// y = fp16(sums + h U_s^T): one workgroup per row and 256 columns, every
// product and sum in fp32.
__global__ __launch_bounds__(256) void lora_join_kernel(const SegParams p, const float *sums, const int32_t *ids) {
    const int r = blockIdx.y, n = (int)(blockIdx.x * 256 + threadIdx.x);
    if (n >= p.n) return;
    const int s = ids[r];
    float v = sums[(int64_t)r * p.n + n];
    if (s >= 0 && s < p.adapters) {
        const float *h = p.h + (int64_t)r * p.h_ld;
        const _Float16 *u = p.up + ((int64_t)s * p.n + n) * p.rank;
        int j = 0;
        for (; j + 8 <= p.rank; j += 8) {
            const half8 w = __builtin_bit_cast(half8, (int4v)*reinterpret_cast<const int4u *>(u + j));
#pragma unroll
            for (int e = 0; e < 8; ++e) v = __builtin_fmaf(h[j + e], (float)w[e], v);
        }
        for (; j < p.rank; ++j) v = __builtin_fmaf(h[j], (float)u[j], v);
    }
    static_cast<_Float16 *>(p.c)[(int64_t)r * p.n + n] = (_Float16)v;
}

template <class Kernel>
static hipError_t launch_thin(Kernel kernel, int64_t grid, int threads, hipStream_t stream, const ThinParams &p,
                              unsigned grid_y = 1) {
    if (grid <= 0) return hipSuccess;
    if (grid >= (int64_t(1) << 31)) return hipErrorInvalidValue;
    void *args[] = {const_cast<ThinParams *>(&p)};
    return hipLaunchKernel(reinterpret_cast<const void *>(kernel), dim3((unsigned)grid, grid_y), dim3((unsigned)threads),
                           args, 0, stream);
}

// waves that K keeps busy in one pass
static int thin_threads(int k) {
    int w = 1;
    while (w < 16 && w * kThinSteps * 32 < k) w *= 2;
    return w * kWave;
}

hipError_t launch_seg_thin(bool f32, const SegParams &p, hipStream_t s) {
    ThinParams t = {};
    t.main = p;
    t.main.num_n = (p.n + 15) / 16;
    const int64_t grid = (int64_t)(p.groups + 1) * t.main.num_n;
    return f32 ? launch_thin(seg_thin_kernel<true, kThinPlain>, grid, thin_threads(p.k), s, t)
               : launch_thin(seg_thin_kernel<false, kThinPlain>, grid, thin_threads(p.k), s, t);
}

// h of K < 8, where no chunk of a row is whole: one lane per element.
__global__ __launch_bounds__(256) void lora_down_short_kernel(const SegParams p) {
    const int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x, r = x / p.h_ld;
    const int j = (int)(x % p.h_ld);
    if (r >= p.rows) return;
    int g = 0;  // the segment of row r
    while (g < p.groups && r >= seg_bound(p.offsets, g + 1, p.rows)) ++g;
    const int src = p.index[r];
    float sum = 0.0f;
    if (g < p.groups && j < p.n && src >= 0 && src < p.a_rows) {
        for (int k = 0; k < p.k; ++k)
            sum += (float)p.a[(int64_t)src * p.k + k] * (float)p.b[((int64_t)g * p.n + j) * p.k + k];
        if (p.scale) sum *= p.scale[g];
    }
    static_cast<float *>(p.c)[x] = sum;
}

hipError_t launch_lora_down_thin(const SegParams &p, hipStream_t s) {
    if (p.k < 8) {
        const int64_t grid = ((int64_t)p.rows * p.h_ld + 255) / 256;
        if (grid >= (int64_t(1) << 31)) return hipErrorInvalidValue;
        return launch_seg(lora_down_short_kernel, grid, 256, s, p);
    }
    ThinParams t = {};
    t.main = p;
    t.main.num_n = (p.h_ld + 15) / 16;
    // some 64 rows a workgroup of an even split
    const int64_t shares = std::min<int64_t>(std::max<int64_t>(p.rows / (64 * (int64_t)p.groups), 1), 1024);
    return launch_thin(seg_thin_kernel<true, kThinDown>, (int64_t)p.groups * t.main.num_n, thin_threads(p.k), s, t,
                       (unsigned)shares);
}

hipError_t launch_lora_few(const SegParams &p, const SegParams &down, float *sums, const int32_t *ids, hipStream_t s) {
    ThinParams t = {};
    t.main = p;
    t.main.num_n = (p.n + 15) / 16;
    t.down = down;
    t.down.num_n = (down.h_ld + 15) / 16;
    t.sums = sums;
    t.down_blocks = down.groups * t.down.num_n;  // a row without an adapter needs no h
    hipError_t e = launch_thin(seg_thin_kernel<true, kThinLora>, t.down_blocks + (int64_t)t.main.num_n,
                               thin_threads(p.k), s, t);
    if (e != hipSuccess) return e;
    SegParams j = p;
    void *args[] = {&j, &sums, &ids};
    return hipLaunchKernel(reinterpret_cast<const void *>(lora_join_kernel),
                           dim3((unsigned)((p.n + 255) / 256), (unsigned)p.rows), dim3(256), args, 0, s);
}

}  // namespace gemm_f16
