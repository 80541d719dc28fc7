// The elementwise part of the gradient of C = act(A B^T + bias) + residual:
//
//   dz = dy act'(z),   dbias[n] = sum_m dz[m][n]
//
// one pass over dy and z, the sums taken before dz is rounded.
#include "fused.h"

namespace gemm_f16 {

// act'(z) times dy, in place.  Where the fp32 z was past fp16's range pre is an infinity, and a
// product with z would be inf * 0: where the bell (gelu) or s (1 - s) has come to 0, the slope is what
// is left, 0 or 1, at either infinity and short of it.  NaN stays.
template <int ACT, int N>
__device__ __forceinline__ void activate_grad(const float (&z)[N], float (&dy)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if constexpr (ACT == kActRelu) {
            dy[e] = z[e] > 0.0f ? dy[e] : z[e] <= 0.0f ? 0.0f : z[e];  // NaN stays
        } else if constexpr (ACT == kActGelu) {  // Phi(z) + z phi(z)
            float gauss;
            const float cdf = normal_cdf(z[e], gauss);
            dy[e] *= gauss == 0.0f ? cdf : __builtin_fmaf(z[e] * 0.3989422804014327f, gauss, cdf);
        } else if constexpr (ACT == kActGeluTanh) {  // s = sigmoid(w): s + z s (1 - s) dw/dz
            const float q = z[e] * z[e], s = sigmoid_f32(z[e] * __builtin_fmaf(kGeluC1, q, kGeluC0));
            const float bell = s * (1.0f - s);
            dy[e] *= bell == 0.0f ? s : __builtin_fmaf(z[e] * __builtin_fmaf(3.0f * kGeluC1, q, kGeluC0), bell, s);
        } else if constexpr (ACT == kActSilu) {
            const float s = sigmoid_f32(z[e]), bell = s * (1.0f - s);
            dy[e] *= bell == 0.0f ? s : __builtin_fmaf(z[e], bell, s);
        }
    }
}

// A workgroup takes W chunks of 8 columns and the rows of one part, 256 / W of them at a
// time; a thread keeps the sums of its 8 columns, which meet in LDS in a fixed order.
// Bound by bytes: 16384 x 4096 with gelu_tanh 85 us for 403 MB, a copy's rate.  Four rows of dy and
// z are in flight a thread, as they come (as floats they took twice the registers, and half the
// waves were left: 146 us).
constexpr int kGradThreads = 256, kGradRows = 4;

template <int W, bool F32, int ACT>
__global__ __launch_bounds__(kGradThreads) void fused_grad_kernel(const FusedGradParams p) {
    constexpr int H = kGradThreads / W;
    __shared__ float red[H][W * 8 + 1];
    GEMM_POISON_LDS(red);
    const int c = threadIdx.x % W, h = threadIdx.x / W;
    const int64_t n = ((int64_t)blockIdx.x * W + c) * 8;
    const int64_t per = (p.m + p.parts - 1) / p.parts;
    const int64_t lo = (int64_t)blockIdx.y * per, hi = lo + per < p.m ? lo + per : p.m;
    float sum[8] = {};
    // (the last columns, where they are no whole chunk, come with the ones before them)
    const int64_t from = n + 8 <= p.n ? n : p.n - 8;
    const int skip = (int)(n - from);  // elements of the chunk that are another thread's
    if (n < p.n && p.n >= 8) {
        for (int64_t r0 = lo + h; r0 < hi; r0 += H * kGradRows) {
            Chunk8<F32> raw[kGradRows];
            Chunk8<false> pre[kGradRows];
#pragma unroll
            for (int i = 0; i < kGradRows; ++i) {
                const int64_t r = r0 + i * H < hi ? r0 + i * H : r0;  // (the first again: not used)
                raw[i].load(p.dy, r * p.n + from);
                if constexpr (ACT != kActNone) pre[i].load(p.pre, r * p.n + from);
            }
#pragma unroll
            for (int i = 0; i < kGradRows; ++i) {
                const int64_t r = r0 + i * H;
                if (r >= hi) continue;
                float dy[8], z[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dy[e] = raw[i][e];
                    z[e] = ACT != kActNone ? pre[i][e] : 0.0f;
                }
                activate_grad<ACT>(z, dy);
                if (p.dz && skip == 0) store_row(p.dz, false, r * p.n + n, dy, kStoreDefault);
                if (p.dz && skip != 0) {
#pragma unroll
                    for (int e = 1; e < 8; ++e)
                        if (e >= skip) p.dz[r * p.n + from + e] = (_Float16)dy[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += dy[e];
            }
        }
        if (skip != 0) drop_first(sum, skip);
    } else if (n < p.n) {  // rows of fewer than 8 columns
        for (int64_t r = lo + h; r < hi; r += H) {
            const int64_t at = r * p.n + n;
            float dy[8], z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = n + e < p.n;
                dy[e] = in ? load1(p.dy, F32, at + e) : 0.0f;
                z[e] = in && ACT != kActNone ? (float)p.pre[at + e] : 0.0f;
            }
            activate_grad<ACT>(z, dy);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (n + e >= p.n) continue;
                if (p.dz) p.dz[at + e] = (_Float16)dy[e];
                sum[e] += dy[e];
            }
        }
    }
    if (!p.dbias) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) red[h][8 * c + e] = sum[e];
    __syncthreads();
    for (int x = threadIdx.x; x < W * 8; x += kGradThreads) {
        const int64_t col = (int64_t)blockIdx.x * W * 8 + x;
        if (col >= p.n) continue;
        float v = 0.0f;
        for (int i = 0; i < H; ++i) v += red[i][x];
        (p.parts > 1 ? p.sums + (int64_t)blockIdx.y * p.n : p.dbias)[col] = v;
    }
}

// dbias from the parts' sums: 32 columns a workgroup, eight threads a column.
__global__ __launch_bounds__(256) void fused_grad_join_kernel(const FusedGradParams p) {
    __shared__ float red[8][32];
    GEMM_POISON_LDS(red);
    const int x = threadIdx.x % 32, h = threadIdx.x / 32;
    const int64_t col = (int64_t)blockIdx.x * 32 + x;
    float v = 0.0f;
    if (col < p.n) {
#pragma unroll 16
        for (int q = h; q < p.parts; q += 8) v += p.sums[(int64_t)q * p.n + col];
    }
    red[h][x] = v;
    __syncthreads();
    if (h != 0 || col >= p.n) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) v += red[i][x];
    p.dbias[col] = v;
}

// Chunks of 8 columns that a workgroup takes: rows' segments of up to 512 bytes.
static int grad_width(int64_t n) { return n > 128 ? 32 : n > 32 ? 16 : 4; }

// Parts of the rows: workgroups for every CU several times over; up to kGradAlone steps go without
// (64 x 4096 with gelu_tanh: 5.7 us, 6.3 in two parts with their join; 96 rows 7.4 and 6.3).
constexpr int64_t kGradAlone = 2;
int fused_grad_parts(int64_t m, int64_t n) {
    const int w = grad_width(n);
    const int64_t cols = (n + 8 * w - 1) / (8 * w), step = kGradThreads / w * kGradRows;
    int64_t parts = (2048 + cols - 1) / (cols > 0 ? cols : 1);
    if (parts > (m + step - 1) / step) parts = (m + step - 1) / step;
    if (m <= kGradAlone * step) parts = 1;
    return (int)(parts < 1 ? 1 : parts);
}

template <int W, bool F32>
static const void *grad_kernel(int act) {
    switch (act) {
        case kActRelu: return reinterpret_cast<const void *>(fused_grad_kernel<W, F32, kActRelu>);
        case kActGelu: return reinterpret_cast<const void *>(fused_grad_kernel<W, F32, kActGelu>);
        case kActGeluTanh: return reinterpret_cast<const void *>(fused_grad_kernel<W, F32, kActGeluTanh>);
        case kActSilu: return reinterpret_cast<const void *>(fused_grad_kernel<W, F32, kActSilu>);
        default: return reinterpret_cast<const void *>(fused_grad_kernel<W, F32, kActNone>);
    }
}

template <int W>
static const void *grad_kernel(const FusedGradParams &p) {
    return p.dy_f32 ? grad_kernel<W, true>(p.act) : grad_kernel<W, false>(p.act);
}

hipError_t launch_fused_grad(const FusedGradParams &p, hipStream_t s) {
    const int w = grad_width(p.n);
    const void *kernel = w == 32 ? grad_kernel<32>(p) : w == 16 ? grad_kernel<16>(p) : grad_kernel<4>(p);
    void *args[] = {const_cast<FusedGradParams *>(&p)};
    const int64_t cols = (p.n + 8 * w - 1) / (8 * w);
    hipError_t e = hipLaunchKernel(kernel, dim3((unsigned)cols, (unsigned)p.parts), dim3(kGradThreads), args, 0, s);
    if (e != hipSuccess || !p.dbias || p.parts == 1) return e;
    return hipLaunchKernel(reinterpret_cast<const void *>(fused_grad_join_kernel), dim3((unsigned)((p.n + 31) / 32)), dim3(256),
                           args, 0, s);
}

}  // namespace gemm_f16
