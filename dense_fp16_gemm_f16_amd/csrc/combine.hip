// The way back from the experts: their rows, sorted by expert, weighted and summed into their
// tokens, and the gradient.
//
//   y[t] = residual[t] + sum_f gates[t, f] rows[inverse[t, f]]
//   drows[inverse[t, f]] = gates[t, f] dy[t],   dgates[t, f] = sum_n dy[t, n] rows[inverse[t, f], n]
//
// Places from *last on hold the rows of no expert: they add nothing whatever they hold, and
// have zeros as their gradients.  Sums in fp32, over f in order.  Bound by bytes: every row
// is read and written once, 16 bytes a lane.
#include <algorithm>

#include "fused.h"
#include "route.h"

namespace gemm_f16 {

constexpr int kCombineThreads = 256;

// Place of routed row r: -1 where it is out of range, so no content of inverse leads there.
__device__ __forceinline__ int64_t place_of(const CombineParams &p, int64_t r) {
    const int64_t at = p.inverse[r];
    return at >= 0 && at < p.places ? at : -1;
}

// 8 columns of a row (n < p.n), those past the last 0.
template <bool F32>
__device__ __forceinline__ void load_cols(const CombineParams &p, const void *from, int64_t row, int n, Chunk8<F32> &v) {
    if (n + 8 <= p.n || (!F32 && p.n >= 8)) {
        const int at = chunk_at<8>(n, p.n);
        v.load(from, row * p.n + at);
        if constexpr (!F32)  // (as drop_first)
            if (at < n)
                v.v[0] = __builtin_bit_cast(half8, __builtin_bit_cast(unsigned __int128, v.v[0]) >> (16 * (n - at)));
    } else {
        float last[8];
        load_cols(from, F32, row * p.n, n, p.n, last);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (F32)
                v.v[e / 4][e % 4] = last[e];
            else
                v.v[0][e] = (_Float16)last[e];
        }
    }
}

__device__ __forceinline__ void store_cols(const CombineParams &p, void *to, bool f32, int64_t row, int n, const float (&v)[8]) {
    const int64_t at = row * p.n + n;
    if (n + 8 <= p.n) {
        store_row(to, f32, at, v, kStoreDefault);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (n + e >= p.n) continue;
            if (f32)
                static_cast<float *>(to)[at + e] = v[e];
            else
                static_cast<_Float16 *>(to)[at + e] = (_Float16)v[e];
        }
    }
}

// 2^log threads a token, 8 columns each at a time, in as many workgroups as the grid is high; B rows
// in flight.  ROWS, Y: fp32 rows, y.
template <int B, bool ROWS, bool Y>
__global__ __launch_bounds__(kCombineThreads) void combine_kernel(const CombineParams p, int log) {
    const int64_t token = p.first + ((int64_t)blockIdx.x << (8 - log)) + (threadIdx.x >> log);
    if (token >= p.tokens) return;
    const int step = 8 << log, last = *p.last;
    for (int n = (int)blockIdx.y * step + ((int)threadIdx.x & ((1 << log) - 1)) * 8; n < p.n; n += step * (int)gridDim.y) {
        float y[8] = {};
        if (p.residual) {
            Chunk8<Y> r;
            load_cols(p, p.residual, token, n, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = r[e];
        }
        for (int f0 = 0; f0 < p.fan; f0 += B) {
            Chunk8<ROWS> v[B];
            float gate[B];
            bool live[B];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                live[b] = false;
                if (f0 + b >= p.fan) continue;
                const int64_t r = token * p.fan + f0 + b, at = place_of(p, r);
                live[b] = at >= 0 && at < last;
                gate[b] = p.gates ? p.gates[r] : 1.0f;
                if (live[b]) load_cols(p, p.rows, at, n, v[b]);
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                if (!live[b]) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(gate[b], v[b][e], y[e]);
            }
        }
        store_cols(p, p.y, Y, token, n, y);
    }
}

// 2^log waves a token, which share its columns: dy once, B of the token's rows at a time, two
// chunks of columns in flight.  The waves' sums meet in LDS, in their order.
template <int B, bool ROWS, bool Y>
__global__ __launch_bounds__(kCombineThreads) void combine_grad_kernel(const CombineParams p, int log) {
    constexpr int kWaves = kCombineThreads / kWave;
    __shared__ float red[kWaves][B];
    GEMM_POISON_LDS(red);
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int part = wave & ((1 << log) - 1);
    const int64_t token = p.first + (int64_t)blockIdx.x * (kWaves >> log) + (wave >> log);
    const bool in = token < p.tokens;
    const int last = *p.last;
    for (int f0 = 0; f0 < p.fan; f0 += B) {
        int64_t at[B];
        bool live[B];
        float gate[B], dot[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            at[b] = -1;
            gate[b] = dot[b] = 0.0f;
            if (in && f0 + b < p.fan) {
                const int64_t r = token * p.fan + f0 + b;
                at[b] = place_of(p, r);
                if (at[b] < last) gate[b] = p.gates ? p.gates[r] : 1.0f;
            }
            live[b] = at[b] >= 0 && at[b] < last;
        }
        if (in) {
#pragma unroll 2
            for (int n = (part * kWave + lane) * 8; n < p.n; n += (kWave * 8) << log) {
                Chunk8<Y> dy;
                Chunk8<ROWS> v[B];
                load_cols(p, p.y, token, n, dy);
                if (p.dgates) {
#pragma unroll
                    for (int b = 0; b < B; ++b)  // (a row out of play is the first one: not used)
                        load_cols(p, p.rows, live[b] ? at[b] : 0, n, v[b]);
                }
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    if (at[b] < 0) continue;
                    float d[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        d[e] = live[b] ? gate[b] * dy[e] : 0.0f;
                        if (p.dgates) dot[b] = live[b] ? __builtin_fmaf(dy[e], v[b][e], dot[b]) : dot[b];
                    }
                    if (p.drows) store_cols(p, p.drows, p.drows_f32 != 0, at[b], n, d);
                }
            }
        }
        if (!p.dgates) continue;
#pragma unroll
        for (int b = 0; b < B; ++b) {
#pragma unroll
            for (int d = 1; d < kWave; d <<= 1) dot[b] += __shfl_xor(dot[b], d);
        }
        if (log > 0) {
            if (f0 > 0) __syncthreads();  // (read before it is written again)
            if (lane == 0)
#pragma unroll
                for (int b = 0; b < B; ++b) red[wave][b] = dot[b];
            __syncthreads();
            if (part != 0) continue;
            for (int w = 1; w < 1 << log; ++w)
#pragma unroll
                for (int b = 0; b < B; ++b) dot[b] += red[wave + w][b];
        }
        if (lane != 0 || !in) continue;
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (f0 + b < p.fan) p.dgates[token * p.fan + f0 + b] = dot[b];
    }
}

// `per` tokens a workgroup, `high` workgroups a token; a launch holds fewer than 2^32 threads.
static hipError_t launch(const void *kernel, CombineParams p, int per, int high, int log, hipStream_t s) {
    const int64_t kMost = ((int64_t(1) << 32) - 1) / kCombineThreads / high;
    void *args[] = {&p, &log};
    for (int64_t at = 0, all = (p.tokens + per - 1) / per; at < all; at += kMost) {
        p.first = at * per;
        const hipError_t e = hipLaunchKernel(kernel, dim3((unsigned)std::min(kMost, all - at), (unsigned)high),
                                             dim3(kCombineThreads), args, 0, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <bool ROWS, bool Y>
static const void *kernel_of(bool grad, int64_t fan) {
    if (grad)
        return fan <= 1   ? reinterpret_cast<const void *>(combine_grad_kernel<1, ROWS, Y>)
               : fan <= 2 ? reinterpret_cast<const void *>(combine_grad_kernel<2, ROWS, Y>)
                          : reinterpret_cast<const void *>(combine_grad_kernel<4, ROWS, Y>);
    return fan <= 2   ? reinterpret_cast<const void *>(combine_kernel<2, ROWS, Y>)
           : fan <= 4 ? reinterpret_cast<const void *>(combine_kernel<4, ROWS, Y>)
                      : reinterpret_cast<const void *>(combine_kernel<8, ROWS, Y>);
}

static const void *kernel_of(bool grad, const CombineParams &p) {
    if (p.rows_f32) return p.y_f32 ? kernel_of<true, true>(grad, p.fan) : kernel_of<true, false>(grad, p.fan);
    return p.y_f32 ? kernel_of<false, true>(grad, p.fan) : kernel_of<false, false>(grad, p.fan);
}

hipError_t launch_combine(const CombineParams &p, hipStream_t s) {
    int log = 3;  // threads a token: its chunks of 8 columns, or a workgroup
    while (log < 8 && (8 << log) < p.n) ++log;
    // few tokens: long rows go to several workgroups (64 tokens of 8 rows of 7168: 5.5 us,
    // 13.5 with one)
    const int per = kCombineThreads >> log;
    const int64_t blocks = (p.tokens + per - 1) / per, steps = (p.n + (8 << log) - 1) / (8 << log);
    const int high = (int)std::max<int64_t>(1, std::min(steps, 1024 / blocks));
    return launch(kernel_of(false, p), p, per, high, log, s);
}

hipError_t launch_combine_grad(const CombineParams &p, hipStream_t s) {
    // waves a token: one for each 1024 columns (8192 tokens of 2 rows of 4096: 73 us, with one wave each
    // 85, the last of them alone on the chip; 64 tokens 5.0 and 10.2; 1000 of 6 rows of 7168 43 and 71)
    int log = 0;
    while (log < 2 && (1024 << log) < p.n) ++log;
    return launch(kernel_of(true, p), p, (kCombineThreads / kWave) >> log, 1, log, s);
}

}  // namespace gemm_f16
