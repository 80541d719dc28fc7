// C = act(A B^T + bias) + residual of few rows (see fused.h): decoding.  The time is B's
// bytes, so what matters is how many of them are in flight.
#include "fused.h"
#include "thin_load.h"

namespace gemm_f16 {

// A workgroup takes 16 rows of B (columns of C) and all rows of A.  Its waves share K evenly,
// 8 steps of 32 at a time; a wave's part of B goes straight from memory to registers in the
// MFMA's layout (lane l: row l % 16, 8 elements at 8 (l / 16)), all of it in flight at once,
// and serves T tiles of 16 rows of A.  No LDS and no barrier until the waves' sums meet, in
// wave order.  Any K >= 8, N and alignment: global loads take 2-byte aligned addresses.
constexpr int kFewSteps = 8, kFewWaves = 16;

template <int T>
__global__ __launch_bounds__(kFewWaves *kWave) void fused_few_kernel(const FusedParams p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the signature only
    __shared__ floatx4 red[T][kFewWaves][kWave];
    GEMM_POISON_LDS(red);
    const int tid = threadIdx.x, lane = tid % kWave, waves = blockDim.x / kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int n0 = (int)(p.first + blockIdx.x) * 16, kl = 8 * (lane / 16);
    // Lanes past A's rows or B's read the last one again: their results are never stored.
    const _Float16 *br = p.b + (int64_t)min(n0 + lane % 16, p.n - 1) * p.k;
    const int steps = (p.k + 31) / 32;
    const int part0 = (int)((int64_t)steps * wave / waves), part1 = (int)((int64_t)steps * (wave + 1) / waves);
    floatx4 acc[T];
#pragma unroll
    for (int t = 0; t < T; ++t) acc[t] = floatx4{};
    // the bias and residual of what the lane will store: row 16 wave + l % 16, columns n .. (early, but
    // for four tiles, which leave no registers)
    const int n = n0 + 4 * (lane / 16), m = 16 * wave + lane % 16;
    EpilogueRow<4> out = {};
    if (T < 4 && wave < T) out.load(p, m, n);
    // the lane's row of tile t of A (up to 64 rows of less than 2^22 elements; opaque, as held through
    // the pass they cost registers)
    auto row_of = [&](int t) {
        int l = lane;
        asm volatile("" : "+v"(l));
        return p.a + (uint32_t)min(16 * t + l % 16, p.m - 1) * (uint32_t)p.k;
    };
    for (int top = part1; top > part0; top -= kFewSteps) {
        const int count = min(top - part0, kFewSteps);
        const bool partial = 32 * top > p.k;
        if (count == kFewSteps && !partial) {
            // no branch between the loads, and two half passes of A's tiles in flight behind the
            // one that is multiplied
            constexpr int H = kFewSteps / 2, U = 2 * T;
            half8 bf[kFewSteps], af[3][H];
            const uint32_t k0 = 32 * (top - 1) + kl;
            auto load = [&](half8 &v, const _Float16 *at) { v = __builtin_bit_cast(half8, (int4v)*reinterpret_cast<const int4u *>(at)); };
            auto load_a = [&](int u) {
                const _Float16 *at = row_of(u / 2) + k0;
#pragma unroll
                for (int s = 0; s < H; ++s) load(af[u % 3][s], at - 32 * (u % 2 * H + s));
            };
#pragma unroll
            for (int s = 0; s < kFewSteps; ++s) load(bf[s], br + k0 - 32 * s);
            load_a(0);
            load_a(1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u + 2 < U) load_a(u + 2);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int s = 0; s < H; ++s) acc[u / 2] = Mfma<16>::run(bf[u % 2 * H + s], af[u % 3][s], acc[u / 2]);
                __builtin_amdgcn_sched_barrier(0);
            }
            continue;
        }
        half8 bf[kFewSteps] = {};  // (set, so that nothing of a pass is carried into the next)
        thin_load(bf, br, top, count, partial, kl, p.k);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            half8 af[kFewSteps] = {};
            thin_load(af, row_of(t), top, count, partial, kl, p.k);
#pragma unroll
            for (int s = 0; s < kFewSteps; ++s)
                if (s < count) acc[t] = Mfma<16>::run(bf[s], af[s], acc[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < T; ++t) red[t][wave][lane] = acc[t];
    __syncthreads();
    // (a workgroup has a wave for each tile: launch_fused_few)
    if (wave >= T || m >= p.m || n >= p.n) return;
    if (T == 4) out.load(p, m, n);
    floatx4 sum = red[wave][0][lane];
    for (int w = 1; w < waves; ++w) sum += red[wave][w][lane];
    float z[4], res[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = sum[e];
    out.add(p, m, n, z, res);
    finish_row(p, m, n, z, res);
#endif
}

// ---- one or two rows ---------------------------------------------------------------
//
// A wave takes R rows of B and multiplies lane by lane: 16 bytes a lane, so that a load covers a
// whole kilobyte of a row, where the MFMA's layout takes 64 bytes of each of 16 rows.  R rows by S
// steps of 512 elements, 16 loads, are in flight a wave.  The lanes' sums meet in a fixed order.
// Cold weights, us, beside the MFMA's kernel: one row of 4096 x 4096 7.8 (9.5), 1024 x 4096 4.3
// (7.8), 4096 x 1024 4.6 (4.7), two rows 8.8 (9.6), 5.0 (7.9), 5.5 (4.7): taken by dot_takes.
// From three rows on the vector unit's products cost more than the loads gain (four: 11.0, 9.7).
constexpr int kDotWaves = 4;

// Up to S steps of a row (K >= 8), 512 elements each, `count` of them from step top - 1 downwards;
// 8 elements at 8 lane of each.  The first one, where `partial`, reaches past K (as in thin_load).
template <int S>
__device__ __forceinline__ void dot_load(half8 (&v)[S], const _Float16 *row, int top, int count, bool partial, int lane,
                                         int k_elems) {
    const int k0 = 512 * (top - 1) + 8 * lane;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        v[s] = half8{};
        if (s >= count) continue;
        const int k = s == 0 && partial ? min(k0, k_elems - 8) : k0 - 512 * s;
        v[s] = __builtin_bit_cast(half8, (int4v)*reinterpret_cast<const int4u *>(row + k));
    }
    if (partial) {
        const int past = 8 - (k_elems - k0);  // elements to shift out
        unsigned __int128 w = __builtin_bit_cast(unsigned __int128, v[0]);
        if (past > 0) w = past < 8 ? w >> (16 * past) : 0;
        v[0] = __builtin_bit_cast(half8, w);
    }
}

// x from the lane `by` places away in its row of 16.
template <int CTRL>
__device__ __forceinline__ float dot_turn(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// An element as it comes, and its value (as in RawRow).
__device__ __forceinline__ float load_bits(const void *from, bool f32, int64_t at) {
    return f32 ? static_cast<const float *>(from)[at]
               : __builtin_bit_cast(float, (uint32_t) static_cast<const uint16_t *>(from)[at]);
}
__device__ __forceinline__ float value_of(float bits, bool f32) {
    return f32 ? bits : (float)__builtin_bit_cast(_Float16, (uint16_t)__builtin_bit_cast(uint32_t, bits));
}

template <int M, int R, int S>
__global__ __launch_bounds__(kDotWaves *kWave) void fused_dot_kernel(const FusedParams p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the signature only
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t n0 = ((int64_t)(p.first + blockIdx.x) * kDotWaves + wave) * R;
    if (n0 >= p.n) return;
    // lane m R + r stores row m, column n0 + r: its bias and residual
    const int m = lane / R;
    const int64_t n = n0 + lane % R, at = (int64_t)m * p.n + n;
    const bool mine = m < M && n < p.n;
    float bias = 0.0f, res = 0.0f;
    if (mine && p.bias) bias = load_bits(p.bias, p.bias_f32 != 0, n);
    if (mine && p.residual) res = load_bits(p.residual, p.out_f32 != 0, at);
    float sum[M][R] = {};
    for (int top = (p.k + 511) / 512; top > 0; top -= S) {
        const int count = min(top, S);
        const bool partial = 512 * top > p.k;
        half8 a[M][S], b[R][S];
#pragma unroll
        for (int r = 0; r < R; ++r)  // (past the last row the last one again: not stored)
            dot_load(b[r], p.b + (n0 + r < p.n ? n0 + r : p.n - 1) * p.k, top, count, partial, lane, p.k);
#pragma unroll
        for (int m = 0; m < M; ++m) dot_load(a[m], p.a + (int64_t)m * p.k, top, count, partial, lane, p.k);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (s >= count) continue;
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum[m][r] = __builtin_fmaf((float)a[m][s][e], (float)b[r][s][e], sum[m][r]);
        }
    }
    float z = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float x = sum[m][r];
            x += dot_turn<0x128>(x);  // rotations of a row of 16 lanes by 8, 4, 2 and 1
            x += dot_turn<0x124>(x);
            x += dot_turn<0x122>(x);
            x += dot_turn<0x121>(x);
            x += __shfl_xor(x, 16);
            x += __shfl_xor(x, 32);
            z = lane == m * R + r ? x : z;
        }
    if (!mine) return;
    float y[1] = {p.bias ? z + value_of(bias, p.bias_f32 != 0) : z};
    if (p.pre) p.pre[at] = (_Float16)y[0];
    activate(p.act, y);
    if (p.residual) y[0] += value_of(res, p.out_f32 != 0);
    if (p.out_f32)
        static_cast<float *>(p.c)[at] = y[0];
    else
        static_cast<_Float16 *>(p.c)[at] = (_Float16)y[0];
#endif
}

// Short rows, and two that are not long, are the MFMA's: 300 x 200 takes one row 2.8 us there, 3.4 here.
static bool dot_takes(const FusedParams &p) { return p.m <= 2 && p.k > 512 * p.m; }

// Rows a wave by K: its loads stay 16.
static hipError_t launch_dot(const FusedParams &p, hipStream_t s) {
    const int rows = p.k > 2048 ? 2 : p.k > 1024 ? 4 : 8;  // (8: one row of A)
    const void *kernel = p.m == 2    ? (rows == 2 ? reinterpret_cast<const void *>(fused_dot_kernel<2, 2, 8>)
                                                  : reinterpret_cast<const void *>(fused_dot_kernel<2, 4, 4>))
                         : rows == 2 ? reinterpret_cast<const void *>(fused_dot_kernel<1, 2, 8>)
                         : rows == 4 ? reinterpret_cast<const void *>(fused_dot_kernel<1, 4, 4>)
                                     : reinterpret_cast<const void *>(fused_dot_kernel<1, 8, 2>);
    return launch_fused_grid(kernel, ((int64_t)p.n + rows * kDotWaves - 1) / (rows * kDotWaves), 1, kDotWaves * kWave, s, p);
}

hipError_t launch_fused_few(const FusedParams &p, hipStream_t s) {
    if (dot_takes(p)) return launch_dot(p, s);
    int waves = 1;  // that K keeps busy in one pass
    while (waves < kFewWaves && waves * kFewSteps * 32 < p.k) waves *= 2;
    const int tiles = (p.m + 15) / 16;
    while (waves < tiles) waves *= 2;
    const void *kernel = tiles <= 1   ? reinterpret_cast<const void *>(fused_few_kernel<1>)
                         : tiles == 2 ? reinterpret_cast<const void *>(fused_few_kernel<2>)
                         : tiles == 3 ? reinterpret_cast<const void *>(fused_few_kernel<3>)
                                      : reinterpret_cast<const void *>(fused_few_kernel<4>);
    return launch_fused_grid(kernel, (p.n + 15) / 16, 1, waves * kWave, s, p);
}

// C from the parts' sums of A B^T, added in their order (none: K == 0), 8 columns of a row a
// thread.  All of a thread's loads go out before it waits for one: 48 rows of 1024 x
// 4096 in 8 parts take 9.8 us with the join (one after the other, and with the row found by a 64-bit
// division, 11.3).
__global__ __launch_bounds__(256) void fused_join_kernel(const FusedParams p) {
    const int per = (p.n + 7) / 8;
    const int64_t all = (int64_t)p.m * per, stride = (int64_t)gridDim.x * 256, each = (int64_t)p.m * p.n;
    for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < all; x += stride) {
        const int m = all < (int64_t(1) << 31) ? (int)((uint32_t)x / (uint32_t)per) : (int)(x / per);
        const int n = (int)(x - (int64_t)m * per) * 8;
        const float *s = p.sums + (int64_t)m * p.n + n;
        float z[8] = {}, res[8];
        EpilogueRow<8> out;
        if (n + 8 <= p.n && p.parts > 0) {
            constexpr int B = 4;
            RawRow<8> v[B];
            for (int q0 = 0; q0 < p.parts; q0 += B) {
#pragma unroll
                for (int b = 0; b < B; ++b)
                    if (q0 + b < p.parts) v[b].load(s + (q0 + b) * each, true, 0);
                if (q0 == 0) out.load(p, m, n);
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    if (q0 + b >= p.parts) continue;
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[e] += v[b].v[e / 4][e % 4];
                }
            }
        } else {
            out.load(p, m, n);
            for (int q = 0; q < p.parts; ++q)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (n + e < p.n) z[e] += s[q * each + e];
        }
        out.add(p, m, n, z, res);
        finish_row(p, m, n, z, res);
    }
}

hipError_t launch_fused_join(const FusedParams &p, hipStream_t s) {
    const int64_t blocks = ((int64_t)p.m * ((p.n + 7) / 8) + 255) / 256;
    void *args[] = {const_cast<FusedParams *>(&p)};
    return hipLaunchKernel(reinterpret_cast<const void *>(fused_join_kernel), dim3((unsigned)(blocks < 8192 ? blocks : 8192)),
                           dim3(256), args, 0, s);
}

}  // namespace gemm_f16
