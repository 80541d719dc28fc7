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
    for (int top = part1; top > part0; top -= kFewSteps) {
        const int count = min(top - part0, kFewSteps);
        const bool partial = 32 * top > p.k;
        half8 bf[kFewSteps];
        thin_load(bf, br, top, count, partial, kl, p.k);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            half8 af[kFewSteps];
            thin_load(af, p.a + (int64_t)min(16 * t + lane % 16, p.m - 1) * p.k, top, count, partial, kl, p.k);
#pragma unroll
            for (int s = 0; s < kFewSteps; ++s)
                if (s < count) acc[t] = Mfma<16>::run(bf[s], af[s], acc[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < T; ++t) red[t][wave][lane] = acc[t];
    __syncthreads();
    // lane l of tile t: row 16 t + l % 16, columns n0 + 4 (l / 16) ..
    const int n = n0 + 4 * (lane / 16);
    for (int t = wave; t < T; t += waves) {
        const int m = 16 * t + lane % 16;
        if (m >= p.m || n >= p.n) continue;
        float bias[4], res[4], z[4];
        load_bias(p, n, bias);
        load_residual(p, m, n, res);
        floatx4 sum = red[t][0][lane];
        for (int w = 1; w < waves; ++w) sum += red[t][w][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = sum[e] + bias[e];
        finish_row(p, m, n, z, res);
    }
#endif
}

hipError_t launch_fused_few(const FusedParams &p, hipStream_t s) {
    int waves = 1;  // that K keeps busy in one pass
    while (waves < kFewWaves && waves * kFewSteps * 32 < p.k) waves *= 2;
    const int tiles = (p.m + 15) / 16;
    const void *kernel = tiles <= 1   ? reinterpret_cast<const void *>(fused_few_kernel<1>)
                         : tiles == 2 ? reinterpret_cast<const void *>(fused_few_kernel<2>)
                         : tiles == 3 ? reinterpret_cast<const void *>(fused_few_kernel<3>)
                                      : reinterpret_cast<const void *>(fused_few_kernel<4>);
    return launch_fused_grid(kernel, (p.n + 15) / 16, 1, waves * kWave, s, p);
}

// C from the parts' sums of A B^T, added in their order (none: K == 0), 8 columns of a row a
// thread.
__global__ __launch_bounds__(256) void fused_join_kernel(const FusedParams p) {
    const int per = (p.n + 7) / 8;
    const int64_t all = (int64_t)p.m * per, stride = (int64_t)gridDim.x * 256, each = (int64_t)p.m * p.n;
    for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < all; x += stride) {
        const int m = (int)(x / per), n = (int)(x % per) * 8;
        float z[8], res[8];
        load_bias(p, n, z);
        load_residual(p, m, n, res);
        float sum[8] = {};
        const float *s = p.sums + (int64_t)m * p.n + n;
#pragma unroll 4
        for (int q = 0; q < p.parts; ++q, s += each) {
            if (p.vec) {
                float v[8];
                load_row(s, true, 0, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += v[e];
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (n + e < p.n) sum[e] += s[e];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] += sum[e];
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
