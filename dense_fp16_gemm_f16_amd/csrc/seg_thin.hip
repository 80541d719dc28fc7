// Segmented products of few rows (see segments.h): decoding, and the
// adapters there.  The time is the weights' bytes, so what matters is how
// many of them are in flight.
#include <algorithm>

#include "segments.h"
#include "thin_load.h"

namespace gemm_f16 {

// ---- a segment's rows against 16 rows of B ---------------------------------------
//
// The waves share the steps [s0, s1) of K evenly, each taking up to NB at a
// time; a wave's part of B goes straight from memory to registers in the
// MFMA's layout (lane l: row l % 16, 8 elements at 8 (l / 16)), all of it in
// flight at once, and stays there for all of the segment's rows, 16 at a
// time, if that is all.  No LDS and no barrier until the waves' sums meet, in
// wave order.  Any K >= 8, N and alignment: global loads take 2-byte aligned
// addresses, and the part past K is masked.  Bound by B's bytes and a short
// launch's ramp: 1 row, 904 x 3280, 5.9 MB, in 6.2 us.
//
// Rows lo, lo + step, .. (16 from each) below hi, columns n0 .. n0 + 15 of
// segment g.  store(r, n, sum): sum holds columns n .. n + 3 of row r, zeros
// where the row's index lies outside A.
template <int NB, int NA, int W, class Store>
__device__ __forceinline__ void thin_rows(const SegParams &p, floatx4 (*red)[W][kWave], int g, int n0, int lo, int hi,
                                          int step, int s0, int s1, Store store) {
    const int lane = threadIdx.x % kWave, waves = blockDim.x / kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    // Lanes past the segment's rows or B's columns read the last one again:
    // their results are never stored.
    const int kl = 8 * (lane / 16);
    const _Float16 *br = p.b + ((int64_t)g * p.n + min(n0 + lane % 16, p.n - 1)) * p.k;
    // this wave's steps, [part0, part1)
    const int part0 = s0 + (int)((int64_t)(s1 - s0) * wave / waves);
    const int part1 = s0 + (int)((int64_t)(s1 - s0) * (wave + 1) / waves);
    const bool one_pass = part1 - part0 <= NB;
    half8 bf[NB], af[NA];
    int parity = 0;
    for (int r0 = lo; r0 < hi; r0 += step, parity ^= 1) {
        floatx4 acc = {};
        bool found = true;  // an index outside A: a row of zeros
        const _Float16 *ar = nullptr;
        for (int top = part1; top > part0; top -= NB) {
            const int count = min(top - part0, NB);
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
#pragma unroll
            for (int q = 0; q < NB; q += NA) {
                if (q >= count) continue;
                thin_load(af, ar, top - q, count - q, partial && q == 0, kl, p.k);
#pragma unroll
                for (int s = 0; s < NA; ++s)
                    if (q + s < count) acc = Mfma<16>::run(bf[q + s], af[s], acc);
            }
        }
        red[parity][wave][lane] = acc;
        lds_barrier();
        // (the waves that go on write the other half of red next)
        if (wave != 0) continue;
        // lane l holds row l % 16, columns 4 (l / 16) ..
        floatx4 sum = red[parity][0][lane];
        for (int w = 1; w < waves; ++w) sum += red[parity][w][lane];
        const int r = r0 + lane % 16;
        if (r < hi) store(r, n0 + 4 * (lane / 16), found ? sum : floatx4{});
    }
}

// The segment that slot `slot` of a grid stands for, and its rows: the grid
// has a slot for each segment, or (by_row) for each row, of which the first of
// a segment takes it.  The fewer of the two: one row and 2^20 segments would
// else start 2^20 slots of workgroups, more threads than a launch can have.
// false: nothing to do.
__device__ __forceinline__ bool thin_segment(const SegParams &p, int slot, int lane, int &g, int &lo, int &hi) {
    g = p.by_row ? seg_of_row(p, slot, lane) : slot;
    lo = seg_bound(p.offsets, g, p.rows);
    hi = g < p.groups ? seg_bound(p.offsets, g + 1, p.rows) : p.rows;
    return lo < hi && (!p.by_row || lo == slot);
}

// Slots of a grid over `groups` segments.
static int64_t thin_slots(SegParams &p, int64_t groups) {
    p.by_row = p.rows < groups;
    return p.by_row ? p.rows : groups;
}

// Zeros in h's columns past the rank, up to h_ld; the others times f.
__device__ __forceinline__ void store_h(const SegParams &p, float *h, int n, floatx4 sum, float f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = n + e < p.n ? sum[e] * f : 0.0f;
    if (n < p.h_ld) *reinterpret_cast<floatx4 *>(h + n) = sum;
}

// A grouped NT product (DOWN false), or h in adapter order in its parts (DOWN), a
// segment's rows shared by gridDim.y workgroups.
constexpr int kThinSteps = 8, kThinWaves = 16;
template <bool F32, bool DOWN>
__global__ __launch_bounds__(kThinWaves *kWave) void seg_thin_kernel(const SegParams p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the signature only
    __shared__ floatx4 red[2][kThinWaves][kWave];
    GEMM_POISON_LDS(red);
    const int tid = threadIdx.x;
    const uint32_t pid = seg_pid(p);
    const int n0 = (int)(pid % (uint32_t)p.num_n) * 16;
    int g, lo, hi;
    if (!thin_segment(p, (int)(pid / (uint32_t)p.num_n), tid % kWave, g, lo, hi)) return;
    const bool live = g < p.groups;  // false: the rows behind the last segment
    if (DOWN && !live) return;
    const int step = DOWN ? 16 * (int)gridDim.y : 16;
    if (DOWN) lo += 16 * (int)blockIdx.y;
    if (lo >= hi) return;
    using Out = std::conditional_t<F32, float, _Float16>;
    if (!live) {
        for (int r = lo + tid / 16; r < hi; r += (int)blockDim.x / 16)
            if (n0 + tid % 16 < p.n) static_cast<Out *>(p.c)[(int64_t)r * p.n + n0 + tid % 16] = (Out)0.0f;
        return;
    }
    const float f = DOWN && p.scale ? p.scale[g] : 1.0f;
    thin_rows<kThinSteps, kThinSteps, kThinWaves>(p, red, g, n0, lo, hi, step, 0, (p.k + 31) / 32, [&](int r, int n, floatx4 sum) {
        if constexpr (DOWN) {
            if (n < p.h_ld) store_split(static_cast<char *>(p.c) + (int64_t)r * p.h_ld * kSplitValue, n, sum, f, p.rank);
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
    });
#endif
}

// ---- adapters, up to kLoraFewRows rows --------------------------------------------
//
// One launch for both products by x, whose sums meet in lora_join_kernel:
//  * x W^T: a workgroup takes 64 rows of W and a slice of K, 512 elements at
//    a time: its 4 waves hold 16 rows of W each in registers, and x's rows
//    go through LDS, everything of a step in flight at once.  Slicing K and
//    not N keeps what each CU reads of x at 64 rows by a slice (all of x per
//    CU took 4 us more for each 16 rows);
//  * h = scale_s x D_s^T: 16 ranks of an adapter and a slice of K a
//    workgroup, by thin_rows.
// W 4096 x 4096, rank 16: 10 us for one token, 14 for 48 rows of 32 adapters
// (3.3 TB/s of W), and 4.5 us for the join.
constexpr int kFewWaves = 4, kFewCols = 16 * kFewWaves, kFewSteps = 16, kFewK = 32 * kFewSteps;
[[maybe_unused]] constexpr int kFewPitch = kFewK * 2 + 16;  // bytes of a row of x in LDS: 16 rows at one chunk on 16 banks of 16 bytes

struct FewParams {
    SegParams main, down;
    float *sums;                    // fp32 [main_parts][rows, n]
    int32_t down_blocks;            // workgroups of h: (slot, 16 ranks, part)
    int32_t main_parts, main_steps; // slices of K, and steps of a slice (a multiple of kFewSteps)
    int32_t down_parts, down_steps;
};

// x's elements k .. k + 7 of a row, zeros past K (K >= 8).
__device__ __forceinline__ int4v few_chunk(const _Float16 *row, int k, int k_elems) {
    const int4v v = *reinterpret_cast<const int4u *>(row + min(k, k_elems - 8));
    const int past = k + 8 - k_elems;
    if (past <= 0) return v;
    const unsigned __int128 w = __builtin_bit_cast(unsigned __int128, v);
    return __builtin_bit_cast(int4v, past < 8 ? w >> (16 * past) : (unsigned __int128)0);
}

// T: tiles of 16 rows
template <int T>
__global__ __launch_bounds__(kFewWaves *kWave) __attribute__((amdgpu_waves_per_eu(3, 3)))
void lora_few_kernel(const FewParams fp) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the signature only
    constexpr int kRed = 2 * kFewWaves * kWave * 16;
    __shared__ __attribute__((aligned(1024))) char smem[16 * T * kFewPitch > kRed ? 16 * T * kFewPitch : kRed];
    GEMM_POISON_LDS(smem);
    const int tid = threadIdx.x, lane = tid % kWave;
    const int at = (int)seg_pid(fp.main);
    if (at < fp.down_blocks) {
        const SegParams &p = fp.down;
        const int part = at % fp.down_parts, x = at / fp.down_parts;
        const int n0 = x % p.num_n * 16;
        int g, lo, hi;
        if (!thin_segment(p, x / p.num_n, lane, g, lo, hi) || g >= p.groups) return;
        const int steps = (p.k + 31) / 32, s0 = min(steps, part * fp.down_steps), s1 = min(steps, s0 + fp.down_steps);
        const float f = p.scale ? p.scale[g] : 1.0f;
        float *h = static_cast<float *>(p.c) + (int64_t)part * p.rows * p.h_ld;
        thin_rows<kFewSteps, 8, kFewWaves>(p, reinterpret_cast<floatx4(*)[kFewWaves][kWave]>(smem), g, n0, lo, hi, 16, s0, s1,
                                           [&](int r, int n, floatx4 sum) {
                                               // each row in its own place
                                               const int to = min(max(p.index[r], 0), p.rows - 1);
                                               store_h(p, h + (int64_t)to * p.h_ld, n, sum, f);
                                           });
        return;
    }
    const SegParams &p = fp.main;
    const int pid = at - fp.down_blocks, part = pid / p.num_n;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int n0 = pid % p.num_n * kFewCols + 16 * wave;
    const int steps = (p.k + 31) / 32, s0 = min(steps, part * fp.main_steps), s1 = min(steps, s0 + fp.main_steps);
    const int kl = 8 * (lane / 16);
    const _Float16 *wr = p.b + (int64_t)min(n0 + lane % 16, p.n - 1) * p.k;
    floatx4 acc[T];
#pragma unroll
    for (int t = 0; t < T; ++t) acc[t] = floatx4{};
    for (int step = s0; step < s1; step += kFewSteps) {
        const int count = min(s1 - step, kFewSteps), top = step + count;
        half8 bf[kFewSteps];
        // x: 4 T chunks of 16 bytes a thread, the first 8 of them ahead of W's
        // loads (loads return in order); rows past the last are never stored
        constexpr int X = 4 * T, X0 = X < 8 ? X : 8;
        int4v v[X0];
        auto fetch = [&](int i) {
            const int c = i * kFewWaves * kWave + tid;
            return few_chunk(p.a + (int64_t)min(c / 64, p.rows - 1) * p.k, 32 * step + 8 * (c % 64), p.k);
        };
        auto put = [&](int i, int4v u) {
            const int c = i * kFewWaves * kWave + tid;
            *reinterpret_cast<int4v *>(smem + c / 64 * kFewPitch + c % 64 * 16) = u;
        };
#pragma unroll
        for (int i = 0; i < X0; ++i) v[i] = fetch(i);
        thin_load(bf, wr, top, count, 32 * top > p.k, kl, p.k);
        if (step != s0) lds_barrier();  // the last step's reads are done
#pragma unroll
        for (int i = 0; i < X0; ++i) put(i, v[i]);
#pragma unroll
        for (int i = X0; i < X; ++i) v[i - X0] = fetch(i);
#pragma unroll
        for (int i = X0; i < X; ++i) put(i, v[i - X0]);
        lds_barrier();
#pragma unroll
        for (int s = 0; s < kFewSteps; ++s) {
            if (s >= count) continue;
            const char *from = smem + lane % 16 * kFewPitch + (count - 1 - s) * 64 + kl * 2;
#pragma unroll
            for (int t = 0; t < T; ++t)
                acc[t] = Mfma<16>::run(bf[s], *reinterpret_cast<const half8 *>(from + 16 * t * kFewPitch), acc[t]);
        }
    }
    const int n = n0 + 4 * (lane / 16);
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int r = 16 * t + lane % 16;
        if (r >= p.rows) continue;
        float *c = fp.sums + ((int64_t)part * p.rows + r) * p.n + n;
        if (n + 3 < p.n && p.n % 4 == 0) {
            *reinterpret_cast<floatx4 *>(c) = acc[t];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < p.n) c[e] = acc[t][e];
        }
    }
#endif
}

// y = fp16(x W^T + h U_s^T) from the sums' parts: one workgroup per row and
// 256 columns, every product and sum in fp32.
__global__ __launch_bounds__(256) void lora_join_kernel(const SegParams p, const float *sums, int parts,
                                                        const int32_t *ids) {
    const int r = blockIdx.y, n = (int)(blockIdx.x * 256 + threadIdx.x);
    if (n >= p.n) return;
    const int s = ids[r];
    float v = 0.0f;
#pragma unroll 4
    for (int q = 0; q < parts; ++q) v += sums[((int64_t)q * p.rows + r) * p.n + n];
    if (s >= 0 && s < p.adapters) {
        const _Float16 *u = p.up + ((int64_t)s * p.n + n) * p.rank;
        auto h = [&](int j) {
            float x = 0.0f;
            for (int q = 0; q < p.h_parts; ++q) x += p.h[((int64_t)q * p.rows + r) * p.h_ld + j];
            return x;
        };
        int j = 0;
        for (; j + 8 <= p.rank; j += 8) {
            const half8 w = __builtin_bit_cast(half8, (int4v)*reinterpret_cast<const int4u *>(u + j));
#pragma unroll
            for (int e = 0; e < 8; ++e) v = __builtin_fmaf(h(j + e), (float)w[e], v);
        }
        for (; j < p.rank; ++j) v = __builtin_fmaf(h(j), (float)u[j], v);
    }
    static_cast<_Float16 *>(p.c)[(int64_t)r * p.n + n] = (_Float16)v;
}

// h of K < 8, where no chunk of a row is whole: one lane per 4 values.
__global__ __launch_bounds__(256) void lora_down_short_kernel(const SegParams p) {
    const int per = p.h_ld / 4;
    const int64_t x = (int64_t)seg_pid(p) * 256 + threadIdx.x, r = x / per;
    const int n = (int)(x % per) * 4;
    if (r >= p.rows) return;
    int g = 0;  // the segment of row r
    while (g < p.groups && r >= seg_bound(p.offsets, g + 1, p.rows)) ++g;
    const int src = p.index[r];
    floatx4 sum = {};
    if (g < p.groups && src >= 0 && src < p.a_rows) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (n + e >= p.n) continue;
            for (int k = 0; k < p.k; ++k)
                sum[e] += (float)p.a[(int64_t)src * p.k + k] * (float)p.b[((int64_t)g * p.n + n + e) * p.k + k];
        }
    }
    store_split(static_cast<char *>(p.c) + r * p.h_ld * kSplitValue, n, sum, g < p.groups && p.scale ? p.scale[g] : 1.0f, p.rank);
}

// ---- launches -----------------------------------------------------------------------

template <bool F32, bool DOWN>
static hipError_t launch_thin(SegParams p, int cols, int64_t groups, int shares, hipStream_t s) {
    p.num_n = (cols + 15) / 16;
    const int64_t grid = thin_slots(p, groups) * p.num_n;
    int waves = 1;  // that K keeps busy in one pass
    while (waves < kThinWaves && waves * kThinSteps * 32 < p.k) waves *= 2;
    void *args[] = {&p};
    return launch_grid(reinterpret_cast<const void *>(seg_thin_kernel<F32, DOWN>), grid, shares, waves * kWave, s, args,
                       p.first);
}

hipError_t launch_seg_thin(bool f32, const SegParams &p, hipStream_t s) {
    return f32 ? launch_thin<true, false>(p, p.n, p.groups + 1, 1, s)
               : launch_thin<false, false>(p, p.n, p.groups + 1, 1, s);
}

hipError_t launch_lora_down_thin(const SegParams &p, hipStream_t s) {
    if (p.k < 8) {
        const int64_t grid = ((int64_t)p.rows * (p.h_ld / 4) + 255) / 256;
        return launch_seg(lora_down_short_kernel, grid, 256, s, p);
    }
    // some 64 rows a workgroup of an even split
    const int64_t shares = std::min<int64_t>(std::max<int64_t>(p.rows / (64 * (int64_t)p.groups), 1), 1024);
    return launch_thin<true, true>(p, p.h_ld, p.groups, (int)shares, s);
}

// Slices of K for steps of `unit` 32-wide steps: at most `most`, equal but
// for the last.
static int few_slices(int64_t k, int unit, int most, int32_t *steps) {
    const int64_t all = (k + 31) / 32, units = (all + unit - 1) / unit;
    const int64_t parts = std::min<int64_t>(units, most), each = (units + parts - 1) / parts;
    *steps = (int32_t)(each * unit);
    return (int)((units + each - 1) / each);
}

int lora_few_parts(int64_t k) {
    int32_t steps;
    return few_slices(k, kFewSteps, 8, &steps);
}
int lora_few_h_parts(int64_t k) {
    int32_t steps;
    return few_slices(k, kFewSteps * kFewWaves, 4, &steps);
}

hipError_t launch_lora_few(const SegParams &p, const SegParams &down, float *sums, const int32_t *ids, hipStream_t s) {
    FewParams f = {};
    f.main = p;
    f.main.num_n = (p.n + kFewCols - 1) / kFewCols;
    f.main_parts = few_slices(p.k, kFewSteps, 8, &f.main_steps);
    f.down = down;
    f.down.num_n = (down.h_ld + 15) / 16;
    f.down_parts = few_slices(p.k, kFewSteps * kFewWaves, 4, &f.down_steps);
    f.down_blocks = (int32_t)(thin_slots(f.down, down.groups) * f.down.num_n * f.down_parts);
    f.sums = sums;
    const int64_t grid = f.down_blocks + (int64_t)f.main.num_n * f.main_parts;
    void *args[] = {&f};
    const int tiles = (p.rows + 15) / 16;
    const void *kernel = tiles <= 1   ? reinterpret_cast<const void *>(lora_few_kernel<1>)
                         : tiles == 2 ? reinterpret_cast<const void *>(lora_few_kernel<2>)
                         : tiles == 3 ? reinterpret_cast<const void *>(lora_few_kernel<3>)
                                      : reinterpret_cast<const void *>(lora_few_kernel<4>);
    hipError_t e = launch_grid(kernel, grid, 1, kFewWaves * kWave, s, args, f.main.first);
    if (e != hipSuccess) return e;
    SegParams j = p;
    j.h_parts = f.down_parts;
    void *join[] = {&j, &sums, &f.main_parts, &ids};
    return hipLaunchKernel(reinterpret_cast<const void *>(lora_join_kernel),
                           dim3((unsigned)((p.n + 255) / 256), (unsigned)p.rows), dim3(256), join, 0, s);
}

}  // namespace gemm_f16
