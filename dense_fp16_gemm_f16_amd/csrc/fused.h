// C = act(A B^T + bias) + residual for gfx950: the dense product with what
// follows it in a feed-forward layer taken into its epilogue, and the
// elementwise part of its gradient.
//
// The K loops and LDS layouts are those of kernels.h; what is new is the way
// out.  Everything behind the fp32 sum z = A B^T + bias stays in fp32 and C is
// rounded once (nearest even); `pre` is z rounded to fp16, for the gradient.
#pragma once

#include "kernels.h"

namespace gemm_f16 {

// (GEMM_F16_ACT_* of gemm_f16.h)
enum Act : int32_t { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

struct FusedParams : Params {
    const void *bias;      // [n] fp16 or fp32, or null
    const void *residual;  // [m, n] of C's type, or null; C itself, or apart from it
    _Float16 *pre;         // [m, n] or null
    float *sums;           // parts > 1: fp32 [parts][m, n], the parts' sums of A B^T
    int32_t act, bias_f32, out_f32;
    int32_t vec;           // C, pre, residual and bias in whole aligned 16-byte chunks of 8 columns
    int32_t parts, part_kt;  // parts of K (1: none), of part_kt K-tiles each
    uint32_t first;          // workgroups of this grid that earlier launches hold (launch_fused_grid)
};

// ---- activations ---------------------------------------------------------------

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid_f32(float x) {
    // past the range of exp2 this is 0 or 1, as it should be
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -kLog2e));
}

// gelu_tanh(z) = z / 2 (1 + tanh u) = z sigmoid(2 u), u = sqrt(2/pi) (z + 0.044715 z^3):
// this form has no cancellation for negative z.
constexpr float kGeluC0 = 1.5957691216057308f, kGeluC1 = 0.07135481282705285f;  // 2 sqrt(2/pi), times 0.044715

// Phi(z) = erfc(-z / sqrt 2) / 2 and e = exp(-z^2 / 2).  For x = |z| the function
// exp(x^2 / 2) Phi(-x) is smooth and falls like 1/x: a polynomial in t = 1 / (1 + 0.31 x)
// without a constant term, fitted to it for least relative error over 0 <= x <= 15 (where
// Phi(-x) leaves fp32), is off by 1.7e-7 of it, 4.8e-7 in fp32.  So the small values of
// the lower tail keep their relative precision too.
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    const float x = __builtin_fabsf(z);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.31f, x, 1.0f));
    e = __builtin_amdgcn_exp2f(x * x * (-0.5f * kLog2e));
    float q = 0.035890500992536545f;
    q = __builtin_fmaf(q, t, -0.14181861281394958f);
    q = __builtin_fmaf(q, t, 0.15545809268951416f);
    q = __builtin_fmaf(q, t, -0.015285272151231766f);
    q = __builtin_fmaf(q, t, 0.11032592505216599f);
    q = __builtin_fmaf(q, t, 0.10770097374916077f);
    q = __builtin_fmaf(q, t, 0.12407241761684418f);
    q = __builtin_fmaf(q, t, 0.12365606427192688f);
    const float lower = q * t * e;
    return z > 0.0f ? 1.0f - lower : lower;
}

// act(z), uniform over the launch.  What is not finite gives what the formula gives: -inf
// is a NaN past relu and none (0 * inf), NaN stays NaN.
template <int N>
__device__ __forceinline__ void activate(int act, float (&z)[N]) {
    switch (act) {
        case kActRelu:
#pragma unroll
            for (int e = 0; e < N; ++e) z[e] = z[e] < 0.0f ? 0.0f : z[e];
            break;
        case kActGelu:
#pragma unroll
            for (int e = 0; e < N; ++e) {
                float gauss;
                z[e] *= normal_cdf(z[e], gauss);
            }
            break;
        case kActGeluTanh:
#pragma unroll
            for (int e = 0; e < N; ++e) z[e] *= sigmoid_f32(z[e] * __builtin_fmaf(kGeluC1, z[e] * z[e], kGeluC0));
            break;
        case kActSilu:
#pragma unroll
            for (int e = 0; e < N; ++e) z[e] *= sigmoid_f32(z[e]);
            break;
        default: break;
    }
}

// ---- the way out ------------------------------------------------------------------

// 16 bytes at an element's own alignment, which global loads and stores take (rows of other than
// whole chunks, element by element: 4096 x 4100 x 4096 with silu and residual 252 us, 188 now).
typedef float floatx4u __attribute__((ext_vector_type(4), aligned(4)));
typedef int int4nu __attribute__((ext_vector_type(4), aligned(2)));
template <int N>
using halfnu = _Float16 __attribute__((ext_vector_type(N), aligned(2)));

// N (4 or 8) values of a row from element `at` on: fp16 or fp32.
template <int N>
__device__ __forceinline__ void load_row(const void *from, bool f32, int64_t at, float (&v)[N]) {
    if (f32) {
        const floatx4u *q = reinterpret_cast<const floatx4u *>(static_cast<const float *>(from) + at);
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const floatx4 x = q[i];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * i + e] = x[e];
        }
    } else {
        const halfnu<N> x = *reinterpret_cast<const halfnu<N> *>(static_cast<const _Float16 *>(from) + at);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = (float)x[e];
    }
}

__device__ __forceinline__ float load1(const void *from, bool f32, int64_t at) {
    return f32 ? static_cast<const float *>(from)[at] : (float)static_cast<const _Float16 *>(from)[at];
}

// 8 columns of a row as they come, converted where they are used: in half the registers of 8
// floats.
template <bool F32>
struct Chunk8 {
    std::conditional_t<F32, floatx4, half8> v[F32 ? 2 : 1];

    __device__ __forceinline__ void load(const void *from, int64_t at) {
        if constexpr (F32) {
            const floatx4u *q = reinterpret_cast<const floatx4u *>(static_cast<const float *>(from) + at);
            v[0] = q[0];
            v[1] = q[1];
        } else {
            v[0] = *reinterpret_cast<const halfnu<8> *>(static_cast<const _Float16 *>(from) + at);
        }
    }
    __device__ __forceinline__ float operator[](int e) const {
        if constexpr (F32)
            return v[e / 4][e % 4];
        else
            return (float)v[0][e];
    }
};

// 16 bytes under C's cache policy (CStore), where they are aligned.
__device__ __forceinline__ void store16(void *to, int4v v, int policy) {
    if (policy == kStoreDevice)
        store_device_scope(to, v);
    else if (policy == kStoreStream)
        __builtin_nontemporal_store(v, reinterpret_cast<int4v *>(to));
    else
        *reinterpret_cast<int4nu *>(to) = v;
}

// N values rounded to fp16 (nearest even) or kept.
template <int N>
__device__ __forceinline__ void store_row(void *to, bool f32, int64_t at, const float (&v)[N], int policy) {
    if (f32) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            store16(static_cast<float *>(to) + at + 4 * i,
                    __builtin_bit_cast(int4v, floatx4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]}), policy);
    } else {
        halfnu<N> h;
#pragma unroll
        for (int e = 0; e < N; ++e) h[e] = (_Float16)v[e];
        _Float16 *q = static_cast<_Float16 *>(to) + at;
        if constexpr (N == 8)
            store16(q, __builtin_bit_cast(int4v, h), policy);
        else
            *reinterpret_cast<halfnu<N> *>(q) = h;
    }
}

// N (4 or 8) values of a row as they come, fp16 or fp32, for loads that go out before anything
// waits for them.
template <int N>
struct RawRow {
    floatx4 v[N / 4];

    __device__ __forceinline__ void load(const void *from, bool f32, int64_t at) {
        if (f32) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) v[i] = reinterpret_cast<const floatx4u *>(static_cast<const float *>(from) + at)[i];
        } else {
            const halfnu<N> h = *reinterpret_cast<const halfnu<N> *>(static_cast<const _Float16 *>(from) + at);
            __builtin_memcpy(v, &h, sizeof(_Float16) * N);
        }
    }
    __device__ __forceinline__ void values(bool f32, float (&x)[N]) const {
        _Float16 h[N];
        __builtin_memcpy(h, v, sizeof(h));
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = f32 ? v[e / 4][e % 4] : (float)h[e];
    }
};

// Columns n .. n + N - 1 of a row of `cols` (n < cols): where some are outside, the row's last N are
// loaded, one chunk still, and moved down by drop_first; a row of fewer than N has no chunk.
template <int N>
__device__ __forceinline__ int chunk_at(int n, int cols) {
    return n + N <= cols ? n : cols - N;
}

// v[e] = v[e + by], zeros behind, by < N.
template <int N>
__device__ __forceinline__ void drop_first(float (&v)[N], int by) {
#pragma unroll
    for (int d = 1; d < N; d *= 2)
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = (by & d) ? (e + d < N ? v[e + d] : 0.0f) : v[e];
}

// Columns n .. n + N - 1 (n < cols) of the row that begins at element `at`, zeros past the last.
template <int N>
__device__ __forceinline__ void load_cols(const void *from, bool f32, int64_t at, int n, int cols, float (&v)[N]) {
    if (n + N <= cols) {
        load_row(from, f32, at + n, v);
    } else if (cols >= N) {
        load_row(from, f32, at + cols - N, v);
        drop_first(v, n + N - cols);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = n + e < cols ? load1(from, f32, at + n + e) : 0.0f;
    }
}

// The bias of columns n .. n + N - 1, zeros past the last and without one.
template <int N>
__device__ __forceinline__ void load_bias(const FusedParams &p, int n, float (&b)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) b[e] = 0.0f;
    if (p.bias && n < p.n) load_cols(p.bias, p.bias_f32 != 0, 0, n, p.n, b);
}

// The residual of row m, columns n .. n + N - 1 (n < p.n), if there is one.
template <int N>
__device__ __forceinline__ void load_residual(const FusedParams &p, int m, int n, float (&r)[N]) {
    if (p.residual) load_cols(p.residual, p.out_f32 != 0, (int64_t)m * p.n, n, p.n, r);
}

// Bias and residual of row m, columns n .. n + N - 1 (n < p.n): asked for early, taken late.
template <int N>
struct EpilogueRow {
    RawRow<N> bias, res;

    __device__ __forceinline__ void load(const FusedParams &p, int m, int n) {
        if (m >= p.m || n >= p.n || p.n < N) return;
        const int from = chunk_at<N>(n, p.n);
        if (p.bias) bias.load(p.bias, p.bias_f32 != 0, from);
        if (p.residual) res.load(p.residual, p.out_f32 != 0, (int64_t)m * p.n + from);
    }
    // z += bias; r: the residual
    __device__ __forceinline__ void add(const FusedParams &p, int m, int n, float (&z)[N], float (&r)[N]) const {
        float b[N] = {};
        if (p.n < N) {
            load_bias(p, n, b);
            load_residual(p, m, n, r);
        } else {
            if (p.bias) bias.values(p.bias_f32 != 0, b);
            if (p.residual) res.values(p.out_f32 != 0, r);
            if (n + N > p.n) {
                drop_first(b, n + N - p.n);
                if (p.residual) drop_first(r, n + N - p.n);
            }
        }
#pragma unroll
        for (int e = 0; e < N; ++e) z[e] += b[e];
    }
};

// Row m, columns n .. n + N - 1 (n < p.n) of C from z, with r of load_residual.
template <int N>
__device__ __forceinline__ void finish_row(const FusedParams &p, int m, int n, float (&z)[N], const float (&r)[N]) {
    const int64_t at = (int64_t)m * p.n + n;
    const bool whole = n + N <= p.n;
    if (p.pre) {
        if (whole) {
            store_row(p.pre, false, at, z, p.c_store);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (n + e < p.n) p.pre[at + e] = (_Float16)z[e];
        }
    }
    activate(p.act, z);
    if (p.residual) {
#pragma unroll
        for (int e = 0; e < N; ++e) z[e] += r[e];
    }
    if (whole) {
        store_row(p.c, p.out_f32 != 0, at, z, p.c_store);
        return;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        if (n + e >= p.n) continue;
        if (p.out_f32)
            static_cast<float *>(p.c)[at + e] = z[e];
        else
            static_cast<_Float16 *>(p.c)[at + e] = (_Float16)z[e];
    }
}

// The workgroup's tile from its accumulators: fp32 through LDS, each wave its own piece in
// its own share (CStaging's fp32 layout), then 8 consecutive columns a lane, so that the
// bias is read once per wave and residual, pre and C move in whole 16-byte chunks of row
// segments.  The loop is kept rolled: one copy of the epilogue's code, whatever the
// activation.  Four rows' residuals are in flight at a time.
template <class C, int kLds>
__device__ __forceinline__ void fused_store_tile(const typename Mfma<C::MB>::Acc (&acc)[C::FN][C::FM], char *smem,
                                                 const FusedParams &p, int m0, int n0, int wm, int wn, int wave,
                                                 int lane) {
    constexpr int kWaveBytes = kLds / C::kWaves;
    using CS = CStaging<C, true, kWaveBytes>;
    constexpr int CPL = C::TN / 8, RPI = kWave / CPL, IT = CS::SR / RPI, B = IT < 4 ? IT : 4;
    static_assert(IT % B == 0 && IT * RPI == CS::SR, "whole batches of rows");
    const int erow = CS::opaque_row(lane);
    const int c8 = lane % CPL, n = n0 + wn * C::TN + 8 * c8;
    float bias[8];
    load_bias(p, n, bias);
    lds_barrier();
    char *const stg = smem + wave * (CS::SR * CS::RB);
#pragma unroll
    for (int pass = 0; pass < CS::kPasses; ++pass) {
        CS::write_pass(acc, stg, pass, erow, lane);
#pragma unroll 1
        for (int it = 0; it < IT; it += B) {
            float res[B][8];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int m = m0 + wm * C::TM + pass * CS::SR + (it + b) * RPI + lane / CPL;
                if (p.parts == 1 && m < p.m && n < p.n) load_residual(p, m, n, res[b]);
            }
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const int r = (it + b) * RPI + lane / CPL, m = m0 + wm * C::TM + pass * CS::SR + r;
                const char *row = stg + r * CS::RB;
                const floatx4 x = *reinterpret_cast<const floatx4 *>(row + (((2 * c8) ^ (r % CS::CPR)) << 4));
                const floatx4 y = *reinterpret_cast<const floatx4 *>(row + (((2 * c8 + 1) ^ (r % CS::CPR)) << 4));
                if (m >= p.m || n >= p.n) continue;
                if (p.parts > 1) {
                    // this part's sums, each part in rows of its own
                    float *s = p.sums + ((int64_t)blockIdx.y * p.m + m) * p.n + n;
                    if (n + 7 < p.n) {
                        *reinterpret_cast<floatx4u *>(s) = x;
                        *reinterpret_cast<floatx4u *>(s + 4) = y;
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (n + e < p.n) s[e] = e < 4 ? x[e & 3] : y[e & 3];
                    }
                    continue;
                }
                float z[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) z[e] = x[e] + bias[e], z[4 + e] = y[e] + bias[4 + e];
                finish_row(p, m, n, z, res[b]);
            }
        }
    }
}

// The K loop of gemm_f16_direct_ahead_kernel over K-tiles kt0 .. kt0 + kt_count - 1: two LDS
// stages, both k steps' fragments of K-tile t+1 read during K-tile t, a release and an acquire
// barrier per K-tile.
template <class C, class OpA, class OpB>
__device__ __forceinline__ void fused_k_loop(const OpA &opa, const OpB &opb, floatx4 (&acc)[C::FN][C::FM], char *smem, int kt0,
                                             int kt_count) {
    constexpr int FM = C::FM, FN = C::FN;
    constexpr int LA = OpA::kLoads, L = OpA::kLoads + OpB::kLoads;
    static_assert(2 * L < 64, "vmcnt range");
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i) acc[j][i] = floatx4{};
    acc_fence(acc);

    half8 af[3][FM];
    half8 bf[3][FN];
    constexpr int NR = FM + FN;  // fragment reads per k step
    // in the order the MFMAs consume them: B0, A0..A(FM-1), B1..
    auto read_frag = [&](int buf, int stage, int ks, int r) {
        if (r == 0)
            bf[buf][0] = opb.read(smem, stage, ks, 0);
        else if (r <= FM)
            af[buf][r - 1] = opa.read(smem, stage, ks, r - 1);
        else
            bf[buf][r - FM] = opb.read(smem, stage, ks, r - FM);
    };
    auto load = [&](auto s_c, int t, int i) {
        constexpr int S = decltype(s_c)::value;
        if (i < LA)
            opa.template load<S>(smem, t, i);
        else
            opb.template load<S>(smem, t, i - LA);
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    constexpr int NM = FM * FN;
    constexpr int kRelAt = GEMM_AHEAD_REL_MFMA < NM ? GEMM_AHEAD_REL_MFMA : NM - 1;
    constexpr int kAcqAt = GEMM_AHEAD_ACQ_MFMA < NM ? GEMM_AHEAD_ACQ_MFMA : NM - 1;
    constexpr int L0 = L * GEMM_AHEAD_STEP0_LOADS / 16;  // loads of K-tile t+2 in step 0

#pragma unroll
    for (int i = 0; i < L; ++i) load(S0{}, kt0, i);
#pragma unroll
    for (int i = 0; i < L; ++i) load(S1{}, kt0 + 1, i);
    vm_barrier<L>();
#pragma unroll
    for (int r = 0; r < NR; ++r) read_frag(0, 0, 0, r);
#pragma unroll
    for (int r = 0; r < NR; ++r) read_frag(1, 0, 1, r);

    auto k_iter = [&](auto s_c, int t) {
        constexpr int S = decltype(s_c)::value;
        constexpr int SN = S ^ 1;
        constexpr int B1 = S == 0 ? 1 : 2;   // this K-tile's step-1 buffer
        constexpr int NB1 = S == 0 ? 2 : 1;  // the next K-tile's
        static_range<0, NM>([&](auto m_c) {
            constexpr int m = decltype(m_c)::value;
            constexpr int j = m / FM, i = (j & 1) ? FM - 1 - m % FM : m % FM;
            mfma16_tied(bf[0][j], af[0][i], acc[j][i]);
            if constexpr (m == kRelAt) lgkm_barrier();
            if constexpr (m >= kRelAt) {
                constexpr int q = m - kRelAt, slots = NM - kRelAt;
                static_range<q * L0 / slots, (q + 1) * L0 / slots>(
                    [&](auto o_c) { load(s_c, t + 2, decltype(o_c)::value); });
            }
            __builtin_amdgcn_sched_barrier(0);
        });
#pragma unroll
        for (int j = 0; j < FN; ++j) asm volatile("" ::"v"(bf[0][j]));
#pragma unroll
        for (int i = 0; i < FM; ++i) asm volatile("" ::"v"(af[0][i]));
        static_range<0, NM>([&](auto m_c) {
            constexpr int m = decltype(m_c)::value;
            constexpr int j = m / FM, i = (j & 1) ? FM - 1 - m % FM : m % FM;
            mfma16_tied(bf[B1][j], af[B1][i], acc[j][i]);
            if constexpr (m == kAcqAt) vm_only_barrier<L0>();
            if constexpr (m >= kAcqAt) {
                constexpr int nl = L - L0, total = 2 * NR + nl, slots = NM - kAcqAt, q = m - kAcqAt;
                // R R L R R L ...: the reads first while both remain
                static_range<q * total / slots, (q + 1) * total / slots>([&](auto o_c) {
                    constexpr int o = decltype(o_c)::value;
                    constexpr int groups = (2 * NR) / 2 < nl ? (2 * NR) / 2 : nl;  // (R, R, L) groups
                    constexpr bool in_groups = o < 3 * groups;
                    constexpr bool is_read = in_groups ? (o % 3 != 2) : (2 * NR > 2 * groups);
                    constexpr int idx = in_groups ? (is_read ? (o / 3) * 2 + (o % 3) : o / 3)
                                                  : (is_read ? 2 * groups + (o - 3 * groups) : groups + (o - 3 * groups));
                    if constexpr (is_read) {
                        constexpr int ks = idx / NR, r = idx % NR;
                        read_frag(ks == 0 ? 0 : NB1, SN, ks, r);
                    } else {
                        load(s_c, t + 2, L0 + idx);
                    }
                });
            }
            __builtin_amdgcn_sched_barrier(0);
        });
#pragma unroll
        for (int j = 0; j < FN; ++j) asm volatile("" ::"v"(bf[B1][j]));
#pragma unroll
        for (int i = 0; i < FM; ++i) asm volatile("" ::"v"(af[B1][i]));
    };
    // K-tiles in pairs (stage 0, stage 1); an odd count ends with one more on stage 0.
    // Loads past the last fill stages that are never summed.
    int kt = 0;
    for (; kt + 1 < kt_count; kt += 2) {
        k_iter(S0{}, kt0 + kt);
        k_iter(S1{}, kt0 + kt + 1);
    }
    // The accumulators may move where the two ways on meet, and the compiler knows of no MFMA
    // still writing them: each way waits for its own.
    acc_fence(acc);
    if (kt < kt_count) {
        k_iter(S0{}, kt0 + kt);
        acc_fence(acc);
    }
    vm_barrier<0>();  // no load is still writing LDS
}

// One block tile per workgroup, operands straight into LDS (16-byte aligned rows).  With parts
// > 1 blockIdx.y is a part of K, whose sums leave in fp32 for fused_join_kernel.
template <class C>
__global__ __launch_bounds__(C::kThreads)
__attribute__((amdgpu_waves_per_eu(C::kMinWavesPerEU, C::kMinWavesPerEU)))
void fused_tile_kernel(const FusedParams p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the signature only
    constexpr int BM = C::BM, BN = C::BN;
    static_assert(C::MB == 16 && C::KS == 2, "two 32-wide k steps per K-tile");
    using OpA = KMajorDirect<C, BM, false>;
    using OpB = KMajorDirect<C, BN, false>;
    constexpr int kLdsB = OpA::kLdsBytes, kLds = OpA::kLdsBytes + OpB::kLdsBytes;
    static_assert(kLds <= 160 * 1024, "LDS budget");
    __shared__ __attribute__((aligned(1024))) char smem[kLds];
    GEMM_POISON_LDS(smem);

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const TileCoord tc = tile_coord<uint32_t>(p.first + blockIdx.x, p.num_m, p.num_n, p.swizzle, p.xcd != 0);
    const int m0 = (int)tc.m_block * BM, n0 = (int)tc.n_block * BN;
    const int kt0 = (int)blockIdx.y * p.part_kt, kt_count = min(p.part_kt, p.k_tiles - kt0);  // this part's K-tiles
    if (kt_count <= 0) return;  // never launched so

    OpA opa;
    OpB opb;
    opa.init(p.a + (int64_t)m0 * p.k, min(BM, p.m - m0), p.k, kt0 + kt_count, wave, lane, wm * C::TM, 0);
    opb.init(p.b + (int64_t)n0 * p.k, min(BN, p.n - n0), p.k, kt0 + kt_count, wave, lane, wn * C::TN, kLdsB);
    floatx4 acc[C::FN][C::FM];
    fused_k_loop<C>(opa, opb, acc, smem, kt0, kt_count);
    fused_store_tile<C, kLds>(acc, smem, p, m0, n0, wm, wn, wave, lane);
#endif
}

// The same for fp16 results in whole 16-byte chunks, which leave straight from the accumulators:
// B's fragment rows are interleaved (KMajorDirect PERM), so a lane's blocks (2q, i) and (2q + 1,
// i) hold 8 neighbouring columns of row 16 i + l % 16.  With the K loop over, its fragments'
// registers hold the residual of kAhead such units in flight.
// ACT and RES are template arguments: the units are unrolled, and a copy for each activation
// would not fit the instruction cache.
template <class C, int ACT, bool RES>
__global__ __launch_bounds__(C::kThreads)
__attribute__((amdgpu_waves_per_eu(C::kMinWavesPerEU, C::kMinWavesPerEU)))
void fused_direct_kernel(const FusedParams p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the signature only
    constexpr int BM = C::BM, BN = C::BN, FM = C::FM, FN = C::FN;
    static_assert(C::MB == 16 && C::KS == 2 && FN % 2 == 0, "two 32-wide k steps per K-tile, blocks in pairs");
    using OpA = KMajorDirect<C, BM, false>;
    using OpB = KMajorDirect<C, BN, false, true>;
    constexpr int kLdsB = OpA::kLdsBytes, kLds = OpA::kLdsBytes + OpB::kLdsBytes;
    static_assert(kLds <= 160 * 1024, "LDS budget");
    __shared__ __attribute__((aligned(1024))) char smem[kLds];
    GEMM_POISON_LDS(smem);

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const TileCoord tc = tile_coord<uint32_t>(p.first + blockIdx.x, p.num_m, p.num_n, p.swizzle, p.xcd != 0);
    const int m0 = (int)tc.m_block * BM, n0 = (int)tc.n_block * BN;
    if (p.k_tiles == 0) return;  // never launched so

    OpA opa;
    OpB opb;
    opa.init(p.a + (int64_t)m0 * p.k, min(BM, p.m - m0), p.k, p.k_tiles, wave, lane, wm * C::TM, 0);
    opb.init(p.b + (int64_t)n0 * p.k, min(BN, p.n - n0), p.k, p.k_tiles, wave, lane, wn * C::TN, kLdsB);
    floatx4 acc[FN][FM];
    fused_k_loop<C>(opa, opb, acc, smem, 0, p.k_tiles);

    // (opaque copies: what hangs on them is computed here, not held through the K loop)
    int l = lane, row0 = m0 + wm * C::TM, col0 = n0 + wn * C::TN;
    asm volatile("" : "+v"(l), "+s"(row0), "+s"(col0));
    constexpr int U = FM * FN / 2, kAhead = U < 16 ? U : 16;
    const int m_l = row0 + l % 16, n_l = col0 + 8 * (l / 16);
    auto inside = [&](int u) { return m_l + 16 * (u % FM) < p.m && n_l + 32 * (u / FM) < p.n; };
    auto at_of = [&](int u) { return (int64_t)(m_l + 16 * (u % FM)) * p.n + n_l + 32 * (u / FM); };
    float bias[FN / 2][8];
#pragma unroll
    for (int q = 0; q < FN / 2; ++q) load_bias(p, n_l + 32 * q, bias[q]);
    half8 res[RES ? kAhead : 1];
    auto load_res = [&](auto u_c) {
        constexpr int u = decltype(u_c)::value;
        if constexpr (RES && u < U) {
            if (inside(u)) res[u % kAhead] = *reinterpret_cast<const half8 *>(static_cast<const _Float16 *>(p.residual) + at_of(u));
        }
    };
    static_range<0, kAhead>(load_res);
    static_range<0, U>([&](auto u_c) {
        constexpr int u = decltype(u_c)::value, q = u / FM, i = u % FM;
        float z[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            z[e] = acc[2 * q][i][e] + bias[q][e];
            z[4 + e] = acc[2 * q + 1][i][e] + bias[q][4 + e];
        }
        const bool in = inside(u);
        const int64_t at = at_of(u);
        if (p.pre && in) store_row(p.pre, false, at, z, p.c_store);
        activate(ACT, z);
        if constexpr (RES) {
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] += (float)res[u % kAhead][e];
            load_res(std::integral_constant<int, u + kAhead>{});
        }
        if (in) store_row(p.c, false, at, z, p.c_store);
    });
#endif
}

// ---- launches ------------------------------------------------------------------

// A launch holds fewer than 2^32 threads along x, and one of more loses the rest without an
// error: such a grid (below 2^31 workgroups) goes out in several.  parts: the grid's y.
inline hipError_t launch_fused_grid(const void *kernel, int64_t grid, int parts, int threads, hipStream_t s,
                                    FusedParams p) {
    if (grid >= (int64_t(1) << 31)) return hipErrorInvalidValue;
    const int64_t most = ((int64_t(1) << 32) - 1) / threads;
    for (int64_t at = 0; at < grid; at += most) {
        p.first = (uint32_t)at;
        void *args[] = {&p};
        const hipError_t e = hipLaunchKernel(kernel, dim3((unsigned)(grid - at < most ? grid - at : most), (unsigned)parts),
                                             dim3((unsigned)threads), args, 0, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class C, int ACT>
const void *fused_direct(const FusedParams &p) {
    return p.residual ? reinterpret_cast<const void *>(fused_direct_kernel<C, ACT, true>)
                      : reinterpret_cast<const void *>(fused_direct_kernel<C, ACT, false>);
}

template <class C>
hipError_t launch_fused_tile(const FusedParams &p, hipStream_t s) {
    const void *kernel = reinterpret_cast<const void *>(fused_tile_kernel<C>);
    if (p.vec && !p.out_f32 && p.parts == 1) {
        switch (p.act) {
            case kActRelu: kernel = fused_direct<C, kActRelu>(p); break;
            case kActGelu: kernel = fused_direct<C, kActGelu>(p); break;
            case kActGeluTanh: kernel = fused_direct<C, kActGeluTanh>(p); break;
            case kActSilu: kernel = fused_direct<C, kActSilu>(p); break;
            default: kernel = fused_direct<C, kActNone>(p); break;
        }
    }
    return launch_fused_grid(kernel, (int64_t)p.num_m * p.num_n, p.parts, C::kThreads, s, p);
}

// One unit per block tile, so that they compile in parallel.
hipError_t launch_fused_256x256(const FusedParams &p, hipStream_t s);
hipError_t launch_fused_256x128(const FusedParams &p, hipStream_t s);
hipError_t launch_fused_128x256(const FusedParams &p, hipStream_t s);
hipError_t launch_fused_128x128(const FusedParams &p, hipStream_t s);
hipError_t launch_fused_128x64(const FusedParams &p, hipStream_t s);
hipError_t launch_fused_64x128(const FusedParams &p, hipStream_t s);
hipError_t launch_fused_64x64(const FusedParams &p, hipStream_t s);

// More tiles than CUs, fp16 C in whole 16-byte chunks, at least 3 K-tiles (256 x 256: an even
// number of whole ones): fused_walk.h.
hipError_t launch_fused_walk_256x256(const FusedParams &p, int cus, hipStream_t s);
hipError_t launch_fused_walk_256x128(const FusedParams &p, int cus, hipStream_t s);
hipError_t launch_fused_walk_128x256(const FusedParams &p, int cus, hipStream_t s);

// 64 x 64 tiles on a ring of LDS stages (fused_ring.hip).
hipError_t launch_fused_ring(const FusedParams &p, hipStream_t s);

struct TileSize {
    int bm, bn;
};

// Rows that are not 16-byte aligned, any K >= 1 (fused_staged.hip), on a tile of 64 x 64, 128 x 128
// or 128 x 256; dwords: rows of whole dwords.
hipError_t launch_fused_staged(const TileSize &tile, bool dwords, const FusedParams &p, hipStream_t s);

// Few rows (fused_few.hip): K >= 8, any alignment.
constexpr int kFusedFewRows = 64;
hipError_t launch_fused_few(const FusedParams &p, hipStream_t s);

// C from the parts' sums (parts 0: from zeros, K == 0).
hipError_t launch_fused_join(const FusedParams &p, hipStream_t s);

// dz = dy act'(pre), dbias = column sums (fused_grad.hip).
struct FusedGradParams {
    const void *dy;        // [m, n], fp16 or fp32
    const _Float16 *pre;   // [m, n], null without an activation
    _Float16 *dz;          // [m, n] or null
    float *dbias;          // [n] or null
    float *sums;           // dbias: [parts][n]
    int64_t m, n;
    int32_t act, dy_f32, parts;
};
hipError_t launch_fused_grad(const FusedGradParams &p, hipStream_t s);
int fused_grad_parts(int64_t m, int64_t n);

}  // namespace gemm_f16
