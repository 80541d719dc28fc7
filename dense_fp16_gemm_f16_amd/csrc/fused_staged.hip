// C = act(A B^T + bias) + residual of rows that are not 16-byte aligned (see fused.h).
#include "fused.h"

namespace gemm_f16 {

// The K loop of gemm_f16_kernel for such rows (KMajorOperand; G: 2 rows of whole dwords, 1 any),
// over one part of K: K-tile t + 2 comes into registers and t + 1 goes from there to LDS, shifted
// and masked, among the MFMAs of K-tile t.  (Chunks loaded at their own 2-byte addresses, and
// stored between the K-tiles: 4096 x 4096 x 4097 with silu and residual 247 us, 230 now; 1000 x
// 1000 x 1001 18.7, 11.7.)
template <class C, int G>
__global__ __launch_bounds__(C::kThreads)
__attribute__((amdgpu_waves_per_eu(C::kMinWavesPerEU, C::kMinWavesPerEU)))
void fused_staged_kernel(const FusedParams p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the signature only
    constexpr int KS = C::KS, FM = C::FM, FN = C::FN, NM = FM * FN, NR = FM + FN;
    using OpA = KMajorOperand<C, C::BM, C::TM, G, false, 1>;
    using OpB = KMajorOperand<C, C::BN, C::TN, G, false, 1>;
    constexpr int PA = OpA::kPasses, PB = OpB::kPasses, kLdsB = OpA::kLdsBytes, kLds = kLdsB + OpB::kLdsBytes;
    static_assert(kLds <= 160 * 1024, "LDS budget");
    __shared__ __attribute__((aligned(1024))) char smem[kLds];
    GEMM_POISON_LDS(smem);
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const TileCoord tc = tile_coord<uint32_t>(p.first + blockIdx.x, p.num_m, p.num_n, p.swizzle, p.xcd != 0);
    const int m0 = (int)tc.m_block * C::BM, n0 = (int)tc.n_block * C::BN;
    const int kt0 = (int)blockIdx.y * p.part_kt, kt_count = min(p.part_kt, p.k_tiles - kt0);
    if (kt_count <= 0) return;  // never launched so

    OpA opa;
    OpB opb;
    opa.init(p.a + (int64_t)m0 * p.k, min(C::BM, p.m - m0), p.k, kt_count, tid, lane, wm * C::TM, 0);
    opb.init(p.b + (int64_t)n0 * p.k, min(C::BN, p.n - n0), p.k, kt_count, tid, lane, wn * C::TN, kLdsB);
    // the part's K-tiles are 0 .. kt_count - 1: its first element takes K's beginning
    const int skip = kt0 * C::BK;
    opa.tile += 2 * skip, opa.bytes -= 2 * skip, opa.k_elems -= skip;
    opb.tile += 2 * skip, opb.bytes -= 2 * skip, opb.k_elems -= skip;

    using M = Mfma<C::MB>;
    typename M::Acc acc[FN][FM];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i) acc[j][i] = typename M::Acc{};
    half8 af[2][FM], bf[2][FN];
    auto read_frag = [&](int buf, int stage, int ks, int r) {  // in the order of the MFMAs: B0, A0 .., B1 ..
        if (r == 0)
            bf[buf][0] = opb.read(smem, stage, ks, 0);
        else if (r <= FM)
            af[buf][r - 1] = opa.read(smem, stage, ks, r - 1);
        else
            bf[buf][r - FM] = opb.read(smem, stage, ks, r - FM);
    };
    auto load = [&](int t) {
        opa.begin_tile(t);
        opb.begin_tile(t);
#pragma unroll
        for (int i = 0; i < PA; ++i) opa.load(i, 0);
#pragma unroll
        for (int i = 0; i < PB; ++i) opb.load(i, 0);
    };
    load(0);
#pragma unroll
    for (int i = 0; i < PA; ++i) opa.store(smem, i, 0, 0);
#pragma unroll
    for (int i = 0; i < PB; ++i) opb.store(smem, i, 0, 0);
    load(1);
    lds_barrier();
#pragma unroll
    for (int r = 0; r < NR; ++r) read_frag(0, 0, 0, r);

    // K-tile kt on stage STAGE: behind each MFMA of k step ks < KS - 1 its share of the next step's
    // fragments and of (LDS write of K-tile kt + 1, load of K-tile kt + 2) pairs; in the last step the
    // barrier, then the next K-tile's first fragments.  K-tiles past the last one are zeros.
    constexpr int kBarAt = GEMM_BAR_MFMA < NM ? GEMM_BAR_MFMA : NM - 1;
    auto k_iter = [&](auto stage_tag, int kt) {
        constexpr int STAGE = decltype(stage_tag)::value, NXT = STAGE ^ 1;
        opa.begin_tile(kt + 2);
        opb.begin_tile(kt + 2);
        static_range<0, KS>([&](auto ks_c) {
            constexpr int ks = decltype(ks_c)::value, cur = ks & 1;
            constexpr bool last = ks + 1 == KS;
            constexpr int a0 = ks * PA / (KS - 1), a1 = last ? a0 : (ks + 1) * PA / (KS - 1);
            constexpr int b0 = ks * PB / (KS - 1), b1 = last ? b0 : (ks + 1) * PB / (KS - 1);
            constexpr int nw = a1 - a0 + b1 - b0, total = NR + 2 * nw;
            static_range<0, NM>([&](auto m_c) {
                constexpr int m = decltype(m_c)::value;
                constexpr int j = m / FM, i = (j & 1) ? FM - 1 - m % FM : m % FM;
                acc[j][i] = M::run(bf[cur][j], af[cur][i], acc[j][i]);
                // everyone has read this stage, and the other one is complete
                if constexpr (last && m == kBarAt) lds_barrier();
                constexpr int first = last ? kBarAt : 0;
                constexpr int lo = m < first ? 0 : (m - first) * total / (NM - first);
                constexpr int hi = m < first ? 0 : (m - first + 1) * total / (NM - first);
                static_range<lo, hi>([&](auto o_c) {
                    constexpr int o = decltype(o_c)::value;
                    constexpr int kind = step_op_kind(o, NR, nw), idx = step_op_index(o, NR, nw);
                    constexpr bool is_a = idx < a1 - a0;
                    constexpr int pass = is_a ? a0 + idx : b0 + idx - (a1 - a0);
                    if constexpr (kind == 0)
                        read_frag(cur ^ 1, last ? NXT : STAGE, last ? 0 : ks + 1, idx);
                    else if constexpr (kind == 1)
                        is_a ? opa.store(smem, is_a ? pass : 0, NXT, 0) : opb.store(smem, is_a ? 0 : pass, NXT, 0);
                    else
                        is_a ? opa.load(is_a ? pass : 0, 0) : opb.load(is_a ? 0 : pass, 0);
                });
                __builtin_amdgcn_sched_barrier(0);
            });
            // (live to the step's end: the next step's fragments land in other registers)
#pragma unroll
            for (int j = 0; j < FN; ++j) asm volatile("" ::"v"(bf[cur][j]));
#pragma unroll
            for (int i = 0; i < FM; ++i) asm volatile("" ::"v"(af[cur][i]));
        });
    };
    for (int kt = 0; kt < kt_count; kt += 2) {
        k_iter(std::integral_constant<int, 0>{}, kt);
        k_iter(std::integral_constant<int, 1>{}, kt + 1);
    }
    fused_store_tile<C, kLds>(acc, smem, p, m0, n0, wm, wn, wave, lane);
#endif
}

template <class C>
static hipError_t launch_staged(bool dwords, const FusedParams &p, hipStream_t s) {
    const void *kernel = dwords ? reinterpret_cast<const void *>(fused_staged_kernel<C, 2>)
                                : reinterpret_cast<const void *>(fused_staged_kernel<C, 1>);
    return launch_fused_grid(kernel, (int64_t)p.num_m * p.num_n, p.parts, C::kThreads, s, p);
}

hipError_t launch_fused_staged(const TileSize &tile, bool dwords, const FusedParams &p, hipStream_t s) {
    if (tile.bm == 64) return launch_staged<Cfg64>(dwords, p, s);
    return tile.bn == 128 ? launch_staged<Cfg128>(dwords, p, s) : launch_staged<Cfg128x256>(dwords, p, s);
}

}  // namespace gemm_f16
