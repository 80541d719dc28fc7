// C = act(A B^T + bias) + residual where the operands' bytes bound the product (see fused.h): few
// rows or few columns.
#include "fused.h"

namespace gemm_f16 {

// One 64 x 64 tile (or a part of its K) per workgroup, a ring of S LDS stages loaded S - 1 K-tiles
// ahead, one barrier per K-tile: before it every wave has read the stage that the next load fills,
// and has waited for its own loads of the next K-tile.  The two stages of fused_tile_kernel leave
// a CU waiting for memory most of the time here.
//
// Rows a power of two apart put one K-tile of every row on the same memory channels, so workgroups in
// step would all wait for those.  Where one tile holds all rows of A, each starts elsewhere in K by its
// columns (64 x 8192 x 12288: 47.8 us, 56.7 without).  By rows that would make a row's results depend
// on where in the batch it stands: there (EIGHTHS) K is taken in eighths, and a workgroup flips bits
// of their number.  Each starts elsewhere too, and as neighbours, pairs and fours are added up as a
// tree, whose two sides may change places, all have the same sums to the bit (16384 x 64 x 4096,
// fp32: 28.5 us, 33.2 in step).
template <class C, int S, bool EIGHTHS>
__global__ __launch_bounds__(C::kThreads) void fused_ring_kernel(const FusedParams p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the signature only
    constexpr int FM = C::FM, FN = C::FN;
    using OpA = KMajorDirect<C, C::BM, false>;
    using OpB = KMajorDirect<C, C::BN, false>;
    constexpr int kStage = OpA::kStage + OpB::kStage, kLds = S * kStage;
    constexpr int LA = OpA::kLoads, L = OpA::kLoads + OpB::kLoads;
    static_assert(kLds <= 160 * 1024 && S >= 3 && (S - 1) * L < 64, "LDS budget, vmcnt range");
    __shared__ __attribute__((aligned(1024))) char smem[kLds];
    GEMM_POISON_LDS(smem);

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const uint32_t pid = p.first + blockIdx.x;
    const TileCoord tc = tile_coord<uint32_t>(pid, p.num_m, p.num_n, p.swizzle, p.xcd != 0);
    const int m0 = (int)tc.m_block * C::BM, n0 = (int)tc.n_block * C::BN;
    const int kt0 = (int)blockIdx.y * p.part_kt, kt1 = min(kt0 + p.part_kt, p.k_tiles), turns = kt1 - kt0;
    // This part's K-tiles from `start` on, or in eighths: e ^ flip is the e-th.
    const bool eighths = EIGHTHS && p.num_n == 1 && p.num_m > 1 && turns >= 8;
    const int start = p.num_m == 1 && turns > 0 ? (int)((pid * 5u) % (uint32_t)turns) : 0;
    const int flip = eighths ? (int)(pid & 7u) : 0;
    auto first = [&](int e) { return eighths ? (int)((int64_t)turns * e >> 3) : 0; };
    auto past = [&](int e) { return eighths ? (int)((int64_t)turns * (e + 1) >> 3) : turns; };

    OpA opa;
    OpB opb;
    opa.init(p.a + (int64_t)m0 * p.k, min(C::BM, p.m - m0), p.k, kt1, wave, lane, wm * C::TM, 0);
    opb.init(p.b + (int64_t)n0 * p.k, min(C::BN, p.n - n0), p.k, kt1, wave, lane, wn * C::TN, OpA::kStage);
    floatx4 acc[FN][FM];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i) acc[j][i] = floatx4{};
    int loads = 0, e = 0, at = eighths ? first(flip) : start, end = past(flip);  // of the next load
    auto load = [&](int stage) {  // past the last K-tile: empty loads, for the count
        char *to = smem + stage * kStage;
        const int t = loads++ < turns ? kt0 + at : kt1;
        if (++at == end) {
            ++e;
            at = first(e ^ flip), end = past(e ^ flip);
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (i < LA)
                opa.template load<0>(to, t, i);
            else
                opb.template load<0>(to, t, i - LA);
        }
    };
#pragma unroll
    for (int s = 0; s < S - 1; ++s) load(s);
    int stage = 0, done = 0, left = past(flip) - first(flip);
    floatx4 sums[EIGHTHS ? 3 : 1][FN][FM];
    for (int t = 0; t < turns; ++t) {
        vm_barrier<(S - 2) * L>();
        load(stage == 0 ? S - 1 : stage - 1);
        const char *from = smem + stage * kStage;
#pragma unroll
        for (int ks = 0; ks < C::KS; ++ks) {
            half8 af[FM], bf[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i) af[i] = opa.read(from, 0, ks, i);
#pragma unroll
            for (int j = 0; j < FN; ++j) bf[j] = opb.read(from, 0, ks, j);
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int i = 0; i < FM; ++i) acc[j][i] = Mfma<16>::run(bf[j], af[i], acc[j][i]);
        }
        stage = stage == S - 1 ? 0 : stage + 1;
        if (!EIGHTHS || !eighths || --left > 0) continue;
        // An eighth is done: its sum waits for its neighbour's, the two's for theirs, and so on.
        ++done;
        left = past(done ^ flip) - first(done ^ flip);
        static_range<0, EIGHTHS ? 3 : 0>([&](auto b_c) {
            constexpr int b = decltype(b_c)::value;
            if (done % (1 << b) != 0) return;
            const bool second = (done >> b) % 2 == 0;
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    if (second)
                        acc[j][i] += sums[b][j][i];
                    else
                        sums[b][j][i] = acc[j][i], acc[j][i] = floatx4{};
                }
        });
    }
    vm_barrier<0>();  // no load is still writing LDS when C is staged there
    fused_store_tile<C, kLds / 1024 / C::kWaves * C::kWaves * 1024>(acc, smem, p, m0, n0, wm, wn, wave, lane);
#endif
}

// Five stages fill a CU's LDS with two workgroups, three with three: more workgroups where parts of
// K make more than there is room for (64 rows of 4096 x 4096 in 4 parts: 13.7 us, with five 14.2;
// 16384 x 64 x 4096, one workgroup a CU: 35 us, with five 31.4).  No eighths of parts, which cost
// their kernel more than they gain (4096 x 64 x 4096 12.3 us, 15.4 with them; 8192 x 64 x 8192 36.3 and
// 37.3, where starts by rows took 33.7).
hipError_t launch_fused_ring(const FusedParams &p, hipStream_t s) {
    using C = Cfg<64, 64, 2, 2, 16>;
    const void *kernel = p.parts > 1 ? reinterpret_cast<const void *>(fused_ring_kernel<C, 3, false>)
                                     : reinterpret_cast<const void *>(fused_ring_kernel<C, 5, true>);
    return launch_fused_grid(kernel, (int64_t)p.num_m * p.num_n, p.parts, C::kThreads, s, p);
}

}  // namespace gemm_f16
