// C = act(A B^T + bias) + residual of rows that are not 16-byte aligned (see fused.h): the
// operands go through registers into the direct kernels' LDS layout.
#include "fused.h"
#include "segments.h"

namespace gemm_f16 {

template <class C>
__global__ __launch_bounds__(C::kThreads) void fused_staged_kernel(const FusedParams p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the signature only
    using OpA = KMajorStaged<C, C::BM>;
    using OpB = KMajorStaged<C, C::BN>;
    constexpr int kLdsB = 2 * OpA::kStage, kLds = kLdsB + 2 * OpB::kStage;
    __shared__ __attribute__((aligned(1024))) char smem[kLds];
    GEMM_POISON_LDS(smem);
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const TileCoord tc = tile_coord<uint32_t>(p.first + blockIdx.x, p.num_m, p.num_n, p.swizzle, p.xcd != 0);
    const int m0 = (int)tc.m_block * C::BM, n0 = (int)tc.n_block * C::BN;
    const int kt0 = (int)blockIdx.y * p.part_kt, kt1 = min(kt0 + p.part_kt, p.k_tiles);
    OpA opa;
    OpB opb;
    opa.init(p.a + (int64_t)p.m * p.k, p.k, wave, lane, wm * C::TM, 0);
    opb.init(p.b + (int64_t)p.n * p.k, p.k, wave, lane, wn * C::TN, kLdsB);
#pragma unroll
    for (int i = 0; i < OpA::kLoads; ++i) {
        const int r = m0 + OpA::tile_row(i, wave, lane);
        opa.row[i] = r < p.m ? p.a + (int64_t)r * p.k : nullptr;
    }
#pragma unroll
    for (int i = 0; i < OpB::kLoads; ++i) {
        const int r = n0 + OpB::tile_row(i, wave, lane);
        opb.row[i] = r < p.n ? p.b + (int64_t)r * p.k : nullptr;
    }
    floatx4 acc[C::FN][C::FM];
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int i = 0; i < C::FM; ++i) acc[j][i] = floatx4{};
    opa.load(kt0);
    opb.load(kt0);
    opa.store(smem, 0);
    opb.store(smem, 0);
    lds_barrier();
    for (int t = kt0; t < kt1; ++t) {
        const int stage = (t - kt0) & 1;
        const bool more = t + 1 < kt1;
        if (more) {
            opa.load(t + 1);
            opb.load(t + 1);
        }
#pragma unroll
        for (int ks = 0; ks < C::KS; ++ks) {
            half8 af[C::FM];
#pragma unroll
            for (int i = 0; i < C::FM; ++i) af[i] = opa.read(smem, stage, ks, i);
#pragma unroll
            for (int j = 0; j < C::FN; ++j) {
                const half8 bf = opb.read(smem, stage, ks, j);
#pragma unroll
                for (int i = 0; i < C::FM; ++i) acc[j][i] = Mfma<16>::run(bf, af[i], acc[j][i]);
            }
        }
        // the other stage was last read before the barrier that ended the K-tile before
        if (more) {
            opa.store(smem, stage ^ 1);
            opb.store(smem, stage ^ 1);
        }
        lds_barrier();
    }
    fused_store_tile<C, kLds>(acc, smem, p, m0, n0, wm, wn, wave, lane);
#endif
}

template <class C>
static hipError_t launch_staged(const FusedParams &p, hipStream_t s) {
    return launch_fused_grid(reinterpret_cast<const void *>(fused_staged_kernel<C>), (int64_t)p.num_m * p.num_n, p.parts,
                             C::kThreads, s, p);
}

hipError_t launch_fused_staged(bool wide, const FusedParams &p, hipStream_t s) {
    return wide ? launch_staged<Cfg<128, 128, 2, 2, 16>>(p, s) : launch_staged<Cfg<64, 64, 2, 2, 16>>(p, s);
}

}  // namespace gemm_f16
