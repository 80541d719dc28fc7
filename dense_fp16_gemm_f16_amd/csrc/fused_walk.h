// C = act(A B^T + bias) + residual, fp16, on grids of more tiles than CUs: one workgroup per CU
// walks its tiles without a pause between them.
#pragma once

#include "fused.h"

namespace gemm_f16 {

// gemm_f16_stream_kernel's walk: the K-tile stream runs on across tiles (the last two K-tiles
// of a tile load the next tile's first two), B's fragment rows are interleaved so that a lane's
// blocks (2p, i) and (2p + 1, i) hold 8 neighbouring columns of a row, "unit" u = p FM + i, and
// a unit of the finished tile leaves right before the MFMAs that overwrite its accumulators in
// the next tile's first K-tile.  On the way out here:
//  * the bias of the wave's columns comes straight into LDS, one load at the tile's start (an
//    empty range, zeros, without a bias), and is read once per p;
//  * the residual (RES) is loaded kAhead units ahead, into the registers of the fragment buffer
//    that the first K-tile's step 0 leaves free;
//  * pre leaves like C, into an empty range where it is not wanted.
// A unit's arithmetic takes longer than the two MFMAs it stands before, so what it costs, it
// costs: 256 elements a lane and tile.
// ACT, RES, POL (cache policy of the stores) are template arguments: a branch in a unit costs
// scalar registers that the 256-wide tiles do not have.  KFULL: K in an even number of whole
// K-tiles; otherwise chunks past K read zeros, which the 256 x 256 tile has no registers for.
template <class C, int ACT, bool RES, int POL, bool KFULL>
__global__ __launch_bounds__(C::kThreads)
__attribute__((amdgpu_waves_per_eu(C::kMinWavesPerEU, C::kMinWavesPerEU)))
void fused_walk_kernel(const FusedParams p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the signature only
    constexpr int BM = C::BM, BN = C::BN;
    constexpr int TM = C::TM, TN = C::TN, FM = C::FM, FN = C::FN;
    static_assert(C::MB == 16 && C::KS == 2 && FN % 2 == 0, "two 32-wide k steps per K-tile, blocks in pairs");
    using OpA = KMajorDirect<C, BM, KFULL>;
    using OpB = KMajorDirect<C, BN, KFULL, true>;
    constexpr int kLdsB = OpA::kLdsBytes, kLds = OpA::kLdsBytes + OpB::kLdsBytes;
    constexpr int LA = OpA::kLoads, L = OpA::kLoads + OpB::kLoads;
    constexpr int NM = FM * FN;  // MFMAs per k step
    constexpr int U = NM / 2;    // units per wave and tile
    constexpr int kAhead = 8;    // units whose residual is in flight
    constexpr int kBias = TN * 4;  // bytes of a wave's columns (fp32) in LDS, twice: this tile's and the last one's
    static_assert(NM >= 16 && U >= kAhead, "the units need a window of several MFMAs");
    static_assert(TN <= 256, "the bias of a wave's columns is one load");
    static_assert(kLds + 2 * C::kWaves * kBias <= 160 * 1024, "LDS budget");
    static_assert(OpA::kStage + (FM - 1) * C::MB * 128 < 65536 && OpB::kStage + (FN / 2 - 1) * 32 * 128 < 65536,
                  "LDS immediates must fit the 16-bit offset field");
    // one array: with two, the compiler waits for every load in flight before each fragment read
    __shared__ __attribute__((aligned(1024))) char smem[kLds + 2 * C::kWaves * kBias];
    GEMM_POISON_LDS(smem);

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / C::WN, wn = wave % C::WN;

    // K-tiles per tile: even and >= 4.  An odd count is rounded up: the extra K-tile lies past K
    // and reads zeros, whose MFMAs add +0 to accumulators that are never -0.
    const int kt_count = KFULL ? p.k_tiles : (p.k_tiles + 1) & ~1;
    const int ntiles = p.num_m * p.num_n;
    const int G = gridDim.x;
    int idx = blockIdx.x;

    // first rows of A and B of a tile and the bytes of its rows inside the matrices (0 past the
    // last tile: loads read zeros); C's first row and its elements inside
    struct TileRows {
        const _Float16 *a, *b;
        uint32_t a_bytes, b_bytes, c_elems;
        int m0, n0;
    };
    auto tile_rows = [&](int id) {
        TileRows r;
        if (id < ntiles) {
            const TileCoord tc = tile_coord<uint32_t>(id, p.num_m, p.num_n, p.swizzle, p.xcd != 0);
            r.m0 = (int)tc.m_block * BM;
            r.n0 = (int)tc.n_block * BN;
            const uint32_t rows_a = (uint32_t)min(BM, p.m - r.m0), rows_b = (uint32_t)min(BN, p.n - r.n0);
            r.a = p.a + (int64_t)r.m0 * p.k;
            r.b = p.b + (int64_t)r.n0 * p.k;
            r.a_bytes = rows_a * (uint32_t)p.k * 2u;
            r.b_bytes = rows_b * (uint32_t)p.k * 2u;
            r.c_elems = rows_a * (uint32_t)p.n;
        } else {
            r.a = p.a;
            r.b = p.b;
            r.a_bytes = r.b_bytes = r.c_elems = 0u;
            r.m0 = r.n0 = 0;
        }
        // wave-uniform by construction; readfirstlane keeps them in scalar registers
        auto u32 = [](uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane(v); };
        auto uptr = [&](auto *q) {
            const uint64_t v = (uint64_t)(uintptr_t)q;
            return (decltype(q))(uintptr_t)(((uint64_t)u32((uint32_t)(v >> 32)) << 32) | u32((uint32_t)v));
        };
        r.a = uptr(r.a);
        r.b = uptr(r.b);
        r.a_bytes = u32(r.a_bytes);
        r.b_bytes = u32(r.b_bytes);
        r.c_elems = u32(r.c_elems);
        r.m0 = (int)u32((uint32_t)r.m0);
        r.n0 = (int)u32((uint32_t)r.n0);
        return r;
    };
    TileRows cur = tile_rows(idx);
    TileRows nxt = tile_rows(idx + G);

    OpA opa;
    OpB opb;
    opa.init(cur.a, 0, p.k, kt_count, wave, lane, wm * TM, 0);
    opb.init(cur.b, 0, p.k, kt_count, wave, lane, wn * TN, kLdsB);

    // Every tile's first MFMA on a block takes srcC = 0: defining the accumulators is enough.
    floatx4 acc[FN][FM];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i) asm volatile("" : "=a"(acc[j][i]));

    half8 af[3][FM];
    half8 bf[3][FN];
    constexpr int NR = FM + FN;  // fragment reads per k step
    auto read_frag = [&](int buf, int stage, int ks, int r) {
        if (r == 0)
            bf[buf][0] = opb.read(smem, stage, ks, 0);
        else if (r <= FM)
            af[buf][r - 1] = opa.read(smem, stage, ks, r - 1);
        else
            bf[buf][r - FM] = opb.read(smem, stage, ks, r - FM);
    };
    // load i of K-tile u of the stream: K-tile u of this tile, or u - kt_count of the next
    auto load = [&](auto s_c, int u, int i) {
        constexpr int S = decltype(s_c)::value;
        const bool next = u >= kt_count;
        const int t = next ? u - kt_count : u;
        if (i < LA)
            opa.template load_tile<S>(smem, next ? nxt.a : cur.a, next ? nxt.a_bytes : cur.a_bytes, t, i);
        else
            opb.template load_tile<S>(smem, next ? nxt.b : cur.b, next ? nxt.b_bytes : cur.b_bytes, t, i - LA);
    };

    // This lane, computed where it is used and not held through the walk.
    auto lane_here = [] {
        int l;
        asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
        return l;
    };
    // The bias of the wave's columns from n0 on into half `half` of its place: 16 bytes a lane of
    // those that the columns fill (the others would write behind them), zeros past the last
    // column, and for all of them without a bias.
    const uint32_t bias_es = p.bias_f32 ? 4u : 2u;
    char *const bias_lds = smem + kLds + wave * 2 * kBias;
    auto load_bias_tile = [&](int half, int n0) {
        const uint32_t at = (uint32_t)lane_here() * 16u;
        if (at < (uint32_t)TN * bias_es)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                make_rsrc(p.bias ? p.bias : p.a, p.bias ? (uint32_t)p.n * bias_es : 0u),
                (__attribute__((address_space(3))) void *)(bias_lds + half * kBias), 16,
                (uint32_t)(n0 + wn * TN) * bias_es + at, 0, 0, 0);
    };

    // The finished tile: its first column, half of the bias's place, first element and bytes of its
    // rows in C, pre and the residual; and, where it leaves, their descriptors.
    struct Done {
        int n0, half;
        int64_t at;
        uint32_t bytes;
    };
    auto done_with = [&](const TileRows &t, int half) { return Done{t.n0, half, (int64_t)t.m0 * p.n, t.c_elems * 2u}; };
    struct Way {
        int n0, half;
        __amdgpu_buffer_rsrc_t c, pre, res;
    };
    auto way_of = [&](const Done &t) {
        return Way{t.n0, t.half, make_rsrc(static_cast<_Float16 *>(p.c) + t.at, t.bytes),
                   make_rsrc(p.pre ? p.pre + t.at : static_cast<_Float16 *>(p.c), p.pre ? t.bytes : 0u),
                   make_rsrc(RES ? static_cast<const _Float16 *>(p.residual) + t.at : p.a, RES ? t.bytes : 0u)};
    };
    // Lane l of unit (p, i): row 16 i + l % 16 of the wave's rows, columns 32 p + 8 (l / 16) .. + 7;
    // rows past M lie beyond the descriptors, chunks past N get an out-of-range offset.
    const uint32_t lane_off = (uint32_t)((wm * TM + (lane & 15)) * p.n + wn * TN + 8 * (lane >> 4)) * 2u;
    auto unit_off = [&](int u, int n0) {
        uint32_t lo = lane_off;
        asm volatile("" : "+v"(lo));  // (opaque: not held as U loop invariants)
        return (lo + (uint32_t)(16 * (u % FM) * p.n + n0 + 32 * (u / FM)) * 2u) |
               (n0 + wn * TN + 32 * (u / FM) + 8 * (lane_here() >> 4) < p.n ? 0u : kOutOfRange);
    };
    int4v res[RES ? kAhead : 1];
    float bias[8];
    auto load_res = [&](auto u_c, const Way &t) {
        constexpr int u = decltype(u_c)::value;
        if constexpr (RES && u < U) res[u % kAhead] = __builtin_amdgcn_raw_buffer_load_b128(t.res, unit_off(u, t.n0), 0, 0);
    };
    auto store_unit = [&](auto u_c, const Way &t) {
        constexpr int u = decltype(u_c)::value;
        constexpr int pp = u / FM, ii = u % FM;
        if constexpr (ii == 0) {
            // this p's bias: 8 columns of the lane, from LDS
            const char *from = bias_lds + t.half * kBias + (32 * pp + 8 * (lane_here() >> 4)) * bias_es;
            if (p.bias_f32) {
                const floatx4 x = *reinterpret_cast<const floatx4 *>(from), y = *reinterpret_cast<const floatx4 *>(from + 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) bias[e] = x[e], bias[4 + e] = y[e];
            } else {
                const half8 x = *reinterpret_cast<const half8 *>(from);
#pragma unroll
                for (int e = 0; e < 8; ++e) bias[e] = (float)x[e];
            }
        }
        // redefine the unit's accumulators here, so that their copies to VGPRs happen here
        asm volatile("" : "+a"(acc[2 * pp][ii]), "+a"(acc[2 * pp + 1][ii]));
        float z[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            z[e] = acc[2 * pp][ii][e] + bias[e];
            z[4 + e] = acc[2 * pp + 1][ii][e] + bias[4 + e];
        }
        const uint32_t off = unit_off(u, t.n0);
        auto round = [&] {
            half8 h;
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = (_Float16)z[e];  // nearest even
            return __builtin_bit_cast(int4v, h);
        };
        __builtin_amdgcn_raw_buffer_store_b128(round(), t.pre, off, 0, store_aux(POL));
        activate<8>(ACT, z);
        if constexpr (RES) {
            const half8 r = __builtin_bit_cast(half8, res[u % kAhead]);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] += (float)r[e];
        }
        __builtin_amdgcn_raw_buffer_store_b128(round(), t.c, off, 0, store_aux(POL));
        load_res(std::integral_constant<int, u + kAhead>{}, t);
    };

    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    using F = std::false_type;
    using T = std::true_type;
    constexpr int kRelAt = GEMM_AHEAD_REL_MFMA < NM ? GEMM_AHEAD_REL_MFMA : NM - 1;
    constexpr int kAcqAt = GEMM_AHEAD_ACQ_MFMA < NM ? GEMM_AHEAD_ACQ_MFMA : NM - 1;
    constexpr int L0 = L * GEMM_AHEAD_STEP0_LOADS / 16;  // loads of K-tile t+2 in step 0
    // Operations of a tile's first K-tile that go out after the loads of its second one, and may
    // be in flight when those are waited for: the units' two stores, the residual's loads and the
    // bias's, as far as the counter reaches.
    constexpr int kLeave = (RES ? 3 : 2) * U + L0 + 1 < 63 ? (RES ? 3 : 2) * U + L0 + 1 : 63;

    // Prologue: K-tiles 0 and 1 into stages 0 and 1; wait for K-tile 0; both steps' fragments of
    // K-tile 0 into buffers 0 and 1.
#pragma unroll
    for (int i = 0; i < L; ++i) load(S0{}, 0, i);
#pragma unroll
    for (int i = 0; i < L; ++i) load(S1{}, 1, i);
    vm_barrier<L>();
#pragma unroll
    for (int r = 0; r < NR; ++r) read_frag(0, 0, 0, r);
#pragma unroll
    for (int r = 0; r < NR; ++r) read_frag(1, 0, 1, r);

    // One K-tile.  FIRST: a tile's first: step 0 in unit order with srcC = 0, each unit of the
    // tile before leaving before it is overwritten.
    auto k_iter = [&](auto s_c, int t, auto first_c, const Done &ep) {
        constexpr int S = decltype(s_c)::value;
        constexpr bool FIRST = decltype(first_c)::value;
        constexpr int SN = S ^ 1;
        opa.refresh_lds();
        opb.refresh_lds();
        constexpr int B1 = S == 0 ? 1 : 2;   // this K-tile's step-1 buffer
        constexpr int NB1 = S == 0 ? 2 : 1;  // the next K-tile's
        const Way way = way_of(ep);
        if constexpr (FIRST) static_range<0, kAhead>([&](auto u_c) { load_res(u_c, way); });
        static_range<0, NM>([&](auto m_c) {
            constexpr int m = decltype(m_c)::value;
            if constexpr (FIRST) {
                constexpr int u = m / 2, j = 2 * (u / FM) + m % 2, i = u % FM;
                if constexpr (m % 2 == 0) store_unit(std::integral_constant<int, u>{}, way);
                mfma16_first(bf[0][j], af[0][i], acc[j][i]);
            } else {
                constexpr int j = m / FM, i = (j & 1) ? FM - 1 - m % FM : m % FM;
                mfma16_tied(bf[0][j], af[0][i], acc[j][i]);
            }
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
            if constexpr (m == kAcqAt) vm_only_barrier<FIRST ? kLeave : L0>();
            if constexpr (m >= kAcqAt) {
                constexpr int nl = L - L0, total = 2 * NR + nl, slots = NM - kAcqAt, q = m - kAcqAt;
                // R R L R R L ...: the reads first while both remain
                static_range<q * total / slots, (q + 1) * total / slots>([&](auto o_c) {
                    constexpr int o = decltype(o_c)::value;
                    constexpr int groups = (2 * NR) / 2 < nl ? (2 * NR) / 2 : nl;  // (R, R, L) groups
                    constexpr bool in_groups = o < 3 * groups;
                    constexpr bool is_read = in_groups ? (o % 3 != 2) : (2 * NR > 2 * groups);
                    constexpr int idx2 = in_groups ? (is_read ? (o / 3) * 2 + (o % 3) : o / 3)
                                                   : (is_read ? 2 * groups + (o - 3 * groups) : groups + (o - 3 * groups));
                    if constexpr (is_read) {
                        constexpr int ks = idx2 / NR, r = idx2 % NR;
                        read_frag(ks == 0 ? 0 : NB1, SN, ks, r);
                    } else {
                        load(s_c, t + 2, L0 + idx2);
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

    // Every tile runs the same code: the first one has a tile of no rows leave, the last one
    // reads the fragments of a tile past the grid, zeros.
    Done ep = done_with(tile_rows(ntiles), 1);
    int half = 0;
    for (;;) {
        load_bias_tile(half, cur.n0);
        k_iter(S0{}, 0, T{}, ep);
        k_iter(S1{}, 1, F{}, ep);
        for (int kt = 2; kt < kt_count; kt += 2) {
            k_iter(S0{}, kt, F{}, ep);
            k_iter(S1{}, kt + 1, F{}, ep);
        }
        ep = done_with(cur, half);
        if (idx + G >= ntiles) break;
        half ^= 1;
        cur = nxt;
        idx += G;
        nxt = tile_rows(idx + G);
    }
    // the last tile's units
    acc_fence(acc);
    const Way way = way_of(ep);
    static_range<0, kAhead>([&](auto u_c) { load_res(u_c, way); });
    static_range<0, U>([&](auto u_c) {
        store_unit(u_c, way);
        __builtin_amdgcn_sched_barrier(0);
    });
    // the last tile's loads past the tile (zeros into LDS) and its stores are done before the
    // workgroup ends
    __builtin_amdgcn_s_waitcnt(0);
#endif
}

// With a residual the kernels without an activation only (walk_takes in feedforward.hip).  Both in a
// unit's way out, walked and in fused_direct_kernel, us: 16384 x 4096 x 2048 silu 238 and 243, 8192 x
// 8192 x 4096 406 and 418, but 8192 x 4096 x 1024 gelu with pre 109 and 103, 16384 x 2048 x 512 gelu 76
// and 70.  2 to 5% of some sizes is little for 36 more of the largest kernels.
template <class C, int POL, bool KFULL>
hipError_t launch_walk(const FusedParams &p, int cus, hipStream_t s) {
    const void *kernel;
    switch (p.act) {
        case kActRelu: kernel = reinterpret_cast<const void *>(fused_walk_kernel<C, kActRelu, false, POL, KFULL>); break;
        case kActGelu: kernel = reinterpret_cast<const void *>(fused_walk_kernel<C, kActGelu, false, POL, KFULL>); break;
        case kActGeluTanh: kernel = reinterpret_cast<const void *>(fused_walk_kernel<C, kActGeluTanh, false, POL, KFULL>); break;
        case kActSilu: kernel = reinterpret_cast<const void *>(fused_walk_kernel<C, kActSilu, false, POL, KFULL>); break;
        default:
            kernel = p.residual ? reinterpret_cast<const void *>(fused_walk_kernel<C, kActNone, true, POL, KFULL>)
                                : reinterpret_cast<const void *>(fused_walk_kernel<C, kActNone, false, POL, KFULL>);
    }
    return launch_fused_grid(kernel, cus, 1, C::kThreads, s, p);
}

}  // namespace gemm_f16
