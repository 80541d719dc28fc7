// Segmented products with more tiles than CUs: one workgroup per CU walks
// its tiles without a pause between them.
#pragma once

#include "segments_direct.h"

namespace gemm_f16 {

struct WalkTile {
    int g, row0, valid, n0;  // as SegWork
    int k_count, kt;         // contraction length; K-tiles, even
    int unused[2];
};

using TailCfg = Cfg<128, 128, 2, 2, 16>;
using HalfCfg = Cfg<128, 256, 2, 2, 16>;

// As gemm_f16_stream_kernel: the K-tile stream runs on across tiles (the
// last two K-tiles of a tile load the next tile's first two), and a tile's C
// leaves from the accumulators under the next tile's first MFMAs.  What
// differs:
//  * the tiles are listed up front in LDS, with the gathered rows' offsets:
//    a load of offsets or indices inside the K loop would wait, in order,
//    for every operand load before it;
//  * rows behind the last segment take two K-tiles of zeros;
//  * a last round that would leave half the CUs idle is cut into 128 x 128
//    tiles, or halves of a 256 x 256 tile, one per workgroup;
//  * fp16 results: v_permlane16_swap joins two blocks' 8-byte quarters into
//    16-byte stores, so no operand layout is bent for the stores; fp32
//    results leave a block at a time.
// Bound by the MFMAs at the clock that the power limit leaves: 16384 rows in
// 8 uneven segments, 4096 x 2048, take 240-253 us (1090-1145 TFLOP/s), in equal
// segments 196, as long as the dense kernel; the rest is half a row tile lost
// per segment and a last round that does not fill the CUs.
template <int KIND, class C, bool F32, int POL>
__global__ __launch_bounds__(C::kThreads)
__attribute__((amdgpu_waves_per_eu(C::kMinWavesPerEU, C::kMinWavesPerEU)))
void seg_walk_kernel(const SegParams p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the signature only
    constexpr int TM = C::TM, TN = C::TN, FM = C::FM, FN = C::FN;
    static_assert(C::MB == 16 && C::KS == 2 && FN % 2 == 0, "two 32-wide k steps per K-tile, blocks in pairs");
    static_assert(KIND != kSegTN, "segments of unlike lengths leave a fixed walk unbalanced");
    using OpA = KMajorDirect<C, C::BM, false>;
    using OpB = std::conditional_t<KIND == kSegNT, KMajorDirect<C, C::BN, false>, NMajorDirect<C, true>>;
    constexpr int kLdsB = OpA::kLdsBytes, kLds = OpA::kLdsBytes + OpB::kLdsBytes;
    constexpr int LA = OpA::kLoads, L = OpA::kLoads + OpB::kLoads;
    constexpr int kList = kLds, kRows = kList + kWalkTiles * (int)sizeof(WalkTile);
    constexpr int kAll = kRows + (KIND == kSegNT ? kWalkTiles * C::BM * 4 : 0);
    constexpr bool kLarge = C::BM == 256 && C::BN == 256;
    static_assert(seg_tile_lds<KIND, TailCfg>() <= kAll && (!kLarge || seg_tile_lds<KIND, HalfCfg>() <= kAll),
                  "LDS of the last round's tiles");
    constexpr int NM = FM * FN;            // MFMAs per k step
    constexpr int U = F32 ? NM : NM / 2;   // 16-byte store units per wave and tile
    constexpr int ES = F32 ? 4 : 2;
    static_assert(kAll <= 160 * 1024, "LDS budget");
    // one LDS array, as in seg_tile_kernel
    __shared__ __attribute__((aligned(1024))) char smem[kAll];
    GEMM_POISON_LDS(smem);

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int G = (int)gridDim.x;

    // ---- this workgroup's tiles --------------------------------------------
    int count = 0;
    SegMap<C::BM> map;
    int total, whole = 0, parts = 0;  // parts: small tiles that a tile of the last round is cut into
    map.init(p, lane);
    total = whole = map.total * p.num_n;
    const int rest = total % G;
    // One takes 0.42 (a quarter) or 0.5 (half) of a 256 x 256 tile's time,
    // 0.66 (half) of a 256 x 128's (16384 rows, 8 segments, 4096 x 2048, 80 tiles
    // in the last round: 229 us in two rounds of quarters, 220 in halves).
    parts = kLarge && rest * 4 <= G ? 4 : rest * 2 <= G ? 2 : 0;
    if (parts > 0) whole = total - rest;
    for (int round = 0; round * G < whole && count < kWalkTiles; ++round) {
        const int pid = round * G + (int)blockIdx.x;
        if (pid >= whole) break;
        const int slot = count++;
        if (slot % C::kWaves != wave) continue;
        const TileCoord tc = tile_coord<uint32_t>(pid, map.total, p.num_n, 4, true);
        const SegTile st = map.find(p, (int)tc.m_block, lane);
        WalkTile w = {};
        w.g = st.g;
        w.row0 = st.row0;
        w.valid = st.valid;
        w.n0 = (int)tc.n_block * C::BN;
        w.k_count = st.g < p.groups ? p.k : 0;
        // an empty contraction still takes a pair of K-tiles, of zeros
        w.kt = max(2, ((w.k_count + C::BK - 1) / C::BK + 1) & ~1);
        if (KIND == kSegNT && p.index) {
            uint32_t *const rows = reinterpret_cast<uint32_t *>(smem + kRows) + slot * C::BM;
            for (int r = lane; r < C::BM; r += kWave) {
                uint32_t off = kOutOfRange;
                if (r < w.valid && w.k_count) {
                    const int v = p.index[w.row0 + r];
                    const int64_t src = v < 0 ? -1 : v / p.fan;
                    if (src >= 0 && src < p.a_rows) off = (uint32_t)(src * p.k * 2);
                }
                rows[r] = off;
            }
        }
        if (lane == 0) reinterpret_cast<WalkTile *>(smem + kList)[slot] = w;
    }
    __syncthreads();
    if (count > 0) {
        auto tile = [&](int i) {
            const int4v *q = reinterpret_cast<const int4v *>(smem + kList + i * (int)sizeof(WalkTile));
            const int4v u = q[0], v = q[1];
            auto s = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
            return WalkTile{s(u[0]), s(u[1]), s(u[2]), s(u[3]), s(v[0]), s(v[1]), {0, 0}};
        };

        // ---- operands -----------------------------------------------------------
        OpA opa;
        OpB opb;
        const bool gather = KIND == kSegNT && p.index != nullptr;
        // where the loads are: a tile of their own, ahead of the MFMAs' one
        const _Float16 *la = p.a, *lb = p.b;
        uint32_t la_bytes = 0, lb_bytes = 0;
        int ln0 = 0, l_count = 0;
        opa.init(p.a, 0, p.k, 2, wave, lane, wm * TM, 0);
        if constexpr (KIND == kSegNT)
            opb.init(p.b, 0, p.k, 2, wave, lane, wn * TN, kLdsB);
        else
            opb.init(p.b, 0, p.n, p.k, 2, wave, lane, wn * TN, kLdsB);
        auto uptr = [](const _Float16 *q) {
            const uint64_t v = (uint64_t)(uintptr_t)q;
            const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
            return (const _Float16 *)(uintptr_t)(((uint64_t)hi << 32) | lo);
        };
        // The loads' next tile; past the last one they read zeros.  (Each variable
        // is set once, with no branch around it: the compiler then keeps them all
        // in scalar registers, where branches left some in scratch memory.)
        auto aim = [&](int i) {
            const WalkTile w = tile(min(i, count - 1));
            const bool live = i < count && w.k_count > 0;
            ln0 = w.n0;
            l_count = live ? w.k_count : 0;
            const int64_t row0 = gather ? 0 : w.row0, rows = gather ? p.a_rows : w.valid;
            la = uptr(p.a + row0 * p.k);
            la_bytes = live ? (uint32_t)rows * (uint32_t)p.k * 2u : 0u;
            const _Float16 *b = p.b + (int64_t)(live ? w.g : 0) * p.n * p.k;
            if constexpr (KIND == kSegNT) {
                if (gather) {
                    const uint32_t *const r = reinterpret_cast<const uint32_t *>(smem + kRows) + min(i, count - 1) * C::BM;
#pragma unroll
                    for (int q = 0; q < OpA::kLoads; ++q)
                        opa.voff[q] = r[(q * C::kWaves + wave) * 8 + (lane >> 3)] + (uint32_t)opa.kc * 2u;
                }
                lb = uptr(b + (int64_t)w.n0 * p.k);
                lb_bytes = live ? (uint32_t)min(C::BN, p.n - w.n0) * (uint32_t)p.k * 2u : 0u;
            } else {
                lb = uptr(b + w.n0);
            }
        };
        auto load = [&](auto s_c, int t, int i) {
            constexpr int S = decltype(s_c)::value;
            if (i < LA) {
                opa.template load_tile<S>(smem, la, la_bytes, t, i);
            } else {
                if constexpr (KIND == kSegNT)
                    opb.template load_tile<S>(smem, lb, lb_bytes, t, i - LA);
                else
                    opb.template load_tile<S>(smem, lb, ln0, nmajor_bytes<C>(l_count, t, p.n, ln0), t, i - LA);
            }
        };

        // every tile's first MFMA on a block takes srcC = 0: defining the
        // accumulators is enough
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

        // ---- stores ---------------------------------------------------------------
        // Unit u: fp32, block (u / FM, u % FM); fp16, blocks (2 p, i), (2 p + 1, i)
        // with p = u / FM, i = u % FM.  A lane of block (j, i) holds row 16 i +
        // l % 16 and columns 16 j + 4 (l / 16) .. + 3; after the swaps of a pair
        // it holds 8 columns from 32 p + 16 (l / 16 % 2) + 8 (l / 32) on.
        const int q4 = lane >> 4;
        const int col_l = wn * TN + (F32 ? 4 * q4 : 16 * (q4 & 1) + 8 * (q4 >> 1));
        const uint32_t lane_off = (uint32_t)((wm * TM + (lane & 15)) * p.n + col_l) * (uint32_t)ES;
        auto store_unit = [&](auto u_c, int n0, __amdgpu_buffer_rsrc_t rc) {
            constexpr int u = decltype(u_c)::value;
            constexpr int pp = u / FM, ii = u % FM;
            int4v v;
            if constexpr (F32) {
                asm volatile("" : "+a"(acc[pp][ii]));
                v = __builtin_bit_cast(int4v, acc[pp][ii]);
            } else {
                // redefined here, so that their copies to VGPRs happen here
                asm volatile("" : "+a"(acc[2 * pp][ii]), "+a"(acc[2 * pp + 1][ii]));
                half4 x, y;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = (_Float16)acc[2 * pp][ii][e];  // round to nearest even
                    y[e] = (_Float16)acc[2 * pp + 1][ii][e];
                }
                typedef unsigned uint2v __attribute__((ext_vector_type(2)));
                const uint2v xu = __builtin_bit_cast(uint2v, x), yu = __builtin_bit_cast(uint2v, y);
                const auto s0 = __builtin_amdgcn_permlane16_swap(xu[0], yu[0], false, false);
                const auto s1 = __builtin_amdgcn_permlane16_swap(xu[1], yu[1], false, false);
                v = int4v{(int)s0[0], (int)s1[0], (int)s0[1], (int)s1[1]};
            }
            // opaque copies: the offsets are computed here, not held for U units
            uint32_t lo = lane_off;
            int cl = col_l;
            asm volatile("" : "+v"(lo), "+v"(cl));
            constexpr int cols = F32 ? 16 : 32;
            const uint32_t off = (lo + (uint32_t)(16 * ii * p.n + n0 + cols * pp) * (uint32_t)ES) |
                                 (n0 + cl + cols * pp < p.n ? 0u : kOutOfRange);
            __builtin_amdgcn_raw_buffer_store_b128(v, rc, off, 0, store_aux(POL));
        };
        auto c_rsrc = [&](const WalkTile &w) {
            return make_rsrc(static_cast<char *>(p.c) + (int64_t)w.row0 * p.n * ES, (uint32_t)w.valid * (uint32_t)p.n * (uint32_t)ES);
        };

        // ---- the K-tile stream ----------------------------------------------------
        using S0 = std::integral_constant<int, 0>;
        using S1 = std::integral_constant<int, 1>;
        using F = std::false_type;
        using T = std::true_type;
        constexpr int kRelAt = GEMM_AHEAD_REL_MFMA < NM ? GEMM_AHEAD_REL_MFMA : NM - 1;
        constexpr int kAcqAt = GEMM_AHEAD_ACQ_MFMA < NM ? GEMM_AHEAD_ACQ_MFMA : NM - 1;
        constexpr int L0 = L * GEMM_AHEAD_STEP0_LOADS / 16;  // loads of K-tile t+2 in step 0
        // the waits' counter holds 63: past that, some stores are waited for too
        constexpr int kLeave = U + L0 < 63 ? U + L0 : 63;
        static_assert(2 * L < 64, "vmcnt range");

        aim(0);
#pragma unroll
        for (int i = 0; i < L; ++i) load(S0{}, 0, i);
#pragma unroll
        for (int i = 0; i < L; ++i) load(S1{}, 1, i);
        vm_barrier<L>();
#pragma unroll
        for (int r = 0; r < NR; ++r) read_frag(0, 0, 0, r);
#pragma unroll
        for (int r = 0; r < NR; ++r) read_frag(1, 0, 1, r);

        // One K-tile on stage S, which loads K-tile t of the loads' tile into it.
        // FIRST: a tile's first K-tile, its step 0 in unit order with srcC = 0,
        // each unit of the previous tile stored right before it is overwritten.
        auto k_iter = [&](auto s_c, int t, auto first_c, int st_n0, __amdgpu_buffer_rsrc_t rc) {
            constexpr int S = decltype(s_c)::value;
            constexpr bool FIRST = decltype(first_c)::value;
            constexpr int SN = S ^ 1;
            opa.refresh_lds();
            opb.refresh_lds();
            constexpr int B1 = S == 0 ? 1 : 2;   // this K-tile's step-1 buffer
            constexpr int NB1 = S == 0 ? 2 : 1;  // the next K-tile's
            static_range<0, NM>([&](auto m_c) {
                constexpr int m = decltype(m_c)::value;
                if constexpr (FIRST) {
                    constexpr int per = NM / U;
                    constexpr int u = m / per, j = per * (u / FM) + m % per, i = u % FM;
                    if constexpr (m % per == 0) store_unit(std::integral_constant<int, u>{}, st_n0, rc);
                    mfma16_first(bf[0][j], af[0][i], acc[j][i]);
                } else {
                    constexpr int j = m / FM, i = (j & 1) ? FM - 1 - m % FM : m % FM;
                    mfma16_tied(bf[0][j], af[0][i], acc[j][i]);
                }
                if constexpr (m == kRelAt) lgkm_barrier();
                if constexpr (m >= kRelAt) {
                    constexpr int q = m - kRelAt, slots = NM - kRelAt;
                    static_range<q * L0 / slots, (q + 1) * L0 / slots>(
                        [&](auto o_c) { load(s_c, t, decltype(o_c)::value); });
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
                // the next K-tile is in LDS; after its loads went out L0 of this
                // K-tile's and, in a tile's first one, the U stores
                if constexpr (m == kAcqAt) vm_only_barrier<FIRST ? kLeave : L0>();
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
                            load(s_c, t, L0 + idx);
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

        // Every tile runs the same code: the first one stores the units of a
        // tile of no rows, and the last one loads a tile of zeros.
        WalkTile cur = tile(0);
        int st_n0 = 0;
        __amdgpu_buffer_rsrc_t rc = make_rsrc(p.c, 0u);
        int lt = 2;  // K-tile that the loads are at
        for (int at = 0;; ++at) {
            if (cur.kt == 2) {
                aim(at + 1);
                lt = 0;
            }
            k_iter(S0{}, lt, T{}, st_n0, rc);
            k_iter(S1{}, lt + 1, F{}, st_n0, rc);
            lt += 2;
            for (int kt = 2; kt < cur.kt; kt += 2) {
                if (kt + 2 == cur.kt) {
                    aim(at + 1);
                    lt = 0;
                }
                k_iter(S0{}, lt, F{}, st_n0, rc);
                k_iter(S1{}, lt + 1, F{}, st_n0, rc);
                lt += 2;
            }
            st_n0 = cur.n0;
            rc = c_rsrc(cur);
            if (at + 1 >= count) break;
            cur = tile(at + 1);
        }
        acc_fence(acc);
        static_range<0, U>([&](auto u_c) {
            store_unit(u_c, st_n0, rc);
            __builtin_amdgcn_sched_barrier(0);
        });
        // the loads past the last tile (zeros into LDS) and its stores are done
        // before the workgroup ends
        __builtin_amdgcn_s_waitcnt(0);
    }
    // at most one small tile per workgroup
    auto small = [&](auto cfg) {
        using T = decltype(cfg);
        constexpr int kCols = C::BN / T::BN, kParts = C::BM / T::BM * kCols;
        const int at = (int)blockIdx.x;
        __syncthreads();  // every wave is done with the stages
        SegWork<KIND, T, false> w;
        const TileCoord tc = tile_coord<uint32_t>((uint32_t)(whole + at / kParts), map.total, p.num_n, 4, true);
        const SegTile st = map.find(p, (int)tc.m_block, lane);
        const int sm = at % kParts / kCols * T::BM;
        w.g = st.g;
        w.row0 = st.row0 + sm;
        w.valid = min(st.valid - sm, T::BM);
        w.n0 = (int)tc.n_block * C::BN + at % kCols * T::BN;
        w.live = st.g < p.groups;
        w.k_count = w.live ? p.k : 0;
        if (w.valid > 0 && w.n0 < p.n) seg_tile<KIND, T, F32, false>(p, smem, w, tid);
    };
    if ((int)blockIdx.x < (total - whole) * parts) {
        if constexpr (kLarge) {
            if (parts == 4)
                small(TailCfg{});
            else
                small(HalfCfg{});
        } else {
            small(TailCfg{});
        }
    }
#endif
}

template <int KIND, class C>
hipError_t launch_seg_walk(SegParams p, bool f32, bool device_stores, int cus, hipStream_t s) {
    p.num_n = (p.n + C::BN - 1) / C::BN;
    p.num_m = (int32_t)seg_row_tiles(p.rows, p.groups, C::BM);
    const int64_t tiles = (int64_t)p.num_m * p.num_n;
    const int64_t grid = tiles < cus ? tiles : cus;
    if (tiles > grid * kWalkTiles) return hipErrorInvalidValue;
    if (device_stores)
        return f32 ? launch_seg(seg_walk_kernel<KIND, C, true, kStoreDevice>, grid, C::kThreads, s, p)
                   : launch_seg(seg_walk_kernel<KIND, C, false, kStoreDevice>, grid, C::kThreads, s, p);
    return f32 ? launch_seg(seg_walk_kernel<KIND, C, true, kStoreStream>, grid, C::kThreads, s, p)
               : launch_seg(seg_walk_kernel<KIND, C, false, kStoreStream>, grid, C::kThreads, s, p);
}

}  // namespace gemm_f16
