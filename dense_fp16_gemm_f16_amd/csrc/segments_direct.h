// Segmented products with operands loaded straight into LDS: 16-byte
// aligned rows (K, and N where B or A is read along it, multiples of 8).
#pragma once

#include "segments.h"

namespace gemm_f16 {

// A configuration whose columns are C's rows: the layout of TN's A.
template <class C>
struct RowsAsCols : C {
    static constexpr int BN = C::BM, FN = C::FM;
};

// Bytes of K-tile t of an operand with `cols` columns a row, from column n0
// of its first row to the last row inside the contraction (k_count rows);
// 0 past it.  No branch: this sits between the MFMAs.
template <class C>
__device__ __forceinline__ uint32_t nmajor_bytes(int k_count, int t, int cols, int n0) {
    const int rows = max(min(k_count - t * C::BK, C::BK), 0);  // rows * cols < 2^30
    return (uint32_t)max(rows * cols - n0, 0) * 2u;
}

// The segment of the given rank by falling size (equal sizes in order); more
// than 64 segments stay in order.
__device__ __forceinline__ int seg_by_size(const SegParams &p, int rank, int lane) {
    if (p.groups > kWave) return rank;
    int size = -1, mine = 0;
    if (lane < p.groups) size = max(seg_bound(p.offsets, lane + 1, p.rows) - seg_bound(p.offsets, lane, p.rows), 0);
    for (int g = 0; g < p.groups; ++g) {
        const int other = __builtin_amdgcn_readlane(size, g);
        mine += other > size || (other == size && g < lane);
    }
    const uint64_t hit = __ballot(lane < p.groups && mine == rank);
    return __builtin_ctzll(hit);
}

// A tile's place in the product and its operands' first rows.
template <int KIND, class C, bool LORA>
struct SegWork {
    int g, row0, valid, n0, k_count;  // k_count: length of the contraction
    int lo, split;                    // TN: its first row, its part
    bool live;

    // false: past the last tile
    __device__ __forceinline__ bool find(const SegParams &p, uint32_t pid, int lane) {
        live = true;
        if constexpr (KIND == kSegTN) {
            const uint32_t per = (uint32_t)p.num_m * (uint32_t)p.num_n;
            // long segments first, so that the last tiles to start are short
            g = seg_by_size(p, (int)(pid / per), lane);
            split = (int)blockIdx.y;
            const TileCoord tc = tile_coord<uint32_t>(pid % per, p.num_m, p.num_n, 4, true);
            row0 = (int)tc.m_block * C::BM;
            n0 = (int)tc.n_block * C::BN;
            valid = min(C::BM, p.k - row0);
            const SegPart part = seg_part(p, g, split, C::BK);
            lo = part.lo;
            k_count = part.count;
            return true;
        }
        TileCoord tc;
        if constexpr (LORA) {
            g = 0;
            tc = tile_coord<uint32_t>(pid, (p.rows + C::BM - 1) / C::BM, p.num_n, 4, true);
            row0 = (int)tc.m_block * C::BM;
            valid = min(C::BM, p.rows - row0);
        } else {
            SegMap<C::BM> map;
            map.init(p, lane);
            if (pid >= (uint32_t)map.total * (uint32_t)p.num_n) return false;
            tc = tile_coord<uint32_t>(pid, map.total, p.num_n, 4, true);
            const SegTile st = map.find(p, (int)tc.m_block, lane);
            g = st.g;
            row0 = st.row0;
            valid = st.valid;
            live = g < p.groups;
        }
        n0 = (int)tc.n_block * C::BN;
        k_count = live ? p.k : 0;
        return true;
    }
};

// LDS of seg_tile's operands, and behind it the votes of lora_tiles.
template <int KIND, class C>
constexpr int seg_tile_lds() {
    return 2 * C::BK * 2 * (C::BM + C::BN);
}

// One tile.  The K loop is gemm_f16_direct_ahead_kernel's: two LDS stages,
// both k steps' fragments of K-tile t+1 read during K-tile t, a release and
// an acquire barrier per K-tile.  smem: the kernel's one LDS array (with
// two, the compiler waits for every load in flight before each fragment
// read).
// C_g = A_g^T B_g of 16384 rows in 8 uneven segments, 2048 x 4096 in fp32: 260
// us (1055 TFLOP/s), bound as the walking kernel's products and by tiles of
// unlike lengths.  x W^T with adapters: see lora_tiles.
template <int KIND, class C, bool F32, bool LORA>
__device__ __forceinline__ void seg_tile(const SegParams &p, char *smem, const SegWork<KIND, C, LORA> &w, int tid) {
    constexpr int TM = C::TM, TN = C::TN, FM = C::FM, FN = C::FN;
    static_assert(C::MB == 16 && C::KS == 2, "two 32-wide k steps per K-tile");
    using OpA = std::conditional_t<KIND == kSegTN, NMajorDirect<RowsAsCols<C>, true>, KMajorDirect<C, C::BM, false>>;
    using OpB = std::conditional_t<KIND == kSegNT, KMajorDirect<C, C::BN, false>, NMajorDirect<C, true>>;
    constexpr int kLdsB = OpA::kLdsBytes, kLds = OpA::kLdsBytes + OpB::kLdsBytes;
    constexpr int LA = OpA::kLoads, L = OpA::kLoads + OpB::kLoads;
    static_assert(kLds == seg_tile_lds<KIND, C>(), "LDS of the operands");
    static_assert(2 * L < 64, "vmcnt range");
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int kt_count = (w.k_count + C::BK - 1) / C::BK;

    OpA opa;
    OpB opb;
    const _Float16 *a_tile = p.a, *b_tile = p.b;  // operands read along N: the tile's first element
    if constexpr (KIND == kSegTN) {
        a_tile = p.a + (int64_t)w.lo * p.k + w.row0;
        b_tile = p.b + (int64_t)w.lo * p.n + w.n0;
        opa.init(p.a, 0, p.k, w.k_count, kt_count, wave, lane, wm * TM, 0);
        opb.init(p.b, 0, p.n, w.k_count, kt_count, wave, lane, wn * TN, kLdsB);
    } else {
        const int32_t *from = LORA ? p.order : p.index;
        if (from) {
            // gathered rows: the descriptor spans A (below 2 GiB), each lane's
            // rows start where the index says
            opa.init(p.a, (int)p.a_rows, p.k, kt_count, wave, lane, wm * TM, 0);
#pragma unroll
            for (int i = 0; i < OpA::kLoads; ++i) {
                const int r = (i * C::kWaves + wave) * 8 + (lane >> 3);
                uint32_t off = kOutOfRange;
                if (w.live && r < w.valid) {
                    const int v = from[w.row0 + r];
                    const int64_t src = v < 0 ? -1 : LORA ? v : v / p.fan;
                    if (src >= 0 && src < p.a_rows) off = (uint32_t)((src * p.k + opa.kc) * 2);
                }
                opa.voff[i] = off;
            }
        } else {
            opa.init(p.a + (int64_t)w.row0 * p.k, w.valid, p.k, kt_count, wave, lane, wm * TM, 0);
        }
        const _Float16 *b = p.b + (int64_t)(w.live ? w.g : 0) * p.n * p.k;
        if constexpr (KIND == kSegNT)
            opb.init(b + (int64_t)w.n0 * p.k, min(C::BN, p.n - w.n0), p.k, kt_count, wave, lane, wn * TN, kLdsB);
        else
            opb.init(p.b, 0, p.n, p.k, kt_count, wave, lane, wn * TN, kLdsB);
        b_tile = b + w.n0;
    }

    // the first adapter of the tile: its offsets arrive under the K loop
    LoraWalk walk;
    if constexpr (LORA) walk.next(p, w.row0, w.valid, lane);

    floatx4 acc[FN][FM];
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
        if (i < LA) {
            if constexpr (KIND == kSegTN)
                opa.template load_tile<S>(smem, a_tile, w.row0, nmajor_bytes<C>(w.k_count, t, p.k, w.row0), t, i);
            else
                opa.template load<S>(smem, t, i);
        } else {
            if constexpr (KIND == kSegNT)
                opb.template load<S>(smem, t, i - LA);
            else
                opb.template load_tile<S>(smem, b_tile, w.n0, nmajor_bytes<C>(w.k_count, t, p.n, w.n0), t, i - LA);
        }
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    constexpr int NM = FM * FN;
    constexpr int kRelAt = GEMM_AHEAD_REL_MFMA < NM ? GEMM_AHEAD_REL_MFMA : NM - 1;
    constexpr int kAcqAt = GEMM_AHEAD_ACQ_MFMA < NM ? GEMM_AHEAD_ACQ_MFMA : NM - 1;
    constexpr int L0 = L * GEMM_AHEAD_STEP0_LOADS / 16;  // loads of K-tile t+2 in step 0

    if (kt_count > 0) {
#pragma unroll
        for (int i = 0; i < L; ++i) load(S0{}, 0, i);
#pragma unroll
        for (int i = 0; i < L; ++i) load(S1{}, 1, i);
    }
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
    int kt = 0;
    for (; kt + 1 < kt_count; kt += 2) {
        k_iter(S0{}, kt);
        k_iter(S1{}, kt + 1);
    }
    if (kt < kt_count) k_iter(S0{}, kt);

    vm_barrier<0>();  // no load is still writing LDS when C is staged there
    acc_fence(acc);

    // opaque copies: what hangs on them is computed here, not held in
    // registers through the K loop
    int t = tid, row0 = w.row0, n0 = w.n0, valid = w.valid;
    asm volatile("" : "+v"(t), "+s"(row0), "+s"(n0), "+s"(valid));
    const int l = t & (kWave - 1);
    constexpr int kWaveBytes = kLds / C::kWaves;
    char *const stg = smem + wave * kWaveBytes;
    lds_barrier();
    if constexpr (LORA) {
        const bool wild =
            lora_tiles<C, true>(acc, smem, reinterpret_cast<int *>(smem + kLds), p, walk, row0, valid, n0, t, l, wm, wn);
        const int32_t *order = p.order;
        const int rows = p.rows;
        seg_store<C, F32, kWaveBytes>(acc, stg, p.c, valid, p.n, n0, wm, wn, l,
                                      [&](int r) { return min(max(order[row0 + r], 0), rows - 1); });
        if (wild) lora_wild<C>(p, row0, valid, n0, t, l);
    } else {
        using Out = std::conditional_t<F32, float, _Float16>;
        Out *c = static_cast<Out *>(p.c) + (KIND == kSegTN ? w.split * p.part_elems + (int64_t)w.g * p.k * p.n : 0);
        seg_store<C, F32, kWaveBytes>(acc, stg, c, valid, p.n, n0, wm, wn, l, [&](int r) { return row0 + r; });
    }
}

// One workgroup per tile.
template <int KIND, class C, bool F32, bool LORA>
__global__ __launch_bounds__(C::kThreads)
__attribute__((amdgpu_waves_per_eu(C::kMinWavesPerEU, C::kMinWavesPerEU)))
void seg_tile_kernel(const SegParams p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the signature only
    constexpr int kOps = seg_tile_lds<KIND, C>(), kLds = LORA ? lora_lds<C>() : kOps;
    static_assert(kLds <= 160 * 1024 && (!LORA || kOps + C::kWaves * 4 <= kLds), "LDS budget");
    __shared__ __attribute__((aligned(1024))) char smem[kLds];
    GEMM_POISON_LDS(smem);
    SegWork<KIND, C, LORA> w;
    if (!w.find(p, seg_pid(p), (int)threadIdx.x & (kWave - 1))) return;
    seg_tile<KIND, C, F32, LORA>(p, smem, w, (int)threadIdx.x);
#endif
}

// Small tiles, where the operands' bytes bound the product: one workgroup
// per tile, a ring of S LDS stages loaded S - 1 K-tiles ahead, one barrier
// per K-tile (before it, every wave has read the stage that the next load
// fills, and has waited for its own loads of the next K-tile).  Two stages
// leave a CU waiting for memory most of the time here; the ring keeps S - 1
// K-tiles in flight.  KG 2: twice the waves, each half of them with a ring of
// its own over half of K, the halves' sums meeting in LDS: for grids that
// leave CUs with one workgroup or none.
// DOWN: h of the adapters, times their scale, in parts (4096 rows, K 4096, 8
// adapters of rank 64: 16 us, 33 MB of x at 2.1 TB/s, bound by how long 128-byte
// pieces of rows take to come; 32 x 32 tiles, which read x twice: 25 us).
template <int KIND, class C, int S, int KG, bool F32, bool DOWN>
__global__ __launch_bounds__(C::kThreads *KG) void seg_ring_kernel(const SegParams p) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the signature only
    constexpr int TM = C::TM, TN = C::TN, FM = C::FM, FN = C::FN;
    using OpA = KMajorDirect<C, C::BM, false>;
    using OpB = std::conditional_t<KIND == kSegNT, KMajorDirect<C, C::BN, false>, NMajorDirect<C, true>>;
    constexpr int kStage = OpA::kStage + OpB::kStage;
    constexpr int LA = OpA::kLoads, L = OpA::kLoads + OpB::kLoads;
    constexpr int kRing = S * kStage, kLds = KG * kRing;
    static_assert(kLds <= 160 * 1024 && S >= 3 && (S - 1) * L < 64, "LDS budget, vmcnt range");
    __shared__ __attribute__((aligned(1024))) char smem[kLds];
    GEMM_POISON_LDS(smem);

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int group = __builtin_amdgcn_readfirstlane(tid / C::kThreads);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave) - group * C::kWaves;
    char *const ring = smem + group * kRing;
    const int wm = wave / C::WN, wn = wave % C::WN;
    SegWork<KIND, C, false> w;
    if (!w.find(p, seg_pid(p), lane)) return;
    // this group's K-tiles: `turns` for every group, those past kt1 zeros
    const int kt_count = (w.k_count + C::BK - 1) / C::BK, turns = (kt_count + KG - 1) / KG;
    const int kt0 = group * turns, kt1 = min(kt0 + turns, kt_count);
    // Where this workgroup starts in them: rows a power of two apart put one
    // K-tile of every row on the same memory channels, so workgroups in step
    // would all wait for those.
    const int shift = turns > 0 ? (int)((blockIdx.x * 5u) % (uint32_t)turns) : 0;

    OpA opa;
    OpB opb;
    if (p.index) {
        opa.init(p.a, (int)p.a_rows, p.k, kt1, wave, lane, wm * TM, 0);
#pragma unroll
        for (int i = 0; i < OpA::kLoads; ++i) {
            const int r = (i * C::kWaves + wave) * 8 + (lane >> 3);
            uint32_t off = kOutOfRange;
            if (w.live && r < w.valid) {
                const int v = p.index[w.row0 + r];
                const int64_t src = v < 0 ? -1 : v / p.fan;
                if (src >= 0 && src < p.a_rows) off = (uint32_t)((src * p.k + opa.kc) * 2);
            }
            opa.voff[i] = off;
        }
    } else {
        opa.init(p.a + (int64_t)w.row0 * p.k, w.valid, p.k, kt1, wave, lane, wm * TM, 0);
    }
    const _Float16 *b = p.b + (int64_t)(w.live ? w.g : 0) * p.n * p.k;
    if constexpr (KIND == kSegNT)
        opb.init(b + (int64_t)w.n0 * p.k, max(min(C::BN, p.n - w.n0), 0), p.k, kt1, wave, lane, wn * TN, OpA::kStage);
    else
        opb.init(p.b, 0, p.n, p.k, kt1, wave, lane, wn * TN, OpA::kStage);

    floatx4 acc[FN][FM];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i) acc[j][i] = floatx4{};
    auto load = [&](int turn, int stage) {  // past the last turn: empty loads, for the count
        char *to = ring + stage * kStage;
        const int at = turn + shift < turns ? turn + shift : turn + shift - turns;
        const int t = turn < turns ? kt0 + at : kt1;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if (i < LA)
                opa.template load<0>(to, t, i);
            else if constexpr (KIND == kSegNT)
                opb.template load<0>(to, t, i - LA);
            else
                opb.template load_tile<0>(to, b + w.n0, w.n0, nmajor_bytes<C>(min(w.k_count, kt1 * C::BK), t, p.n, w.n0), t, i - LA);
        }
    };
    if (turns > 0) {
#pragma unroll
        for (int s = 0; s < S - 1; ++s) load(s, s);
        int stage = 0;
        for (int t = 0; t < turns; ++t) {
            vm_barrier<(S - 2) * L>();
            load(t + S - 1, stage == 0 ? S - 1 : stage - 1);
            const char *from = ring + stage * kStage;
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
        }
    }
    vm_barrier<0>();  // no load is still writing LDS when C is staged there
    if constexpr (KG == 2) {
        static_assert(C::kThreads * FN * FM * 16 <= kRing, "the second half's sums");
        floatx4 *const sums = reinterpret_cast<floatx4 *>(smem) + (tid - group * C::kThreads);
        if (group == 1) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int i = 0; i < FM; ++i) sums[(j * FM + i) * C::kThreads] = acc[j][i];
        }
        lds_barrier();
        if (group == 0) {
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int i = 0; i < FM; ++i) acc[j][i] += sums[(j * FM + i) * C::kThreads];
        }
        lds_barrier();
        if (group == 1) return;
    }

    constexpr int kWaveBytes = kLds / C::kWaves / 1024 * 1024;
    char *const stg = smem + wave * kWaveBytes;
    const int row0 = w.row0;
    if constexpr (DOWN) {
        const float f = w.live && p.scale ? p.scale[w.g] : 1.0f;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int r = wm * TM + 16 * i + lane % 16;
            if (r >= w.valid) continue;
            char *row = static_cast<char *>(p.c) + (int64_t)(row0 + r) * p.h_ld * kSplitValue;
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int n = w.n0 + wn * TN + 16 * j + 4 * (lane / 16);
                if (n < p.h_ld) store_split(row, n, acc[j][i], f, p.rank);
            }
        }
    } else {
        seg_store<C, F32, kWaveBytes>(acc, stg, p.c, w.valid, p.n, w.n0, wm, wn, lane, [&](int r) { return row0 + r; });
    }
#endif
}

template <int KIND, class C, int S, int KG>
hipError_t launch_seg_ring(SegParams p, bool f32, hipStream_t s) {
    p.num_n = (p.n + C::BN - 1) / C::BN;
    p.num_m = (int32_t)seg_row_tiles(p.rows, p.groups, C::BM);
    const int64_t grid = (int64_t)p.num_m * p.num_n;
    return f32 ? launch_seg(seg_ring_kernel<KIND, C, S, KG, true, false>, grid, C::kThreads * KG, s, p)
               : launch_seg(seg_ring_kernel<KIND, C, S, KG, false, false>, grid, C::kThreads * KG, s, p);
}

// Launch of tile C: the grid holds every tile that any sizes could need.
template <int KIND, class C, bool LORA = false>
hipError_t launch_seg_tile(SegParams p, bool f32, hipStream_t s) {
    p.num_n = (p.n + C::BN - 1) / C::BN;
    int64_t grid;
    if constexpr (KIND == kSegTN) {
        p.num_m = (p.k + C::BM - 1) / C::BM;
        grid = (int64_t)p.groups * p.num_m * p.num_n;
    } else {
        const int64_t m_tiles = LORA ? (p.rows + C::BM - 1) / C::BM : seg_row_tiles(p.rows, p.groups, C::BM);
        p.num_m = (int32_t)m_tiles;
        grid = m_tiles * p.num_n;
    }
    const int parts = KIND == kSegTN ? p.splits : 1;
    if constexpr (LORA)
        return launch_seg(seg_tile_kernel<KIND, C, false, LORA>, grid, C::kThreads, s, p);
    else
        return f32 ? launch_seg(seg_tile_kernel<KIND, C, true, LORA>, grid, C::kThreads, s, p, parts)
                   : launch_seg(seg_tile_kernel<KIND, C, false, LORA>, grid, C::kThreads, s, p, parts);
}

}  // namespace gemm_f16
