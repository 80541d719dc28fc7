// Segmented products for gfx950: matrix products whose rows fall into
// consecutive segments ("groups") of ragged sizes that only the GPU knows.
//
//   NT  C[r] = A[src(r)] B_g^T   r in segment g, B_g [N,K]   (forward)
//   NN  C[r] = A[r] B_g          r in segment g, B_g [K,N]   (data gradient)
//   TN  C_g  = A_g^T B_g         A_g, B_g the rows of segment g: [K,N] (weight gradient)
//
// Segment g holds rows offsets[g] .. offsets[g+1]-1.  The offsets are read
// by the kernels: every workgroup scans them, finds the tile it owns, and
// those past the last tile leave.  Offsets are clamped to [0, rows] and
// gathered rows to A, so no content of them leads to an access out of
// range; rows behind the last segment come out as zeros.
//
// The building blocks (LDS layouts, fragment reads, C staging) are those of
// kernels.h.
#pragma once

#include <algorithm>

#include "kernels.h"

namespace gemm_f16 {

enum SegKind : int { kSegNT = 0, kSegNN = 1, kSegTN = 2 };

struct SegParams {
    const _Float16 *a;      // NT, NN: [a_rows, k]; TN: [rows, k]
    const _Float16 *b;      // NT: [groups, n, k]; NN: [groups, k, n]; TN: [rows, n]
    void *c;                // NT, NN: [rows, n]; TN: [groups, k, n]; fp16 or fp32
    const int32_t *offsets; // [groups + 1]
    const int32_t *index;   // NT: row r takes A's row index[r] / fan; null: row r
    int64_t a_rows;
    int32_t rows, groups, n, k, fan;
    int32_t num_m;          // TN: tiles along k; otherwise the most row tiles there can be
    int32_t num_n;          // tiles along n
    // TN: each segment's rows in `splits` parts of whole K-tiles, part s in
    // fp32 at c + s part_elems (1: C itself)
    int32_t splits;
    int64_t part_elems;
    // low-rank adapters (kLora kernels): rows sorted by adapter, row r of
    // C and A is order[r]
    const int32_t *order;
    const float *h;         // TN: the parts; adapters: up to kLoraFewRows rows: [h_parts][rows, h_ld] fp32, whose sum is scale_s (x D_s^T)
    const char *h_split;    // more rows: rows of h_ld values, zeros past the rank (store_split)
    const _Float16 *up;     // [adapters, n, rank]
    const float *scale;     // [adapters]: multiplies the rows of h (null: 1)
    int32_t adapters, rank, h_ld;
    int32_t h_parts;
    int32_t by_row;         // few-row kernels: workgroups per row, not per segment (thin_segment)
    uint32_t first;         // workgroups of this grid that earlier launches hold (launch_seg)
};

// This workgroup's place in a grid of launch_seg.
__device__ __forceinline__ uint32_t seg_pid(const SegParams &p) { return p.first + blockIdx.x; }

// Segment bounds, clamped so that any content of offsets stays in range.
__device__ __forceinline__ int seg_bound(const int32_t *offsets, int g, int rows) {
    return g <= 0 ? 0 : min(max(offsets[g], 0), rows);
}

// Rows [lo, lo + count) of part s of segment g (TN).
struct SegPart {
    int lo, count;
};

__device__ __forceinline__ SegPart seg_part(const SegParams &p, int g, int s, int bk) {
    const int lo = seg_bound(p.offsets, g, p.rows), len = max(seg_bound(p.offsets, g + 1, p.rows) - lo, 0);
    const int part = ((len + bk - 1) / bk + p.splits - 1) / p.splits * bk, at = min(s * part, len);
    return {lo + at, min(part, len - at)};
}

// The segment that row `row` lies in; groups: it lies behind the last one.  A
// search by the whole wave, 65 ways a step (offsets that decrease give some
// segment).
__device__ __forceinline__ int seg_of_row(const SegParams &p, int row, int lane) {
    int g = 0, span = p.groups + 1;  // one of g .. g + span - 1
    while (span > 1) {
        const int stride = (span + kWave) / (kWave + 1), at = (lane + 1) * stride;
        const uint64_t past = ~__ballot(at < span && seg_bound(p.offsets, g + at, p.rows) <= row);
        const int step = (past ? __builtin_ctzll(past) : kWave) * stride;
        g += step;
        span = min(stride, span - step);
    }
    return g;
}

struct SegTile {
    int g;      // segment; groups: the rows behind the last one
    int row0;   // first row of the tile
    int valid;  // rows of the tile inside the segment
};

__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int u = __shfl_up(v, d);
        if (lane >= d) v += u;
    }
    return v;
}

// The row tiles of all segments, BM rows each and none across a border, in
// segment order.  One wave-wide scan per 64 segments: lane l holds segment
// base + l.
template <int BM>
struct SegMap {
    int lo, hi, tiles, scan;  // this lane's segment of the first 64
    int total;

    __device__ __forceinline__ void chunk(const SegParams &p, int base, int lane, int &l, int &h, int &t) const {
        const int g = base + lane;
        l = h = 0;
        if (g <= p.groups) {  // segment `groups`: the rows behind the last one
            l = seg_bound(p.offsets, g, p.rows);
            h = g < p.groups ? seg_bound(p.offsets, g + 1, p.rows) : p.rows;
        }
        t = h > l ? (int)(((int64_t)(h - l) + BM - 1) / BM) : 0;
    }

    __device__ __forceinline__ void init(const SegParams &p, int lane) {
        chunk(p, 0, lane, lo, hi, tiles);
        scan = wave_scan(tiles, lane);
        total = __builtin_amdgcn_readlane(scan, kWave - 1);
        for (int base = kWave; base <= p.groups; base += kWave) {
            int l, h, t;
            chunk(p, base, lane, l, h, t);
            total += __builtin_amdgcn_readlane(wave_scan(t, lane), kWave - 1);
        }
        // offsets that decrease could claim more tiles than the grid has
        total = min(max(total, 0), p.num_m);
    }

    // tile m < total
    __device__ __forceinline__ SegTile find(const SegParams &p, int m, int lane) const {
        int l = lo, h = hi, t = tiles, s = scan, base = 0, before = 0;
        for (;;) {
            const uint64_t hit = __ballot(before + s > m);
            if (hit) {
                const int who = __builtin_ctzll(hit);
                SegTile r;
                r.g = base + who;
                const int seg_lo = __builtin_amdgcn_readlane(l, who), seg_hi = __builtin_amdgcn_readlane(h, who);
                const int first = before + __builtin_amdgcn_readlane(s, who) - __builtin_amdgcn_readlane(t, who);
                r.row0 = seg_lo + (m - first) * BM;
                // (always inside, unless decreasing offsets made the counts wrap)
                r.valid = r.row0 >= seg_lo && r.row0 < seg_hi ? min(BM, seg_hi - r.row0) : 0;
                return r;
            }
            before += __builtin_amdgcn_readlane(s, kWave - 1);
            base += kWave;
            if (base > p.groups) return SegTile{p.groups, 0, 0};  // not reached for m < total
            chunk(p, base, lane, l, h, t);
            s = wave_scan(t, lane);
        }
    }
};

// ---- operands staged through registers -----------------------------------------
//
// For rows that are not 16-byte aligned (K or N not a multiple of 8) and
// gathers from more than 2 GiB: 16-byte global loads at any 2-byte aligned
// address, written to the LDS layouts that the direct-to-LDS operands of
// kernels.h use, so both share their fragment reads.

typedef int int4u __attribute__((ext_vector_type(4), aligned(2)));
typedef int int2u __attribute__((ext_vector_type(2), aligned(2)));

// 8 elements from p; those at or past end (the tensor's end) are zero and
// never touched.
__device__ __forceinline__ int4v load_chunk(const _Float16 *p, const _Float16 *end) {
    if ((uintptr_t)(p + 8) <= (uintptr_t)end) return *reinterpret_cast<const int4u *>(p);
    union {
        int4v v;
        _Float16 e[8];
    } u;
    u.v = int4v{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if ((uintptr_t)(p + i) < (uintptr_t)end) u.e[i] = p[i];
    return u.v;
}

// elements e >= kv of a chunk become zero
__device__ __forceinline__ int4v mask_chunk(int4v v, int kv) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] &= (kv > 2 * j + 1) ? -1 : (kv > 2 * j) ? 0xffff : 0;
    return v;
}

// Rows of K contiguous elements (KMajorDirect's layout).
template <class C, int ROWS>
struct KMajorStaged {
    static constexpr int kRow = 128;
    static constexpr int kStage = ROWS * kRow;
    static constexpr int kLoads = kStage / 1024 / C::kWaves;
    static_assert(kLoads * 1024 * C::kWaves == kStage, "whole blocks per wave");

    const _Float16 *row[kLoads];  // this lane's row of load i, null past the tile
    const _Float16 *end;
    int4v regs[kLoads];
    int kc, k_elems, kv;
    int lds_w, r_lane[C::KS];

    static __device__ __forceinline__ int sw(int r) { return (r >> 1) & 7; }
    // tile row of load i
    static __device__ __forceinline__ int tile_row(int i, int wave, int lane) {
        return (i * C::kWaves + wave) * 8 + (lane >> 3);
    }

    __device__ __forceinline__ void init(const _Float16 *tensor_end, int K, int wave, int lane, int frag_row, int lds) {
        end = tensor_end;
        k_elems = K;
        kc = ((lane & 7) ^ sw(tile_row(0, wave, lane))) * 8;
        lds_w = lds + wave * 1024 + lane * 16;
        const int q = lane / 16, frow = frag_row + lane % 16;
#pragma unroll
        for (int ks = 0; ks < C::KS; ++ks) r_lane[ks] = lds + frow * kRow + (((4 * ks + q) ^ sw(frow)) << 4);
    }

    __device__ __forceinline__ void load(int t) {
        const int k0 = t * C::BK + kc;
        kv = k_elems - k0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            regs[i] = (row[i] && kv > 0) ? load_chunk(row[i] + k0, end) : int4v{0, 0, 0, 0};
    }

    __device__ __forceinline__ void store(char *smem, int stage) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            *reinterpret_cast<int4v *>(smem + lds_w + stage * kStage + i * C::kWaves * 1024) = mask_chunk(regs[i], kv);
    }

    __device__ __forceinline__ half8 read(const char *smem, int stage, int ks, int f) const {
        return *reinterpret_cast<const half8 *>(smem + r_lane[ks] + stage * kStage + f * 16 * kRow);
    }
};

// COLS columns of a [contraction, ld] matrix (NMajorDirect's layout).
// Columns past the matrix hold whatever follows in memory: they reach only
// outputs that are never stored.  Contraction rows past the last are zero.
template <class C, int COLS, int F>
struct NMajorStaged {
    static constexpr int CPR = COLS / 8, kRowB = COLS * 2;
    static constexpr int kStage = C::BK * kRowB;
    static constexpr int kRowsPerBlock = 1024 / kRowB;
    static constexpr int kLoads = kStage / 1024 / C::kWaves;
    static_assert(CPR >= 16 && CPR <= 64 && kLoads * 1024 * C::kWaves == kStage, "layout");

    const _Float16 *base, *end;  // first contraction row, first column of the tile
    int64_t ld;
    int count, cols;             // contraction rows; columns from the tile's first on
    int r0[kLoads], c0[kLoads];
    int4v regs[kLoads];
    int lds_w, r_lane[F];

    static __device__ __forceinline__ int sw(int r) { return 2 * ((r & 3) | ((r >> 1) & 4)); }

    __device__ __forceinline__ void init(const _Float16 *first, const _Float16 *tensor_end, int64_t pitch, int rows,
                                         int columns, int wave, int lane, int frag_col, int lds) {
        base = first;
        end = tensor_end;
        ld = pitch;
        count = rows;
        cols = columns;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            r0[i] = (i * C::kWaves + wave) * kRowsPerBlock + lane / CPR;
            c0[i] = ((lane % CPR) ^ sw(r0[i])) * 8;
        }
        lds_w = lds + wave * 1024 + lane * 16;
        const int g = lane >> 4, j = lane & 15;
        const int row = 8 * g + (j >> 2);
        const int fsw = sw(row) >> 1;
#pragma unroll
        for (int f = 0; f < F; ++f)
            r_lane[f] = lds + row * kRowB + ((((frag_col >> 4) + f) ^ fsw) << 5) + (((j >> 1) & 1) << 4) + ((j & 1) << 3);
    }

    __device__ __forceinline__ void load(int t) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = t * C::BK + r0[i];
            regs[i] = (r < count && c0[i] < cols) ? load_chunk(base + r * ld + c0[i], end) : int4v{0, 0, 0, 0};
        }
    }

    __device__ __forceinline__ void store(char *smem, int stage) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            *reinterpret_cast<int4v *>(smem + lds_w + stage * kStage + i * C::kWaves * 1024) = regs[i];
    }

    __device__ __forceinline__ half8 read(const char *smem, int stage, int ks, int f) const {
        char *p0 = const_cast<char *>(smem) + r_lane[f] + stage * kStage + ks * 32 * kRowB;
        const fp16x4 lo = lds_read_tr16((lds_fp16x4 *)p0);
        const fp16x4 hi = lds_read_tr16((lds_fp16x4 *)(p0 + 4 * kRowB));
        half8 r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r[e] = (_Float16)lo[e];
            r[4 + e] = (_Float16)hi[e];
        }
        return r;
    }
};

// ---- epilogue ------------------------------------------------------------------
//
// The wave's accumulators through its share of LDS (CStaging) into rows of
// C: 16-byte stores where C's rows are 16-byte aligned, else element by
// element.  rows: valid rows of the tile; n: columns of C; row_of(r): row of
// C of tile row r.
template <class C, bool F32, int kWaveBytes, class RowOf>
__device__ __forceinline__ void seg_store(const floatx4 (&acc)[C::FN][C::FM], char *stg, void *c, int rows, int n,
                                          int n0, int wm, int wn, int lane, RowOf row_of) {
    using CS = CStaging<C, F32, kWaveBytes>;
    using Out = typename CS::Out;
    constexpr int E = 16 / CS::ES;
    const int erow = CS::opaque_row(lane);
    const bool vec = (n % E) == 0 && ((uintptr_t)c % 16) == 0;
#pragma unroll
    for (int pass = 0; pass < CS::kPasses; ++pass) {
        CS::write_pass(acc, stg, pass, erow, lane);
#pragma unroll
        for (int s = 0; s < CS::kPerPass; ++s) {
            const int idx = s * kWave + lane;
            const int r = wm * C::TM + pass * CS::SR + idx / CS::CPR;
            const int col = n0 + wn * C::TN + (idx % CS::CPR) * E;
            const int4v v = CS::read_chunk(stg, s, lane);
            if (r < rows && col < n) {
                Out *dst = static_cast<Out *>(c) + (int64_t)row_of(r) * n + col;
                if (vec) {
                    *reinterpret_cast<int4v *>(dst) = v;
                } else {
                    union {
                        int4v v;
                        Out e[E];
                    } u;
                    u.v = v;
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (col + e < n) dst[e] = u.e[e];
                }
            }
        }
    }
}

// ---- adapters: the low-rank product on top of a tile ---------------------------
//
// Adds h U_s^T, h = scale_s x D_s^T, to a tile of x W^T whose rows are
// sorted by adapter: for each adapter with rows in the tile and each 32 of its
// ranks, one K-tile whose A is h, zero in rows of other adapters, and whose
// B is U_s.  h is an fp32 sum, so it goes through the MFMA as three bf16 parts,
// which hold it exactly, and U_s as two that do.  Five products of parts
// make h U: the sixth, h2 u1, is at most 2^-24 of it, half a step of an fp32
// product (|h2| <= 2^-16 |h|, |u1| <= 2^-8 |u|).  Two parts of h, with three
// products, lost 2^-17 of h and took 3 to 5% less (4096 rows, 4096 x 4096, 8
// adapters of rank 64: 139 to 145 us on three hosts, against 146 to 150).
//
// An infinity or NaN in U_s would reach the rows of other adapters as
// 0 * inf: it is taken as 1 of its sign here (not as 0: h may be infinite
// there), and lora_wild adds its products, none of them finite, to the rows of
// its adapter afterwards.  An infinity in h has to give u * inf, so it
// travels as h2, which meets u0 alone: u's sign, and 0 where u is 0 (times
// u1, of 0 or the other sign, it would be a NaN).

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ void mfma16_tied_bf16(bf16x8 a, bf16x8 b, floatx4 &c) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}

// x's upper 16 bits, the rest cut off
__device__ __forceinline__ __bf16 bf16_cut(float x) {
    return __builtin_bit_cast(__bf16, (uint16_t)(__builtin_bit_cast(uint32_t, x) >> 16));
}

constexpr int kSplit = 192;  // bytes of 32 values of h
constexpr int kSplitValue = kSplit / 32;

// h as its consumer's K-tiles: a row holds, for each 32 ranks, 32 values h0,
// the 32 next parts h1 and the 32 last h2, bf16.  Four values of a row, times
// f; zeros past the rank (n % 4 == 0, n < h_ld).
__device__ __forceinline__ void store_split(char *row, int n, floatx4 v, float f, int rank) {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    bf16x4 top, next, last;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float x = n + e < rank ? v[e] * f : 0.0f;
        const bool finite = fabsf(x) < __builtin_inff();
        top[e] = (__bf16)(finite ? x : 0.0f);
        // what rounds up to infinity is cut instead
        if (!(fabsf((float)top[e]) < __builtin_inff())) top[e] = bf16_cut(x);
        const float rest = finite ? x - (float)top[e] : 0.0f;  // both differences are exact
        next[e] = (__bf16)rest;
        last[e] = (__bf16)(finite ? rest - (float)next[e] : x);
    }
    char *to = row + n / 32 * kSplit + n % 32 * 2;
    *reinterpret_cast<bf16x4 *>(to) = top;
    *reinterpret_cast<bf16x4 *>(to + 64) = next;
    *reinterpret_cast<bf16x4 *>(to + 128) = last;
}

// The adapters with rows in [row0, row0 + valid), in order: lane l looks at
// adapter base + l.
struct LoraWalk {
    int base = -kWave, seg_lo = 0, seg_hi = 0;
    uint64_t todo = 0;
    int s = -1, lo = 0, hi = 0;  // the current one (-1: none left), its rows inside the tile

    __device__ __forceinline__ void next(const SegParams &p, int row0, int valid, int lane) {
        while (todo == 0 && base + kWave < p.adapters) {
            base += kWave;
            const int t = base + lane;
            seg_lo = seg_hi = 0;
            if (t < p.adapters) {
                seg_lo = max(seg_bound(p.offsets, t, p.rows) - row0, 0);
                seg_hi = min(seg_bound(p.offsets, t + 1, p.rows) - row0, valid);
            }
            todo = __ballot(seg_lo < seg_hi);
        }
        const int who = todo ? __builtin_ctzll(todo) : 0;
        s = todo ? base + who : -1;
        todo &= todo - 1;
        lo = __builtin_amdgcn_readlane(seg_lo, who);
        hi = __builtin_amdgcn_readlane(seg_hi, who);
    }
};

// Bytes of LDS that lora_tiles takes: two stages of the three parts of h, each
// a plane of 64-byte rows whose 16-byte chunk c sits at c ^ (row / 4) % 4 (so
// that 16 rows' chunks c lie on different banks), and of U_s.
template <class C>
constexpr int lora_lds() {
    return 2 * (C::BM * kSplit + C::BN * 128);
}

// Returns (to every thread) whether some U_s of the tile is not finite.
// w: the first adapter with rows in the tile.  votes: one int per wave, in
// the kernel's one LDS array (a library vote would bring an array of its own,
// see seg_tile), behind what the epilogue uses: the last stage is done with
// by then.  RANK4: the rank is a multiple of 4, so half chunks lie
// wholly inside a row of U_s; the tails of other ranks cost scalar registers
// that the 256-wide tiles do not have.
//
// Two LDS stages.  h's K-tile comes straight into the other stage under the
// MFMAs of this one; U_s comes through registers two K-tiles ahead, and is
// split and written an element at a time between the MFMAs.
//
// 4096 rows, 4096 x 4096, 8 adapters of rank 64 in runs: 133 us against 104
// without adapters; a tile across three adapters does six such K-tiles of 5
// MFMAs per block beside its 64 of 2.
template <class C, bool RANK4>
__device__ __forceinline__ bool lora_tiles(floatx4 (&acc)[C::FN][C::FM], char *smem, int *votes, const SegParams &p,
                                           LoraWalk w, int row0, int valid, int n0, int tid, int lane, int wm, int wn) {
    constexpr int kRow = 128, kPlane = C::BM * 64, kB = 3 * kPlane, kStage = kB + C::BN * kRow;
    static_assert(2 * kStage == lora_lds<C>(), "LDS of the stages");
    auto sw = [](int r) { return (r >> 1) & 7; };
    auto sw_h = [](int r) { return (r >> 2) & 3; };
    constexpr int BA = kB / 1024, LA = (BA + C::kWaves - 1) / C::kWaves, HB = C::BN * 4 / C::kThreads;  // blocks of 16 rows
    static_assert(C::BM % 16 == 0 && HB * C::kThreads == C::BN * 4, "whole passes");
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const uint32_t pitch = (uint32_t)p.h_ld * kSplitValue;
    const __amdgpu_buffer_rsrc_t h_rows = make_rsrc(p.h_split + (int64_t)row0 * pitch, (uint32_t)valid * pitch);
    const _Float16 *up_end = p.up + (int64_t)p.adapters * p.n * p.rank;
    int c = 0;  // w's next K-tile starts at rank c
    auto load_h = [&](int stage) {
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            const int block = i * C::kWaves + wave;
            if (BA % C::kWaves != 0 && block >= BA) continue;
            const int r = block % (C::BM / 16) * 16 + (lane >> 2);
            const uint32_t off = (uint32_t)r * pitch + (uint32_t)(block / (C::BM / 16) * 64 + (((lane & 3) ^ sw_h(r)) << 4));
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                h_rows, (__attribute__((address_space(3))) void *)(smem + stage * kStage + block * 1024), 16,
                r >= w.lo && r < w.hi ? off : kOutOfRange, (uint32_t)c * (uint32_t)kSplitValue, 0, 0);
        }
    };
    auto fetch_u = [&](int4v (&u)[HB]) {
        const _Float16 *up = p.up + (int64_t)w.s * p.n * p.rank;
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            const int x = i * C::kThreads + tid, r = n0 + (x >> 2), k = c + 8 * (x & 3);
            u[i] = int4v{0, 0, 0, 0};
            const _Float16 *row = up + (int64_t)r * p.rank + k;
            if constexpr (RANK4) {
                if (r < p.n && k < p.rank) {
                    const int2u v = *reinterpret_cast<const int2u *>(row);
                    u[i][0] = v[0];
                    u[i][1] = v[1];
                }
                if (r < p.n && k + 4 < p.rank) {
                    const int2u v = *reinterpret_cast<const int2u *>(row + 4);
                    u[i][2] = v[0];
                    u[i][3] = v[1];
                }
            } else {
                if (r < p.n && k < p.rank) u[i] = mask_chunk(load_chunk(row, up_end), p.rank - k);
            }
        }
    };
    auto advance = [&]() {
        c += 32;
        if (c >= p.rank) {
            w.next(p, row0, valid, lane);
            c = 0;
        }
    };
    // Element e of this thread's chunks of U_s split into its bf16 parts; a
    // whole chunk goes to LDS.
    int wild = 0;
    bf16x8 top, rest;
    int4v u[HB], ahead[HB];
    auto split = [&](auto e_c, char *to) {
        constexpr int i = decltype(e_c)::value / 8, e = decltype(e_c)::value % 8;
        float v = (float)__builtin_bit_cast(half8, u[i])[e];
        if (!(fabsf(v) < __builtin_inff())) {
            v = copysignf(1.0f, v);
            wild = 1;
        }
        top[e] = (__bf16)v;
        rest[e] = (__bf16)(v - (float)top[e]);  // exact: at most 3 bits are left
        if constexpr (e == 7) {
            const int x = i * C::kThreads + tid, r = x >> 2, q = x & 3;
            *reinterpret_cast<bf16x8 *>(to + kB + r * kRow + ((q ^ sw(r)) << 4)) = top;
            *reinterpret_cast<bf16x8 *>(to + kB + r * kRow + (((q + 4) ^ sw(r)) << 4)) = rest;
        }
    };
    constexpr int E = HB * 8;
    // u0 h0, u1 h0, u0 h1, u1 h1, then u0 h2
    constexpr int NM = C::FM * C::FN, M = 5 * NM;

    int stage = 0;
    bool more = w.s >= 0;
#pragma unroll
    for (int i = 0; i < HB; ++i) ahead[i] = int4v{0, 0, 0, 0};
    if (more) {
        load_h(0);
        fetch_u(u);
        advance();
        if (w.s >= 0) fetch_u(ahead);
        static_range<0, E>([&](auto e_c) { split(e_c, smem); });
    }
    vm_barrier<0>();
    while (more) {
        // stage holds this K-tile; w and c are at the next one, whose U_s is
        // in `ahead` (past the last, what is split is never read)
#pragma unroll
        for (int i = 0; i < HB; ++i) u[i] = ahead[i];
        more = w.s >= 0;
        if (more) {
            load_h(stage ^ 1);
            advance();
            if (w.s >= 0) fetch_u(ahead);
        }
        const char *from = smem + stage * kStage;
        char *to = smem + (stage ^ 1) * kStage;
        bf16x8 af[C::FM], bf = {};
        static_range<0, M>([&](auto m_c) {
            constexpr int m = decltype(m_c)::value;
            constexpr int ka = m / (2 * NM), kb = m / NM % 2, j = m % NM / C::FM, i = m % C::FM;
            if constexpr (m % (2 * NM) == 0) {
#pragma unroll
                for (int q = 0; q < C::FM; ++q) {
                    const int r = wm * C::TM + q * 16 + lane % 16;
                    af[q] = *reinterpret_cast<const bf16x8 *>(from + ka * kPlane + r * 64 + (((lane / 16) ^ sw_h(r)) << 4));
                }
            }
            if constexpr (i == 0) {
                const int r = wn * C::TN + j * 16 + lane % 16;
                bf = *reinterpret_cast<const bf16x8 *>(from + kB + r * kRow + (((4 * kb + lane / 16) ^ sw(r)) << 4));
            }
            mfma16_tied_bf16(bf, af[i], acc[j][i]);
            static_range<m * E / M, (m + 1) * E / M>([&](auto e_c) { split(e_c, to); });
            __builtin_amdgcn_sched_barrier(0);
        });
        vm_barrier<0>();
        stage ^= 1;
    }
    acc_fence(acc);
    const uint64_t ballot = __ballot(wild);
    if (lane == 0) votes[tid / kWave] = ballot != 0;
    lds_barrier();
    int r = 0;
#pragma unroll
    for (int q = 0; q < C::kWaves; ++q) r |= votes[q];
    return __builtin_amdgcn_readfirstlane(r) != 0;
}

// Adds the products with the elements of U_s that are not finite to the
// stored tile (never on a model's path: such weights are broken, and this
// keeps the other adapters' rows whole).
template <class C>
__device__ __forceinline__ void lora_wild(const SegParams &p, int row0, int valid, int n0, int tid, int lane) {
    __threadfence();
    __syncthreads();  // the tile is stored
    const int cols = min(C::BN, p.n - n0);
    LoraWalk w;
    for (w.next(p, row0, valid, lane); w.s >= 0; w.next(p, row0, valid, lane)) {
        for (int r = row0 + w.lo; r < row0 + w.hi; ++r) {
            _Float16 *y = static_cast<_Float16 *>(p.c) + (int64_t)min(max(p.order[r], 0), p.rows - 1) * p.n + n0;
            for (int n = tid; n < cols; n += C::kThreads) {
                const _Float16 *up = p.up + ((int64_t)w.s * p.n + n0 + n) * p.rank;
                float sum = 0.0f;
#pragma unroll 1
                for (int j = 0; j < p.rank; ++j) {
                    const float f = (float)up[j];
                    if (fabsf(f) < __builtin_inff()) continue;
                    const __bf16 *h = reinterpret_cast<const __bf16 *>(p.h_split + (int64_t)r * p.h_ld * kSplitValue + j / 32 * kSplit);
                    sum += ((float)h[j % 32] + (float)h[32 + j % 32] + (float)h[64 + j % 32]) * f;
                }
                if (!(fabsf(sum) < __builtin_inff())) y[n] = (_Float16)((float)y[n] + sum);
            }
        }
    }
}

// ---- the any-alignment kernel --------------------------------------------------
//
// One workgroup per tile, operands staged through registers one K-tile
// ahead, two LDS stages, one barrier per K-tile.  Every size, alignment and
// gather.  16384 rows in 8 segments of 4096 x 2048 took 419 us on it, where the
// direct-to-LDS tiles take 240-253: the loads' way through registers and the
// wait at each K-tile bound it.
// LORA: x W^T over rows sorted by adapter, then lora_tiles; rows leave through
// order.
template <int KIND, class C, bool F32, bool LORA>
__global__ __launch_bounds__(C::kThreads) void seg_staged_kernel(const SegParams p) {
    static_assert(C::MB == 16 && C::KS == 2, "16x16x32 tiles");
    static_assert(!LORA || KIND == kSegNT, "adapters are NT products");
    using OpA = std::conditional_t<KIND == kSegTN, NMajorStaged<C, C::BM, C::FM>, KMajorStaged<C, C::BM>>;
    using OpB = std::conditional_t<KIND == kSegNT, KMajorStaged<C, C::BN>, NMajorStaged<C, C::BN, C::FN>>;
    constexpr int kLdsB = 2 * OpA::kStage, kLds = kLdsB + 2 * OpB::kStage;
    // one LDS array: with two, the compiler waits for every load in flight
    // before each fragment read
    constexpr int kAll = LORA ? lora_lds<C>() : kLds;
    static_assert(kAll <= 160 * 1024 && (!LORA || kLds + C::kWaves * 4 <= kAll), "LDS budget");
    __shared__ __attribute__((aligned(1024))) char smem[kAll];
    GEMM_POISON_LDS(smem);

    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int wm = wave / C::WN, wn = wave % C::WN;

    OpA opa;
    OpB opb;
    int g, row0, valid, n0, kt_count, split = 0;
    if constexpr (KIND == kSegTN) {
        const uint32_t per = (uint32_t)p.num_m * (uint32_t)p.num_n;
        g = (int)(seg_pid(p) / per);
        split = (int)blockIdx.y;
        const TileCoord tc = tile_coord<uint32_t>(seg_pid(p) % per, p.num_m, p.num_n, 4, false);
        const int m0 = (int)tc.m_block * C::BM;
        n0 = (int)tc.n_block * C::BN;
        const auto [lo, cnt] = seg_part(p, g, split, C::BK);
        row0 = m0;
        valid = min(C::BM, p.k - m0);
        kt_count = (cnt + C::BK - 1) / C::BK;
        opa.init(p.a + (int64_t)lo * p.k + m0, p.a + (int64_t)p.rows * p.k, p.k, cnt, p.k - m0, wave, lane, wm * C::TM,
                 0);
        opb.init(p.b + (int64_t)lo * p.n + n0, p.b + (int64_t)p.rows * p.n, p.n, cnt, p.n - n0, wave, lane,
                 wn * C::TN, kLdsB);
    } else {
        const uint32_t pid = seg_pid(p);
        if constexpr (LORA) {
            g = 0;
            const TileCoord tc = tile_coord<uint32_t>(pid, (p.rows + C::BM - 1) / C::BM, p.num_n, 4, true);
            row0 = (int)tc.m_block * C::BM;
            valid = min(C::BM, p.rows - row0);
            n0 = (int)tc.n_block * C::BN;
        } else {
            SegMap<C::BM> map;
            map.init(p, lane);
            if (pid >= (uint32_t)map.total * (uint32_t)p.num_n) return;  // num_m * num_n < 2^31
            const TileCoord tc = tile_coord<uint32_t>(pid, map.total, p.num_n, 4, true);
            const SegTile st = map.find(p, (int)tc.m_block, lane);
            g = st.g;
            row0 = st.row0;
            valid = st.valid;
            n0 = (int)tc.n_block * C::BN;
        }
        // the rows behind the last segment: no K-tile, so zeros
        const bool live = LORA || g < p.groups;
        kt_count = live ? (p.k + C::BK - 1) / C::BK : 0;
        const _Float16 *a_end = p.a + p.a_rows * p.k;
        const int32_t *from = LORA ? p.order : p.index;
        opa.init(a_end, p.k, wave, lane, wm * C::TM, 0);
#pragma unroll
        for (int i = 0; i < OpA::kLoads; ++i) {
            const int r = OpA::tile_row(i, wave, lane);
            int64_t src = row0 + r;
            if (from && r < valid) {
                const int v = from[row0 + r];
                src = v < 0 ? -1 : LORA ? v : v / p.fan;
            }
            opa.row[i] = (live && r < valid && src >= 0 && src < p.a_rows) ? p.a + src * p.k : nullptr;
        }
        const int64_t per_group = (int64_t)p.n * p.k;
        const int64_t count = LORA ? 1 : p.groups;
        const _Float16 *b = p.b + (live ? g : 0) * per_group, *b_end = p.b + count * per_group;
        if constexpr (KIND == kSegNT) {
            opb.init(b_end, p.k, wave, lane, wn * C::TN, kLdsB);
#pragma unroll
            for (int i = 0; i < OpB::kLoads; ++i) {
                const int r = n0 + OpB::tile_row(i, wave, lane);
                opb.row[i] = r < p.n ? b + (int64_t)r * p.k : nullptr;
            }
        } else {
            opb.init(b + n0, b_end, p.n, p.k, p.n - n0, wave, lane, wn * C::TN, kLdsB);
        }
    }

    floatx4 acc[C::FN][C::FM];
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int i = 0; i < C::FM; ++i) acc[j][i] = floatx4{};

    if (kt_count > 0) {
        opa.load(0);
        opb.load(0);
        opa.store(smem, 0);
        opb.store(smem, 0);
    }
    lds_barrier();
    for (int t = 0; t < kt_count; ++t) {
        const bool more = t + 1 < kt_count;
        if (more) {
            opa.load(t + 1);
            opb.load(t + 1);
        }
#pragma unroll
        for (int ks = 0; ks < C::KS; ++ks) {
            half8 af[C::FM];
#pragma unroll
            for (int i = 0; i < C::FM; ++i) af[i] = opa.read(smem, t & 1, ks, i);
#pragma unroll
            for (int j = 0; j < C::FN; ++j) {
                const half8 bf = opb.read(smem, t & 1, ks, j);
#pragma unroll
                for (int i = 0; i < C::FM; ++i) acc[j][i] = Mfma<16>::run(bf, af[i], acc[j][i]);
            }
        }
        // the other stage was last read before the barrier that ended K-tile t-1
        if (more) {
            opa.store(smem, (t + 1) & 1);
            opb.store(smem, (t + 1) & 1);
        }
        lds_barrier();
    }

    constexpr int kWaveBytes = kLds / C::kWaves;
    char *const stg = smem + wave * kWaveBytes;
    if constexpr (LORA) {
        LoraWalk walk;
        walk.next(p, row0, valid, lane);
        const bool wild = lora_tiles<C, false>(acc, smem, reinterpret_cast<int *>(smem + kLds), p, walk, row0, valid, n0, tid, lane, wm, wn);
        const int32_t *order = p.order;
        const int rows = p.rows;
        seg_store<C, F32, kWaveBytes>(acc, stg, p.c, valid, p.n, n0, wm, wn, lane, [&](int r) {
            return min(max(order[row0 + r], 0), rows - 1);
        });
        if (wild) lora_wild<C>(p, row0, valid, n0, tid, lane);
    } else if constexpr (KIND == kSegTN) {
        using Out = std::conditional_t<F32, float, _Float16>;
        Out *c = static_cast<Out *>(p.c) + split * p.part_elems + (int64_t)g * p.k * p.n;
        seg_store<C, F32, kWaveBytes>(acc, stg, c, valid, p.n, n0, wm, wn, lane, [&](int r) { return row0 + r; });
    } else {
        seg_store<C, F32, kWaveBytes>(acc, stg, p.c, valid, p.n, n0, wm, wn, lane, [&](int r) { return row0 + r; });
    }
}

// A launch holds fewer than 2^32 threads along x, and one of more loses the
// rest without an error: such a grid (below 2^31 workgroups) goes out in
// several launches.  args: the kernel's, with `first` inside one of them.
inline hipError_t launch_grid(const void *kernel, int64_t grid, int parts, int threads, hipStream_t stream, void **args,
                              uint32_t &first) {
    if (grid >= (int64_t(1) << 31)) return hipErrorInvalidValue;
    const int64_t most = ((int64_t(1) << 32) - 1) / threads;
    for (int64_t at = 0; at < grid; at += most) {
        first = (uint32_t)at;
        const hipError_t e = hipLaunchKernel(kernel, dim3((unsigned)std::min(most, grid - at), (unsigned)parts),
                                             dim3((unsigned)threads), args, 0, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <class Kernel>
inline hipError_t launch_seg(Kernel kernel, int64_t grid, int threads, hipStream_t stream, SegParams p, int parts = 1) {
    void *args[] = {&p};
    return launch_grid(reinterpret_cast<const void *>(kernel), grid, parts, threads, stream, args, p.first);
}

// Row tiles that the segments can need at most, whatever their sizes: each
// segment that is not empty (at most one per row; the rows behind the last
// one count as one) takes ceil(size / bm) <= (size - 1) / bm + 1.
inline int64_t seg_row_tiles(int64_t rows, int64_t groups, int64_t bm) {
    const int64_t used = groups + 1 < rows ? groups + 1 : rows;
    return (rows - used) / bm + used;
}

using SegCfg128 = Cfg<128, 128, 2, 2, 16>;

constexpr int kGroupOneBlock = 8192;  // rows that one workgroup sorts
constexpr int kGroupMax = 2048;       // groups (a wave's counters of every group fit in LDS)
int64_t group_blocks(int64_t rows);
// counts: group_blocks(rows) * (groups + 1) ints, used with more than one block
hipError_t launch_group_rows(int64_t rows, int groups, const void *ids, int id_bytes, int32_t *order, int32_t *inverse,
                             int32_t *offsets, int32_t *counts, hipStream_t s);
// Direct-to-LDS kernels (segments_direct.h), by block tile.
enum SegTileId : int { kSeg256x256, kSeg256x128, kSeg128x256, kSeg128x128, kSeg64x128, kSeg32x128, kSegRing, kSegRing2 };
hipError_t launch_seg_nt(int tile, bool f32, const SegParams &p, hipStream_t s);
hipError_t launch_seg_nn(int tile, bool f32, const SegParams &p, hipStream_t s);
hipError_t launch_seg_tn(int tile, bool f32, const SegParams &p, hipStream_t s);
// Tiles of one walking workgroup at most (its list is in LDS).
constexpr int kWalkTiles = 24;
// The same with one workgroup per CU walking its tiles (segments_walk.h).
hipError_t launch_seg_walk_nt(int tile, bool f32, bool device_stores, int cus, const SegParams &p, hipStream_t s);
hipError_t launch_seg_walk_nn(int tile, bool f32, bool device_stores, int cus, const SegParams &p, hipStream_t s);
hipError_t launch_seg_lora(int tile, const SegParams &p, hipStream_t s);

// Few rows (seg_thin.hip).
constexpr int64_t kLoraFewRows = 64;  // rows up to here: launch_lora_few
hipError_t launch_seg_thin(bool f32, const SegParams &p, hipStream_t s);
// h in its parts, rows in adapter order: direct-to-LDS tiles, or any rows
hipError_t launch_lora_down(SegParams p, hipStream_t s);
hipError_t launch_lora_down_thin(const SegParams &p, hipStream_t s);
// sums: fp32 [lora_few_parts(k)][rows, n]; down.c is h with rows in their own
// order, lora_few_h_parts(k) arrays
int lora_few_parts(int64_t k);
int lora_few_h_parts(int64_t k);
hipError_t launch_lora_few(const SegParams &p, const SegParams &down, float *sums, const int32_t *ids, hipStream_t s);

// C = the sum of the parts at p.h, in their order
hipError_t launch_seg_join(bool f32, const SegParams &p, hipStream_t s);

hipError_t launch_seg_staged(int kind, bool f32, bool lora, SegParams p, hipStream_t s);

}  // namespace gemm_f16
