// Host side of the segmented products: argument checks, the choice of
// kernel and the launches (see segments.h).
#include "segments.h"

#include <algorithm>
#include <cmath>
#include <iterator>

#include "device.h"
#include "gemm_f16.h"

namespace gemm_f16 {

constexpr int64_t kMaxRows = int64_t(1) << 30, kMaxK = int64_t(1) << 22, kMaxNMajor = int64_t(1) << 25;
// gfx950's CUs (the sizes alone say what workspace a call takes), and the most parts
constexpr int kTnCus = 256, kTnSplits = 64;
constexpr int64_t kMaxElems = int64_t(1) << 47, kMaxGroups = int64_t(1) << 20;

// One buffer of a call, for the checks on pointers.
struct Buffer {
    const void *p;
    int64_t bytes;
    int align;
    bool out;
};

// Null, alignment and overlap: outputs (and the workspace) against every
// other buffer.
template <int N>
static int check_buffers(const Buffer (&bufs)[N]) {
    for (const Buffer &b : bufs)
        if (b.bytes > 0 && !b.p) return GEMM_F16_ENULL;
    for (const Buffer &b : bufs)
        if (b.bytes > 0 && ((uintptr_t)b.p % (uintptr_t)b.align) != 0) return GEMM_F16_EALIGN;
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < N; ++j) {
            if (i == j || !bufs[i].out || bufs[i].bytes <= 0 || bufs[j].bytes <= 0) continue;
            const uintptr_t a0 = (uintptr_t)bufs[i].p, a1 = a0 + (uintptr_t)bufs[i].bytes;
            const uintptr_t b0 = (uintptr_t)bufs[j].p, b1 = b0 + (uintptr_t)bufs[j].bytes;
            if (a0 < b1 && b0 < a1) return GEMM_F16_EOVERLAP;
        }
    return GEMM_F16_OK;
}

static bool below(int64_t limit, int64_t a, int64_t b, int64_t c = 1) {
    // a, b, c >= 0 and below 2^31: a * b cannot wrap
    if (a == 0 || b == 0 || c == 0) return true;
    return a * b < limit && a * b <= (limit - 1) / c;
}

static int check_grouped(int kind, int64_t rows, int64_t groups, int64_t n, int64_t k) {
    if (kind < kSegNT || kind > kSegTN) return GEMM_F16_EINVAL;
    if (rows < 0 || n < 0 || k < 0 || rows >= kMaxRows || n >= kMaxRows || k >= kMaxK) return GEMM_F16_EINVAL;
    if (kind != kSegNT && n >= kMaxNMajor) return GEMM_F16_EINVAL;
    if (groups < 1 || groups > kMaxGroups) return GEMM_F16_EINVAL;
    if (!below(kMaxElems, rows, n) || !below(kMaxElems, n, k, groups)) return GEMM_F16_EINVAL;
    return GEMM_F16_OK;
}

static int status(hipError_t e) { return e == hipSuccess ? GEMM_F16_OK : e == hipErrorInvalidValue ? GEMM_F16_EINVAL : GEMM_F16_EHIP; }

// Whether the operands' rows can go straight into LDS: 16-byte chunks, and
// a gathered A below 2 GiB (one descriptor spans it).
static bool direct_rows(int kind, const SegParams &p) {
    if ((((uintptr_t)p.a | (uintptr_t)p.b) % 16) != 0 || p.k % 8 != 0 || p.k == 0) return false;
    // (64 rows of B below 2^31 bytes)
    if (kind != kSegNT && (p.n % 8 != 0 || p.n >= (1 << 24))) return false;
    return !(p.index || p.order) || p.a_rows * p.k * 2 < (int64_t(1) << 31);
}

static int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Whether the walking kernel can run the product on a bm x bn tile: more
// tiles than CUs but no more than fit its lists, and C's rows in whole
// 16-byte stores.
static bool can_walk(int kind, int bm, int bn, bool f32, const SegParams &p, int cus) {
    const int es = f32 ? 4 : 2;
    if (kind == kSegTN || p.order || p.n % (16 / es) != 0 || (uintptr_t)p.c % 16 != 0 ||
        (int64_t)bm * p.n * es >= (int64_t(1) << 31))
        return false;
    const int64_t tiles = seg_row_tiles(p.rows, p.groups, bm) * cdiv64(p.n, bn);
    return tiles > cus && tiles <= (int64_t)cus * kWalkTiles;
}

// Kernel of a product: a block tile (SegTileId), and whether its tiles are
// walked.
struct SegPlan {
    int tile;
    bool walk;
    double us;  // modelled
};

// The plan with the smallest modelled time (us)
//     c + a rounds k_tiles + b tiles / cus,
// rounds of one workgroup per CU, over the row tiles to expect (half a tile
// more per segment than the rows fill; the sizes are on the GPU).  For the
// walking kernels a last round in small tiles counts as 0.42 or 0.5 (256 x
// 256) or 0.66 of a round.  The coefficients are least-squares fits, in relative
// error, to sweeps of every tile over 500 shapes (rows 1 to 16384, 1 to 64
// segments, N and K from 64 to 4096, inputs cold in the caches) on MI355X.
// On 350 other shapes of that range the plan's time was 1.03 (tn) to 1.05 (nn)
// of the fastest tile's in the geometric mean and at most 1.7 of it.  With tiles to
// walk, walking measured 0.88 to 0.97 of the one-tile kernel's time on most
// shapes (nt, 256 x 128, 1 to 2 rounds: 0.91) and up to 1.15 on few.  The
// 32-row rings serve few rows per segment, where B's bytes bound the
// product.
static SegPlan pick_plan(int kind, bool f32, const SegParams &p, int cus) {
    struct Cand {
        int id, bm, bn;
        double c, a, b;     // one tile per workgroup
        double wc, wa, wb;  // walked
    };
    static const Cand nt[] = {
        {kSeg256x256, 256, 256, 6.85, 1.054, 14.80, 2.0, 1.330, 10.0},
        {kSeg256x128, 256, 128, 4.42, 0.675, 9.38, 6.4, 0.888, 5.2},
        {kSeg128x256, 128, 256, 4.46, 0.685, 9.56, 6.5, 0.909, 5.2},
        {kSeg128x128, 128, 128, 3.42, 0.461, 5.81, 0, 0, 0},
        {kSeg64x128, 64, 128, 2.84, 0.375, 3.87, 0, 0, 0},
        {kSeg32x128, 32, 128, 2.67, 0.315, 2.72, 0, 0, 0},
        {kSegRing, 32, 64, 3.57, 0.180, 0.55, 0, 0, 0},
        {kSegRing2, 32, 64, 3.30, 0.165, 1.00, 0, 0, 0},
    };
    static const Cand nn[] = {
        {kSeg256x256, 256, 256, 6.97, 1.070, 11.80, 2.0, 1.360, 10.0},
        {kSeg256x128, 256, 128, 4.36, 0.687, 7.40, 2.2, 0.887, 7.1},
        {kSeg128x256, 128, 256, 5.00, 0.632, 8.36, 1.0, 0.813, 9.5},
        {kSeg128x128, 128, 128, 3.50, 0.468, 5.00, 0, 0, 0},
        {kSeg64x128, 64, 128, 3.03, 0.405, 3.13, 0, 0, 0},
        {kSeg32x128, 32, 128, 2.73, 0.343, 2.27, 0, 0, 0},
        {kSegRing, 32, 128, 3.59, 0.284, 1.14, 0, 0, 0},
        {kSegRing2, 32, 128, 3.40, 0.250, 1.00, 0, 0, 0},
    };
    static const Cand tn[] = {
        {kSeg256x256, 256, 256, 10.0, 1.390, 8.20, 0, 0, 0},
        {kSeg256x128, 256, 128, 6.40, 0.800, 5.75, 0, 0, 0},
        {kSeg128x256, 128, 256, 6.66, 0.770, 5.87, 0, 0, 0},
        {kSeg128x128, 128, 128, 4.76, 0.520, 3.95, 0, 0, 0},
    };
    const Cand *first = kind == kSegNT ? nt : kind == kSegNN ? nn : tn;
    const Cand *last = kind == kSegNT ? std::end(nt) : kind == kSegNN ? std::end(nn) : std::end(tn);
    const int64_t segments = std::min<int64_t>(p.groups, p.rows);
    SegPlan best = {kSeg128x128, false, 1e300};
    for (const Cand *c = first; c != last; ++c) {
        if (p.order && c->id >= kSegRing) continue;  // no adapters there
        double m_tiles, k_tiles;
        if (kind == kSegTN) {
            m_tiles = (double)(cdiv64(p.k, c->bm) * p.groups);
            k_tiles = (double)std::max<int64_t>(1, cdiv64(cdiv64(p.rows, p.groups), 64));
        } else {
            m_tiles = p.order || segments == 1 ? (double)cdiv64(p.rows, c->bm)
                                               : (double)p.rows / c->bm + 0.5 * (double)segments;
            k_tiles = (double)cdiv64(p.k, 64);
        }
        const double share = m_tiles * (double)cdiv64(p.n, c->bn) / cus;
        const bool walk = can_walk(kind, c->bm, c->bn, f32, p, cus) && c->wa > 0 && share > 1;
        // half of K to each half of the waves: where the grid leaves CUs idle
        // (nt, 64 tiles of 57 K-tiles: 0.77 of the ring's time; 400 tiles: 1.1)
        if (c->id == kSegRing2 && share > (kind == kSegNT ? 0.7 : 0.4)) continue;
        double t;
        if (walk) {
            const double whole = std::floor(share), rest = share - whole;
            const bool large = c->id == kSeg256x256;
            const double tail = rest == 0 ? 0 : large && rest <= 0.25 ? 0.42 : rest <= 0.5 ? (large ? 0.5 : 0.66) : 1;
            t = c->wc + c->wa * (whole + tail) * k_tiles + c->wb * share;
        } else {
            t = c->c + c->a * std::ceil(share) * k_tiles + c->b * share;
        }
        if (t < best.us) best = {c->id, walk, t};
    }
    return best;
}

// Parts of each segment's rows for a TN product whose 128 x 128 tiles leave
// CUs idle (1: not split): the parts' sums go to the workspace in fp32 and
// a second launch adds them, in their order.  The model of pick_plan with the
// longest segment, taken as twice the mean, as the least time of a round, and
// the second launch's.  (16384 rows in one segment of 512 x 512, 16 tiles:
// 159 us unsplit, 24 in 16 parts; 4 uneven segments of 1024 x 768, 192 tiles:
// 76 and, in 2 parts, 53; 1024 rows of 512 x 512: 10.7 and 12, not split.)
static int tn_splits(int64_t rows, int64_t groups, int64_t n, int64_t k) {
    const int64_t tiles = groups * cdiv64(n, 128) * cdiv64(k, 128);
    if (tiles >= kTnCus || rows < 4 * 64) return 1;
    const int64_t longest = groups > 1 ? rows * 2 : rows;  // times groups
    const int64_t mean_kt = cdiv64(cdiv64(rows, groups), 64), long_kt = cdiv64(cdiv64(longest, groups), 64);
    SegParams p = {};
    p.rows = (int32_t)std::min<int64_t>(longest, kMaxRows);
    p.groups = (int32_t)groups;
    p.n = (int32_t)n;
    p.k = (int32_t)k;
    double best = pick_plan(kSegTN, true, p, kTnCus).us;
    int splits = 1;
    for (int s = 2; s <= kTnSplits && s <= long_kt && tiles * s <= 2 * kTnCus; ++s) {
        const double share = (double)(tiles * s) / kTnCus;
        const double round = std::max((double)cdiv64(long_kt, s), std::ceil(share) * (double)cdiv64(mean_kt, s));
        const double t = 4.76 + 0.52 * round + 3.95 * share + 7.0 + 6.0 * share;
        if (t < best) {
            best = t;
            splits = s;
        }
    }
    return splits;
}

// fp32 elements of a part: whole 16-byte chunks.
static int64_t tn_part_elems(int64_t groups, int64_t n, int64_t k) { return cdiv64(groups * n * k, 4) * 4; }

// Up to 16 rows per segment, where B's bytes bound an NT product: the few-row
// kernel while the ring's 32 x 64 tiles would be too few to fill the CUs, for
// its waves' share of K is what keeps loads in flight then (1 row, 904 x 3280:
// 6.3 us against the ring's 12.6; 10 rows over 10 segments of 608 x 2032: 8.4
// against 10.8), else the ring (16 rows over 8 segments of 4096 x 2048: 28.9
// against 31.6; 45 rows, 4 segments of 3056 x 2520: 13.1 against 19.5).  On 327
// shapes of more than 176 tiles (1 to 16 rows in each of 2 to 64 segments, N from 1024 to
// 8192, K from 256 to 8192) the ring took 1.010 of the fastest kernel's time in
// the geometric mean and 1.17 at most; pick_plan, whose fit does not tell the ring from a
// 32 x 128 tile there, 1.06 and 1.38.  Rows that cannot go straight into LDS
// have no ring to go to.
static bool byte_bound(const SegParams &p) { return p.rows <= 16 * std::min<int64_t>(p.groups, p.rows); }

static bool few_rows(const SegParams &p, bool direct) {
    const int64_t segments = std::min<int64_t>(p.groups, p.rows);
    return p.k >= 8 && byte_bound(p) && (!direct || segments * cdiv64(p.n, 64) <= 176);
}

static int grouped(int kind, int64_t rows, int64_t groups, int64_t n, int64_t k, const void *a, int64_t a_rows,
                   const void *b, const int32_t *offsets, const int32_t *index, int64_t fan, void *c, int32_t out_f32,
                   void *stream, void *workspace = nullptr, int64_t workspace_bytes = 0, int splits = 1) {
    int rc = check_grouped(kind, rows, groups, n, k);
    if (rc != GEMM_F16_OK) return rc;
    if (a_rows < 0 || a_rows >= kMaxRows || fan < 1 || fan >= kMaxRows || out_f32 < 0 || out_f32 > 1)
        return GEMM_F16_EINVAL;
    if (!index && a_rows < rows) return GEMM_F16_EINVAL;
    const int64_t out = kind == kSegTN ? groups * n * k : rows * n;
    if (out == 0) return GEMM_F16_OK;
    const int es = out_f32 ? 4 : 2;
    const int64_t part = tn_part_elems(groups, n, k), need = splits > 1 ? splits * part * 4 : 0;
    if (workspace_bytes < need) return GEMM_F16_EINVAL;
    const Buffer bufs[] = {{c, out * es, es, true},
                           {workspace, need, 16, true},
                           {a, a_rows * k * 2, 2, false},
                           {b, (kind == kSegTN ? rows * n : groups * n * k) * 2, 2, false},
                           {offsets, (groups + 1) * 4, 4, false},
                           {index, index ? rows * 4 : 0, 4, false}};
    rc = check_buffers(bufs);
    if (rc != GEMM_F16_OK) return rc;
    int cus;
    rc = current_device(&cus);
    if (rc != GEMM_F16_OK) return rc;

    SegParams p = {};
    p.a = static_cast<const _Float16 *>(a);
    p.b = static_cast<const _Float16 *>(b);
    p.c = c;
    p.offsets = offsets;
    p.index = index;
    p.a_rows = a_rows;
    p.rows = (int32_t)rows;
    p.groups = (int32_t)groups;
    p.n = (int32_t)n;
    p.k = (int32_t)k;
    p.fan = (int32_t)fan;
    p.splits = 1;
    const bool direct = direct_rows(kind, p);
    // (the few-row kernel reads some row of A even for an index outside it)
    if (kind == kSegNT && a_rows > 0 && few_rows(p, direct))
        return status(launch_seg_thin(out_f32 != 0, p, (hipStream_t)stream));
    if (splits > 1) {
        SegParams q = p;
        q.c = workspace;
        q.splits = splits;
        q.part_elems = part;
        rc = status(direct ? launch_seg_tn(kSeg128x128, true, q, (hipStream_t)stream)
                           : launch_seg_staged(kind, true, false, q, (hipStream_t)stream));
        if (rc != GEMM_F16_OK) return rc;
        q.c = c;
        q.h = static_cast<const float *>(workspace);
        return status(launch_seg_join(out_f32 != 0, q, (hipStream_t)stream));
    }
    if (direct && kind == kSegNT && byte_bound(p))
        return status(launch_seg_nt(kSegRing, out_f32 != 0, p, (hipStream_t)stream));
    if (direct) {
        const SegPlan plan = pick_plan(kind, out_f32 != 0, p, cus);
        const int tile = plan.tile;
        hipError_t e;
        if (plan.walk) {
            // cache policy of the stores: see c_store_policy in gemm_f16.hip
            const int64_t bytes = (a_rows * k + (kind == kSegTN ? rows * n : groups * n * k)) * 2 + out * es;
            const bool dev = bytes <= (int64_t(256) << 20) || (n * es) % 128 != 0 || (uintptr_t)c % 128 != 0;
            switch (kind) {
                case kSegNT: e = launch_seg_walk_nt(tile, out_f32 != 0, dev, cus, p, (hipStream_t)stream); break;
                default: e = launch_seg_walk_nn(tile, out_f32 != 0, dev, cus, p, (hipStream_t)stream); break;
            }
            return status(e);
        }
        switch (kind) {
            case kSegNT: e = launch_seg_nt(tile, out_f32 != 0, p, (hipStream_t)stream); break;
            case kSegNN: e = launch_seg_nn(tile, out_f32 != 0, p, (hipStream_t)stream); break;
            default: e = launch_seg_tn(tile, out_f32 != 0, p, (hipStream_t)stream); break;
        }
        return status(e);
    }
    return status(launch_seg_staged(kind, out_f32 != 0, false, p, (hipStream_t)stream));
}

// The few-row kernel's loads need a whole chunk of K.
static bool lora_few(int64_t rows, int64_t k) { return rows <= kLoraFewRows && k >= 8; }

// Values of h in a row: whole 16-byte stores, or lora_tiles' whole 32 ranks in
// parts
static int64_t lora_h_ld(int64_t rows, int64_t k, int64_t rank) {
    const int64_t to = lora_few(rows, k) ? 4 : 32;
    return (rank + to - 1) / to * to;
}

// Arrays whose sum is h.
static int lora_parts(int64_t rows, int64_t k) { return lora_few(rows, k) ? lora_few_h_parts(k) : 1; }

static int check_lora(int64_t rows, int64_t n, int64_t k, int64_t adapters, int64_t rank) {
    if (rows < 0 || n < 0 || k < 0 || rows >= kMaxRows || n >= kMaxRows || k >= kMaxK) return GEMM_F16_EINVAL;
    if (adapters < 1 || adapters > kMaxGroups || rank < 1 || rank > 4096) return GEMM_F16_EINVAL;
    if (!below(kMaxElems, rows, n) || !below(kMaxElems, n, k) || !below(kMaxElems, n + k, rank, adapters) ||
        !below(kMaxElems, rows, rank))
        return GEMM_F16_EINVAL;
    return GEMM_F16_OK;
}

}  // namespace gemm_f16

using namespace gemm_f16;

extern "C" {

int64_t gemm_f16_group_rows_workspace(int64_t rows, int64_t groups) {
    if (rows < 0 || rows >= kMaxRows || groups < 1 || groups > kGroupMax) return GEMM_F16_EINVAL;
    const int64_t blocks = group_blocks(rows);
    return blocks > 1 ? blocks * (groups + 1) * 4 : 0;
}

int gemm_f16_group_rows(int64_t rows, int64_t groups, const void *ids, int32_t id_bytes, int32_t *order,
                        int32_t *inverse, int32_t *offsets, void *workspace, int64_t workspace_bytes, void *stream) {
    const int64_t need = gemm_f16_group_rows_workspace(rows, groups);
    if (need < 0 || workspace_bytes < need || (id_bytes != 4 && id_bytes != 8)) return GEMM_F16_EINVAL;
    const Buffer bufs[] = {{order, rows * 4, 4, true},
                           {inverse, rows * 4, 4, true},
                           {offsets, (groups + 1) * 4, 4, true},
                           {workspace, need, 16, true},
                           {ids, rows * id_bytes, id_bytes, false}};
    int rc = check_buffers(bufs);
    if (rc != GEMM_F16_OK) return rc;
    int cus;
    rc = current_device(&cus);
    if (rc != GEMM_F16_OK) return rc;
    return status(launch_group_rows(rows, (int)groups, ids, id_bytes, order, inverse, offsets,
                                    static_cast<int32_t *>(workspace), (hipStream_t)stream));
}

int gemm_f16_grouped_nt(int64_t rows, int64_t groups, int64_t n, int64_t k, const void *a, int64_t a_rows,
                        const void *b, const int32_t *offsets, const int32_t *index, int64_t fan, void *c,
                        int32_t out_f32, void *stream) {
    return grouped(kSegNT, rows, groups, n, k, a, a_rows, b, offsets, index, fan, c, out_f32, stream);
}

int gemm_f16_grouped_nn(int64_t rows, int64_t groups, int64_t n, int64_t k, const void *a, const void *b,
                        const int32_t *offsets, void *c, int32_t out_f32, void *stream) {
    return grouped(kSegNN, rows, groups, n, k, a, rows, b, offsets, nullptr, 1, c, out_f32, stream);
}

int gemm_f16_grouped_tn(int64_t rows, int64_t groups, int64_t n, int64_t k, const void *a, const void *b,
                        const int32_t *offsets, void *c, int32_t out_f32, void *stream) {
    return grouped(kSegTN, rows, groups, n, k, a, rows, b, offsets, nullptr, 1, c, out_f32, stream);
}

int64_t gemm_f16_grouped_tn_workspace(int64_t rows, int64_t groups, int64_t n, int64_t k) {
    const int rc = check_grouped(kSegTN, rows, groups, n, k);
    if (rc != GEMM_F16_OK) return rc;
    const int splits = tn_splits(rows, groups, n, k);
    return splits > 1 ? splits * tn_part_elems(groups, n, k) * 4 : 0;
}

int gemm_f16_grouped_tn_ws(int64_t rows, int64_t groups, int64_t n, int64_t k, const void *a, const void *b,
                           const int32_t *offsets, void *c, int32_t out_f32, void *workspace, int64_t workspace_bytes,
                           void *stream) {
    const int rc = check_grouped(kSegTN, rows, groups, n, k);
    if (rc != GEMM_F16_OK) return rc;
    return grouped(kSegTN, rows, groups, n, k, a, rows, b, offsets, nullptr, 1, c, out_f32, stream, workspace,
                   workspace_bytes, tn_splits(rows, groups, n, k));
}

int64_t gemm_f16_lora_workspace(int64_t rows, int64_t n, int64_t k, int64_t adapters, int64_t rank) {
    const int rc = check_lora(rows, n, k, adapters, rank);
    if (rc != GEMM_F16_OK) return rc;
    const int64_t h = rows * lora_h_ld(rows, k, rank);
    if (!lora_few(rows, k)) return h * kSplitValue;
    // h, and x W^T, in fp32
    return (h * lora_parts(rows, k) + rows * n * lora_few_parts(k)) * 4;
}

int gemm_f16_lora_nt(int64_t rows, int64_t n, int64_t k, int64_t adapters, int64_t rank, const void *x, const void *w,
                     const void *down, const void *up, const int32_t *ids, const int32_t *order,
                     const int32_t *offsets, const float *scale, void *y, void *workspace, int64_t workspace_bytes,
                     void *stream) {
    int rc = check_lora(rows, n, k, adapters, rank);
    if (rc != GEMM_F16_OK) return rc;
    const int64_t need = gemm_f16_lora_workspace(rows, n, k, adapters, rank);
    if (workspace_bytes < need) return GEMM_F16_EINVAL;
    if (rows == 0 || n == 0) return GEMM_F16_OK;
    const Buffer bufs[] = {{y, rows * n * 2, 2, true},
                           {workspace, need, 16, true},
                           {x, rows * k * 2, 2, false},
                           {w, n * k * 2, 2, false},
                           {down, adapters * rank * k * 2, 2, false},
                           {up, adapters * rank * n * 2, 2, false},
                           {ids, rows * 4, 4, false},
                           {order, rows * 4, 4, false},
                           {offsets, (adapters + 1) * 4, 4, false},
                           {scale, scale ? adapters * 4 : 0, 4, false}};
    rc = check_buffers(bufs);
    if (rc != GEMM_F16_OK) return rc;
    int cus;
    rc = current_device(&cus);
    if (rc != GEMM_F16_OK) return rc;

    SegParams p = {};
    p.a = static_cast<const _Float16 *>(x);
    p.offsets = offsets;
    p.a_rows = rows;
    p.rows = (int32_t)rows;
    p.k = (int32_t)k;
    p.fan = 1;
    p.adapters = (int32_t)adapters;
    p.rank = (int32_t)rank;
    p.h_ld = (int32_t)lora_h_ld(rows, k, rank);
    p.scale = scale;
    // h = scale_s (x D_s^T), rows in adapter order
    SegParams d = p;
    d.b = static_cast<const _Float16 *>(down);
    d.c = workspace;
    d.index = order;
    d.groups = (int32_t)adapters;
    d.n = (int32_t)rank;
    p.b = static_cast<const _Float16 *>(w);
    p.c = y;
    p.h = static_cast<const float *>(workspace);
    p.h_split = static_cast<const char *>(workspace);
    p.up = static_cast<const _Float16 *>(up);
    p.groups = 1;
    p.n = (int32_t)n;
    if (lora_few(rows, k))
        return status(launch_lora_few(p, d, static_cast<float *>(workspace) + rows * lora_h_ld(rows, k, rank) * lora_parts(rows, k), ids, (hipStream_t)stream));
    const bool direct = direct_rows(kSegNT, d) && direct_rows(kSegNT, p);
    rc = status(direct ? launch_lora_down(d, (hipStream_t)stream)
                       : launch_lora_down_thin(d, (hipStream_t)stream));
    if (rc != GEMM_F16_OK) return rc;
    // x W^T + h U_s^T
    p.order = order;
    if (direct && rank % 4 == 0)
        return status(launch_seg_lora(pick_plan(kSegNT, false, p, cus).tile, p, (hipStream_t)stream));
    return status(launch_seg_staged(kSegNT, false, true, p, (hipStream_t)stream));
}

}  // extern "C"
