// Host side of the segmented products: argument checks, the choice of
// kernel and the launches (see segments.h).
#include "segments.h"

#include <algorithm>
#include <cstdlib>

#include "device.h"
#include "gemm_f16.h"

namespace gemm_f16 {

constexpr int64_t kMaxRows = int64_t(1) << 30, kMaxK = int64_t(1) << 22, kMaxNMajor = int64_t(1) << 25;
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
    if (kind != kSegNT && p.n % 8 != 0) return false;
    return !(p.index || p.order) || p.a_rows * p.k * 2 < (int64_t(1) << 31);
}

static int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Block tile with the smallest modelled time c + a rounds k_tiles + b
// tiles / cus (us; the dense product's model, auto_tile in gemm_f16.hip),
// over the row tiles to expect: half a tile more per segment than the rows
// fill.
static int pick_tile(int kind, const SegParams &p, int cus) {
    struct Cand {
        int id, bm, bn;
        double c, a, b;
    };
    static const Cand cands[] = {
        {kSeg256x256, 256, 256, 8.280, 1.115, 6.212}, {kSeg256x128, 256, 128, 5.825, 0.663, 3.036},
        {kSeg128x256, 128, 256, 5.856, 0.661, 2.886}, {kSeg128x128, 128, 128, 4.492, 0.436, 1.517},
        {kSeg64x128, 64, 128, 3.545, 0.391, 0.780},   {kSeg32x128, 32, 128, 3.3, 0.30, 0.45},
    };
#ifdef GEMM_F16_SEG_TUNE
    if (const char *force = std::getenv("SEG_TILE")) return std::atoi(force);
#endif
    const int64_t segments = std::min<int64_t>(p.groups, p.rows);
    int best = kSeg128x128;
    double best_t = 1e300;
    for (const Cand &c : cands) {
        if (kind == kSegTN && c.bm < 128) continue;
        double m_tiles;
        int64_t k_tiles;
        if (kind == kSegTN) {
            m_tiles = (double)(cdiv64(p.k, c.bm) * p.groups);
            k_tiles = cdiv64(cdiv64(p.rows, p.groups), 64);
        } else {
            m_tiles = p.order || p.groups == 1 ? (double)cdiv64(p.rows, c.bm)
                                               : (double)p.rows / c.bm + 0.5 * (double)segments;
            k_tiles = cdiv64(p.k, 64);
        }
        const double tiles = m_tiles * (double)cdiv64(p.n, c.bn), rounds = (double)(int64_t)((tiles + cus - 1) / cus);
        const double t = c.c + c.a * rounds * (double)k_tiles + c.b * tiles / cus;
        if (t < best_t) {
            best_t = t;
            best = c.id;
        }
    }
    return best;
}

static int grouped(int kind, int64_t rows, int64_t groups, int64_t n, int64_t k, const void *a, int64_t a_rows,
                   const void *b, const int32_t *offsets, const int32_t *index, int64_t fan, void *c, int32_t out_f32,
                   void *workspace, int64_t workspace_bytes, void *stream) {
    int rc = check_grouped(kind, rows, groups, n, k);
    if (rc != GEMM_F16_OK) return rc;
    if (a_rows < 0 || a_rows >= kMaxRows || fan < 1 || fan >= kMaxRows || out_f32 < 0 || out_f32 > 1)
        return GEMM_F16_EINVAL;
    if (!index && a_rows < rows) return GEMM_F16_EINVAL;
    const int64_t need = gemm_f16_grouped_workspace(kind, rows, groups, n, k);
    if (workspace_bytes < need) return GEMM_F16_EINVAL;
    const int64_t out = kind == kSegTN ? groups * n * k : rows * n;
    if (out == 0) return GEMM_F16_OK;
    const int es = out_f32 ? 4 : 2;
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
#ifdef GEMM_F16_SEG_TUNE
    if (kind == kSegNT && std::getenv("SEG_TILE") && std::atoi(std::getenv("SEG_TILE")) == kSegTiles)
        return status(launch_seg_thin(out_f32 != 0, p, (hipStream_t)stream));
#endif
    if (kind == kSegNT && k >= 8 && rows <= 16 * std::min(groups, rows)) return status(launch_seg_thin(out_f32 != 0, p, (hipStream_t)stream));
    if (direct_rows(kind, p)) {
        const int tile = pick_tile(kind, p, cus);
        hipError_t e;
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

// h's row pitch: whole 16-byte stores, and for lora_tiles whole 32-wide steps
static int64_t lora_h_ld(int64_t rows, int64_t k, int64_t rank) {
    const int64_t to = lora_few(rows, k) ? 4 : 32;
    return (rank + to - 1) / to * to;
}

// Slices of K that h is summed in: 64 x 64 tiles alone fill too few CUs.
static int lora_parts(int64_t rows, int64_t k) {
    if (lora_few(rows, k)) return 1;
#ifdef GEMM_F16_SEG_TUNE
    if (const char *f = std::getenv("SEG_PARTS")) return std::atoi(f);
#endif
    const int64_t tiles = (rows + 63) / 64;
    int parts = 1;
    while (parts < 4 && tiles * parts < 256 && k >= parts * 1024) parts *= 2;
    return parts;
}

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

int64_t gemm_f16_grouped_workspace(int32_t kind, int64_t rows, int64_t groups, int64_t n, int64_t k) {
    const int rc = check_grouped(kind, rows, groups, n, k);
    return rc != GEMM_F16_OK ? rc : 0;
}

int gemm_f16_grouped_nt(int64_t rows, int64_t groups, int64_t n, int64_t k, const void *a, int64_t a_rows,
                        const void *b, const int32_t *offsets, const int32_t *index, int64_t fan, void *c,
                        int32_t out_f32, void *workspace, int64_t workspace_bytes, void *stream) {
    return grouped(kSegNT, rows, groups, n, k, a, a_rows, b, offsets, index, fan, c, out_f32, workspace,
                   workspace_bytes, stream);
}

int gemm_f16_grouped_nn(int64_t rows, int64_t groups, int64_t n, int64_t k, const void *a, const void *b,
                        const int32_t *offsets, void *c, int32_t out_f32, void *workspace, int64_t workspace_bytes,
                        void *stream) {
    return grouped(kSegNN, rows, groups, n, k, a, rows, b, offsets, nullptr, 1, c, out_f32, workspace, workspace_bytes,
                   stream);
}

int gemm_f16_grouped_tn(int64_t rows, int64_t groups, int64_t n, int64_t k, const void *a, const void *b,
                        const int32_t *offsets, void *c, int32_t out_f32, void *workspace, int64_t workspace_bytes,
                        void *stream) {
    return grouped(kSegTN, rows, groups, n, k, a, rows, b, offsets, nullptr, 1, c, out_f32, workspace, workspace_bytes,
                   stream);
}

int64_t gemm_f16_lora_workspace(int64_t rows, int64_t n, int64_t k, int64_t adapters, int64_t rank) {
    const int rc = check_lora(rows, n, k, adapters, rank);
    if (rc != GEMM_F16_OK) return rc;
    // h, and x W^T in fp32 for few rows
    return rows * lora_h_ld(rows, k, rank) * lora_parts(rows, k) * 4 + (lora_few(rows, k) ? rows * n * 4 : 0);
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
    p.up = static_cast<const _Float16 *>(up);
    p.groups = 1;
    p.n = (int32_t)n;
    if (lora_few(rows, k))
        return status(launch_lora_few(p, d, static_cast<float *>(workspace) + rows * lora_h_ld(rows, k, rank), ids, (hipStream_t)stream));
    const bool direct = direct_rows(kSegNT, d) && direct_rows(kSegNT, p);
    p.h_parts = direct ? lora_parts(rows, k) : 1;
    rc = status(direct ? launch_lora_down(d, p.h_parts, (hipStream_t)stream)
                       : launch_lora_down_thin(d, (hipStream_t)stream));
    if (rc != GEMM_F16_OK) return rc;
    // x W^T + h U_s^T
    p.order = order;
    if (direct && rank % 4 == 0)
        return status(launch_seg_lora(pick_tile(kSegNT, p, cus), p, (hipStream_t)stream));
    return status(launch_seg_staged(kSegNT, false, true, p, (hipStream_t)stream));
}

}  // extern "C"
