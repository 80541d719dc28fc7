// Host side of the feed-forward layer's operators: argument checks, the choice of kernel and
// the launches (see fused.h and route.h).
#include <algorithm>

#include "checks.h"
#include "device.h"
#include "fused.h"
#include "gemm_f16.h"
#include "route.h"

namespace gemm_f16 {

// gfx950's CUs.  A plan counts with them whatever the device has (a part of one, say): the sizes
// alone say what workspace a call takes, and they are asked for it with no device at hand.
constexpr int kFusedCus = 256;
constexpr int64_t kMaxSide = int64_t(1) << 30, kMaxDepth = int64_t(1) << 22, kMaxArea = int64_t(1) << 47;

static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

static bool aligned16(const void *p) { return (uintptr_t)p % 16 == 0; }

// Whether all rows are whole 128-byte lines.
static bool whole_lines(const void *p, int64_t row_bytes) { return !p || ((uintptr_t)p % 128 == 0 && row_bytes % 128 == 0); }

static int check_fused(int64_t m, int64_t n, int64_t k) {
    if (m < 0 || n < 0 || k < 0 || m >= kMaxSide || n >= kMaxSide || k >= kMaxDepth) return GEMM_F16_EINVAL;
    return below(kMaxArea, m, n) ? GEMM_F16_OK : GEMM_F16_EINVAL;
}

static TileSize tile_size(int tile) {
    switch (tile) {
        case GEMM_F16_TILE_256x256: return {256, 256};
        case GEMM_F16_TILE_256x128: return {256, 128};
        case GEMM_F16_TILE_128x256: return {128, 256};
        case GEMM_F16_TILE_128x128: return {128, 128};
        case GEMM_F16_TILE_128x64: return {128, 64};
        case GEMM_F16_TILE_64x128: return {64, 128};
        default: return {64, 64};
    }
}

// Whether the product can walk its tiles: more of them than CUs, fp16 results in whole 16-byte
// chunks, and what the kernels of fused_walk.h take (launch_walk there says why not an activation with
// a residual).
static bool walk_takes(int tile, const TileSize &ts, int cus, const FusedParams &p) {
    if ((int64_t)p.num_m * p.num_n <= cus || !p.vec || p.out_f32 || (p.residual && p.act != kActNone) ||
        (int64_t)ts.bm * p.n * 2 >= (int64_t(1) << 31))
        return false;
    if (tile == GEMM_F16_TILE_256x256) return p.k % 128 == 0 && p.k >= 256;
    return (tile == GEMM_F16_TILE_256x128 || tile == GEMM_F16_TILE_128x256) && p.k_tiles >= 3;
}

// Tile of rows that are not 16-byte aligned: their loads hold too many registers for the
// largest.
static int staged_tile(int tile) {
    switch (tile) {
        case GEMM_F16_TILE_256x256:
        case GEMM_F16_TILE_128x256: return GEMM_F16_TILE_128x256;
        case GEMM_F16_TILE_256x128:
        case GEMM_F16_TILE_128x128: return GEMM_F16_TILE_128x128;
        default: return GEMM_F16_TILE_64x64;
    }
}

// direct: 16-byte aligned rows; otherwise the tile is one of staged_tile.
static hipError_t launch_tile(bool direct, bool ring, int tile, const FusedParams &p, hipStream_t s) {
    if (!direct) {
        const bool dwords = p.k % 2 == 0 && (uintptr_t)p.a % 4 == 0 && (uintptr_t)p.b % 4 == 0;
        return launch_fused_staged(tile_size(tile), dwords, p, s);
    }
    if (ring) return launch_fused_ring(p, s);
    switch (tile) {
        case GEMM_F16_TILE_256x256: return launch_fused_256x256(p, s);
        case GEMM_F16_TILE_256x128: return launch_fused_256x128(p, s);
        case GEMM_F16_TILE_128x256: return launch_fused_128x256(p, s);
        case GEMM_F16_TILE_128x128: return launch_fused_128x128(p, s);
        case GEMM_F16_TILE_128x64: return launch_fused_128x64(p, s);
        case GEMM_F16_TILE_64x128: return launch_fused_64x128(p, s);
        default: return launch_fused_64x64(p, s);
    }
}

// Modelled time (us) of a product, or of one in parts of K:
//     c + a K-tiles of a part x (1, or e share where more than a workgroup falls to a CU) + b share
// with share the workgroups per CU, no less for the K loop than 0.175 us for each MB of A and B, and
// up to 2.5 times that where CUs are left over; with parts, 1.6 + 0.12 a part + 0.123 for each MB of
// their sums, written and read, for the join.  Least-squares fits, in relative error, to 1852 timings
// of 120 shapes (rows 17 to 16384, N 8 to 8192, K 64 to 8192, six copies of the inputs in turn) on
// MI355X, the join's and the left-over CUs' to 48 of them (rows 24 to 1024).
struct FusedCost {
    int tile, bm, bn;
    bool ring;
    double c, a, e, b;
    bool rounds;  // share in whole rounds: a workgroup has its CU alone, and a tile is long
};

static int64_t fused_tiles(const FusedCost &f, int64_t m, int64_t n) { return cdiv(m, f.bm) * cdiv(n, f.bn); }

static double fused_us(const FusedCost &f, int64_t tiles, int64_t m, int64_t n, int64_t k, int parts, int part_kt) {
    double share = (double)(tiles * parts) / kFusedCus;
    if (f.rounds && share > 1) share = (double)cdiv(tiles * parts, kFusedCus);
    const double loop = f.a * part_kt * (share > 1 ? std::max(1.0, f.e * share) : 1.0);
    const double inputs = 0.175 * 2e-6 * (double)((m + n) * k) * std::min(std::max(1.0, 1 / share), 2.5);
    const double join = parts > 1 ? 1.6 + 0.12 * parts + 0.123 * 8e-6 * (double)(m * n) * parts : 0;
    return f.c + std::max(loop, inputs) + f.b * share + join;
}

// Block tile of a product, and the parts of its K (1: none) of part_kt K-tiles each; or the
// few-row kernel.  By the sizes alone: they say what workspace a call takes.
struct FusedPlan {
    int tile;
    bool ring;
    int parts, part_kt;
    double us;
    bool few;
};

// Takes the parts of K into which `f` is divided at less than best's time, if there are any; `whole`:
// or not divided.
static void fused_parts(const FusedCost &f, int64_t m, int64_t n, int64_t k, bool whole, FusedPlan &best) {
    const int64_t tiles = fused_tiles(f, m, n);
    const int k_tiles = (int)cdiv(k, 64);
    for (int parts : {1, 2, 3, 4, 6, 8, 12, 16}) {
        if (parts == 1 ? !whole : 2 * parts > k_tiles || tiles * parts > 10 * kFusedCus) continue;
        const int part_kt = (k_tiles + parts - 1) / parts, really = (k_tiles + part_kt - 1) / part_kt;
        const double us = fused_us(f, tiles, m, n, k, really, part_kt);
        if (us < best.us) best = {f.tile, f.ring, really, part_kt, us, false};
    }
}

// Rows that are not 16-byte aligned, as K says: a fit to 396 timings of 31 shapes (rows 24 to
// 16384, K 333 to 4097), whose choice took 1.01 of the fastest variant's time in the geometric mean;
// 719 x 784 x 1899 takes 17.7 us, 23.9 with the aligned rows' choice, 128 x 4096 x 4097 23 and 29.6.
static FusedPlan fused_staged_plan(int64_t m, int64_t n, int64_t k) {
    static const FusedCost costs[] = {
        {GEMM_F16_TILE_64x64, 64, 64, false, 4.77, 0.373, 1.163, 2.15, false},
        {GEMM_F16_TILE_128x128, 128, 128, false, 7.73, 0.734, 1.526, 3.02, false},
        {GEMM_F16_TILE_128x256, 128, 256, false, 9.38, 1.171, 1.449, 3.96, true},
    };
    FusedPlan best = {GEMM_F16_TILE_128x256, false, 1, (int)cdiv(k, 64), 1e300, false};
    for (const FusedCost &f : costs) fused_parts(f, m, n, k, true, best);
    return best;
}

// The dense product's choice of tile, unless the model has one in parts of K, or on the ring, at
// less than 0.9 of its time.  On those 120 shapes the plan took 1.034 of the fastest variant's time
// in the geometric mean (the dense choice alone: 1.28); 128 rows of 4096 x 4096 take 16.7 us in 3
// parts, 26 undivided; 1024 of 64 x 4096 11 and 26; 512 of 4096 x 4096 32, undivided.
static FusedPlan fused_tile_plan(int64_t m, int64_t n, int64_t k) {
    if (k % 8 != 0) return fused_staged_plan(m, n, k);
    static const FusedCost costs[] = {
        {GEMM_F16_TILE_64x64, 64, 64, false, 2.41, 0.358, 1.253, 1.63, false},
        {GEMM_F16_TILE_64x128, 64, 128, false, 3.19, 0.408, 1.438, 2.11, false},
        {GEMM_F16_TILE_128x64, 128, 64, false, 3.12, 0.412, 1.493, 2.02, false},
        {GEMM_F16_TILE_128x256, 128, 256, false, 7.56, 0.645, 2.536, 4.27, false},
        {GEMM_F16_TILE_128x128, 128, 128, false, 4.99, 0.444, 1.519, 3.56, false},  // from here on also in parts
        {GEMM_F16_TILE_256x128, 256, 128, false, 7.45, 0.619, 1.896, 4.03, false},
        {GEMM_F16_TILE_64x64, 64, 64, true, 4.14, 0.294, 0.808, 1.00, false},
    };
    const int k_tiles = (int)cdiv(k, 64);
    FusedPlan plan = {auto_tile(m, n, k, kFusedCus), false, 1, k_tiles, 1e300, false};
    double whole = 1e300;  // 256 x 256: enough tiles, or nearly
    for (const FusedCost &f : costs)
        if (f.tile == plan.tile && !f.ring) whole = fused_us(f, fused_tiles(f, m, n), m, n, k, 1, k_tiles);
    if (whole == 1e300) return plan;
    plan.us = whole;
    // One tile's width holds all of the columns (rows), and the rows' (columns') bytes, read
    // once, are what the time is: the ring keeps more of them in flight (16384 rows of 64 x 4096:
    // 31.6 us, 44.9 with two stages).
    if (plan.tile == GEMM_F16_TILE_64x64 && std::min(m, n) <= 64 && (m + n) * k * 2 >= int64_t(32) << 20) {
        plan.ring = true;
        plan.us = whole = fused_us(costs[6], fused_tiles(costs[6], m, n), m, n, k, 1, k_tiles);
    }
    FusedPlan best = {0, false, 1, k_tiles, 0.9 * whole, false};
    for (const FusedCost &f : costs)
        if (f.ring || f.tile == GEMM_F16_TILE_128x128 || f.tile == GEMM_F16_TILE_256x128) fused_parts(f, m, n, k, f.ring, best);
    return best.tile ? best : plan;
}

// The few-row kernel takes one and two rows always, up to 64 where the model has it ahead.  Its time
// is what each workgroup of 16 columns reads of A, for each round of them over the CUs (whole
// rounds where K takes a CU's 16 waves), and B's bytes.  With it 160 timings (rows 3 to 64, N 64 to
// 16384, K 200 to 8192) are 1.014 of the faster way's in the geometric mean; 16384 x 4096 takes 32
// rows 56 us there and 31 on a tile, 4096 x 1024 6.4 and 8.6.
static FusedPlan fused_plan(int64_t m, int64_t n, int64_t k) {
    const FusedPlan few = {0, false, 1, 0, 0, true};
    if (k >= 8 && m <= 2) return few;
    const FusedPlan plan = fused_tile_plan(m, n, k);
    if (k < 8 || m > kFusedFewRows) return plan;
    double rounds = std::max(1.0, (double)n / (16 * kFusedCus));
    if (k > 2048) rounds = (double)cdiv(n, 16 * kFusedCus);
    const double reads = k % 8 ? 13 + 0.8 * (double)m : 4.5 + 0.22 * (double)m;  // (chunks across lines)
    const double us = 2.4 + rounds * (0.8 + (double)k / 4096 * reads) + 0.075 * 2e-6 * (double)(n * k);
    return us < plan.us ? few : plan;
}

// Bytes of workspace.
static int64_t fused_need(const FusedPlan &plan, int64_t m, int64_t n) {
    return plan.parts > 1 ? plan.parts * m * n * 4 : 0;
}

static int fused(int64_t m, int64_t n, int64_t k, const void *a, const void *b, void *c, const gemm_f16_epilogue &e,
                 void *workspace, int64_t workspace_bytes, hipStream_t s) {
    int rc = check_fused(m, n, k);
    if (rc != GEMM_F16_OK) return rc;
    if (e.act < GEMM_F16_ACT_NONE || e.act > GEMM_F16_ACT_LAST || e.bias_f32 < 0 || e.bias_f32 > 1 || e.out_f32 < 0 ||
        e.out_f32 > 1)
        return GEMM_F16_EINVAL;
    FusedPlan plan = {};
    if (m > 0 && n > 0 && k > 0) plan = fused_plan(m, n, k);
    const int64_t need = fused_need(plan, m, n);
    if (workspace_bytes < need) return GEMM_F16_EINVAL;
    if (m == 0 || n == 0) return GEMM_F16_OK;
    const int es = e.out_f32 ? 4 : 2, bs = e.bias_f32 ? 4 : 2;
    // C may be the residual itself: each element is read and written by one thread
    const bool in_place = e.residual == c;
    const Buffer bufs[] = {{c, m * n * es, es, true},
                           {e.pre, e.pre ? m * n * 2 : 0, 2, true},
                           {workspace, need, 16, true},
                           {a, m * k * 2, 2, false},
                           {b, n * k * 2, 2, false},
                           {e.bias, e.bias ? n * bs : 0, bs, false},
                           {e.residual, e.residual && !in_place ? m * n * es : 0, es, false}};
    rc = check_buffers(bufs);
    if (rc != GEMM_F16_OK) return rc;
    int cus;
    rc = current_device(&cus);
    if (rc != GEMM_F16_OK) return rc;

    FusedParams p = {};
    p.a = static_cast<const _Float16 *>(a);
    p.b = static_cast<const _Float16 *>(b);
    p.c = c;
    p.m = (int32_t)m;
    p.n = (int32_t)n;
    p.k = (int32_t)k;
    p.k_tiles = p.part_kt = (int32_t)cdiv(k, 64);
    p.parts = 1;
    p.bias = e.bias;
    p.residual = e.residual;
    p.pre = static_cast<_Float16 *>(e.pre);
    p.sums = static_cast<float *>(workspace);
    p.act = e.act;
    p.bias_f32 = e.bias_f32;
    p.out_f32 = e.out_f32;
    p.vec = n % 8 == 0 && aligned16(c) && aligned16(e.bias) && aligned16(e.residual) && aligned16(e.pre);
    // as the dense product's: device scope while everything fits in the 256 MiB Infinity Cache, past
    // it streaming stores on rows of whole 128-byte lines and the default on others (60000 x 1544 x 512
    // with silu and pre 240 us, 350 streaming; 16384 x 4104 x 2048 with gelu_tanh and pre 320 and 355; 16384
    // x 4128 x 2048 in fp32 with pre, whose rows alone end inside a line, 314 and 351)
    const int64_t each = es * (e.residual ? 2 : 1) + (e.pre ? 2 : 0);
    p.c_store = kStoreDefault;
    if (p.vec && (m + n) * k * 2 + m * n * each <= (int64_t(256) << 20))
        p.c_store = kStoreDevice;
    else if (p.vec && whole_lines(c, n * es) && whole_lines(e.pre, n * 2))
        p.c_store = kStoreStream;
    if (k == 0) {
        p.parts = 0;
        return status(launch_fused_join(p, s));
    }
    if (plan.few) return status(launch_fused_few(p, s));
    const bool direct = k % 8 == 0 && aligned16(a) && aligned16(b);
    const int tile = direct ? plan.tile : staged_tile(plan.tile);
    const TileSize ts = tile_size(tile);
    p.num_m = (int32_t)cdiv(m, ts.bm);
    p.num_n = (int32_t)cdiv(n, ts.bn);
    if ((int64_t)p.num_m * p.num_n >= (int64_t(1) << 31)) return GEMM_F16_EINVAL;
    p.swizzle = 4;
    p.xcd = gemm_f16_select_xcd(p.num_m, p.num_n, p.swizzle, cus);
    if (plan.parts > 1) {
        FusedParams q = p;
        q.parts = plan.parts;
        q.part_kt = plan.part_kt;
        const hipError_t e = launch_tile(direct, plan.ring, tile, q, s);
        if (e != hipSuccess) return status(e);
        return status(launch_fused_join(q, s));
    }
    if (direct && !plan.ring && walk_takes(tile, ts, cus, p)) {
        switch (tile) {
            case GEMM_F16_TILE_256x256: return status(launch_fused_walk_256x256(p, cus, s));
            case GEMM_F16_TILE_256x128: return status(launch_fused_walk_256x128(p, cus, s));
            default: return status(launch_fused_walk_128x256(p, cus, s));
        }
    }
    return status(launch_tile(direct, plan.ring, tile, p, s));
}

static int check_routing(int64_t tokens, int64_t experts, int64_t fan, int32_t logits_f32, const gemm_f16_routing *r) {
    if (!r) return GEMM_F16_ENULL;
    if (tokens < 0 || tokens >= kMaxSide || experts < 1 || experts > kRouteExperts || fan < 1 || fan > kRouteFan ||
        fan > experts || logits_f32 < 0 || logits_f32 > 1)
        return GEMM_F16_EINVAL;
    if (r->score < GEMM_F16_SCORE_SOFTMAX || r->score > GEMM_F16_SCORE_SIGMOID || r->renormalize < 0 || r->renormalize > 1 ||
        !(r->scale - r->scale == 0.0f))
        return GEMM_F16_EINVAL;
    return GEMM_F16_OK;
}

static RouteParams route_params(int64_t tokens, int64_t experts, int64_t fan, const void *logits, int32_t logits_f32,
                                const gemm_f16_routing &r) {
    RouteParams p = {};
    p.logits = logits;
    p.tokens = tokens;
    p.experts = (int32_t)experts;
    p.fan = (int32_t)fan;
    p.f32 = logits_f32;
    p.sigmoid = r.score == GEMM_F16_SCORE_SIGMOID;
    p.renormalize = r.renormalize;
    p.scale = r.scale;
    p.groups = p.top_groups = p.group_top = 1;
    p.vec = experts % 4 == 0 && aligned16(logits);
    return p;
}

static int check_combine(int64_t tokens, int64_t fan, int64_t n) {
    if (tokens < 0 || fan < 1 || n < 0 || tokens >= kMaxSide || fan >= kMaxSide || n >= kMaxSide) return GEMM_F16_EINVAL;
    if (!below(kMaxSide, tokens, fan) || !below(kMaxArea, tokens * fan, n)) return GEMM_F16_EINVAL;
    return GEMM_F16_OK;
}

}  // namespace gemm_f16

using namespace gemm_f16;

extern "C" {

int64_t gemm_f16_fused_workspace(int64_t m, int64_t n, int64_t k) {
    const int rc = check_fused(m, n, k);
    if (rc != GEMM_F16_OK || m == 0 || n == 0 || k == 0) return rc;
    return fused_need(fused_plan(m, n, k), m, n);
}

int gemm_f16_fused_nt(int64_t m, int64_t n, int64_t k, const void *a, const void *b, void *c,
                      const gemm_f16_epilogue *epilogue, void *workspace, int64_t workspace_bytes, void *stream) {
    static const gemm_f16_epilogue none = {};
    return fused(m, n, k, a, b, c, epilogue ? *epilogue : none, workspace, workspace_bytes, (hipStream_t)stream);
}

int64_t gemm_f16_fused_grad_workspace(int64_t m, int64_t n) {
    const int rc = check_fused(m, n, 0);
    if (rc != GEMM_F16_OK) return rc;
    const int parts = m > 0 && n > 0 ? fused_grad_parts(m, n) : 1;
    return parts > 1 ? parts * n * 4 : 0;
}

int gemm_f16_fused_grad(int64_t m, int64_t n, const void *dy, int32_t dy_f32, const void *pre, int32_t act, void *dz,
                        float *dbias, void *workspace, int64_t workspace_bytes, void *stream) {
    int rc = check_fused(m, n, 0);
    if (rc != GEMM_F16_OK) return rc;
    if (act < GEMM_F16_ACT_NONE || act > GEMM_F16_ACT_LAST || dy_f32 < 0 || dy_f32 > 1) return GEMM_F16_EINVAL;
    const int64_t need = dbias ? gemm_f16_fused_grad_workspace(m, n) : 0;
    if (workspace_bytes < need) return GEMM_F16_EINVAL;
    if (n == 0 || (!dz && !dbias) || (m == 0 && !dbias)) return GEMM_F16_OK;
    const int ds = dy_f32 ? 4 : 2;
    // dz may be dy itself, where both are fp16: each element is read and written by one thread
    const bool in_place = dz == dy && !dy_f32;
    const Buffer bufs[] = {{dz, dz ? m * n * 2 : 0, 2, true},
                           {dbias, dbias ? n * 4 : 0, 4, true},
                           {workspace, need, 16, true},
                           {dy, in_place ? 0 : m * n * ds, ds, false},
                           {pre, act != GEMM_F16_ACT_NONE ? m * n * 2 : 0, 2, false}};
    rc = check_buffers(bufs);
    if (rc != GEMM_F16_OK) return rc;
    int cus;
    rc = current_device(&cus);
    if (rc != GEMM_F16_OK) return rc;
    FusedGradParams p = {};
    p.dy = dy;
    p.pre = static_cast<const _Float16 *>(pre);
    p.dz = static_cast<_Float16 *>(dz);
    p.dbias = dbias;
    p.sums = static_cast<float *>(workspace);
    p.m = m;
    p.n = n;
    p.act = act;
    p.dy_f32 = dy_f32;
    p.parts = m > 0 ? fused_grad_parts(m, n) : 1;
    return status(launch_fused_grad(p, (hipStream_t)stream));
}

int gemm_f16_route(int64_t tokens, int64_t experts, int64_t fan, const void *logits, int32_t logits_f32, const float *bias,
                   const gemm_f16_routing *routing, int32_t *ids, float *gates, void *stream) {
    int rc = check_routing(tokens, experts, fan, logits_f32, routing);
    if (rc != GEMM_F16_OK) return rc;
    const gemm_f16_routing &r = *routing;
    if (r.groups < 1 || r.groups > kRouteGroups || experts % r.groups != 0 || r.top_groups < 1 || r.top_groups > r.groups ||
        r.group_top < 1 || r.group_top > 2 || fan > experts / r.groups * r.top_groups)
        return GEMM_F16_EINVAL;
    if (tokens == 0) return GEMM_F16_OK;
    const int es = logits_f32 ? 4 : 2;
    const Buffer bufs[] = {{ids, tokens * fan * 4, 4, true},
                           {gates, tokens * fan * 4, 4, true},
                           {logits, tokens * experts * es, es, false},
                           {bias, bias ? experts * 4 : 0, 4, false}};
    rc = check_buffers(bufs);
    if (rc != GEMM_F16_OK) return rc;
    int cus;
    rc = current_device(&cus);
    if (rc != GEMM_F16_OK) return rc;
    RouteParams p = route_params(tokens, experts, fan, logits, logits_f32, r);
    p.bias = bias;
    p.bias_vec = experts % 4 == 0 && aligned16(bias);
    p.ids = ids;
    p.gates = gates;
    p.groups = r.groups;
    p.top_groups = r.top_groups;
    p.group_top = r.group_top;
    return status(launch_route(p, (hipStream_t)stream));
}

int gemm_f16_route_grad(int64_t tokens, int64_t experts, int64_t fan, const void *logits, int32_t logits_f32,
                        const int32_t *ids, const float *dgates, const gemm_f16_routing *routing, void *dlogits,
                        void *stream) {
    int rc = check_routing(tokens, experts, fan, logits_f32, routing);
    if (rc != GEMM_F16_OK) return rc;
    if (tokens == 0) return GEMM_F16_OK;
    const int es = logits_f32 ? 4 : 2;
    const Buffer bufs[] = {{dlogits, tokens * experts * es, es, true},
                           {logits, tokens * experts * es, es, false},
                           {ids, tokens * fan * 4, 4, false},
                           {dgates, tokens * fan * 4, 4, false}};
    rc = check_buffers(bufs);
    if (rc != GEMM_F16_OK) return rc;
    int cus;
    rc = current_device(&cus);
    if (rc != GEMM_F16_OK) return rc;
    RouteParams p = route_params(tokens, experts, fan, logits, logits_f32, *routing);
    p.ids = const_cast<int32_t *>(ids);
    p.dgates = dgates;
    p.dlogits = dlogits;
    p.vec = p.vec && aligned16(dlogits);
    return status(launch_route_grad(p, (hipStream_t)stream));
}

int gemm_f16_combine_rows(int64_t tokens, int64_t fan, int64_t n, int64_t groups, const void *rows, int32_t rows_f32,
                          const int32_t *inverse, const int32_t *offsets, const float *gates, const void *residual, void *y,
                          int32_t y_f32, void *stream) {
    int rc = check_combine(tokens, fan, n);
    if (rc != GEMM_F16_OK) return rc;
    if (groups < 1 || groups >= kMaxSide || rows_f32 < 0 || rows_f32 > 1 || y_f32 < 0 || y_f32 > 1) return GEMM_F16_EINVAL;
    if (tokens == 0 || n == 0) return GEMM_F16_OK;
    const int rs = rows_f32 ? 4 : 2, ys = y_f32 ? 4 : 2;
    const bool in_place = residual == y;  // each element is read and written by one thread
    const Buffer bufs[] = {{y, tokens * n * ys, ys, true},
                           {rows, tokens * fan * n * rs, rs, false},
                           {inverse, tokens * fan * 4, 4, false},
                           {offsets, (groups + 1) * 4, 4, false},
                           {gates, gates ? tokens * fan * 4 : 0, 4, false},
                           {residual, residual && !in_place ? tokens * n * ys : 0, ys, false}};
    rc = check_buffers(bufs);
    if (rc != GEMM_F16_OK) return rc;
    int cus;
    rc = current_device(&cus);
    if (rc != GEMM_F16_OK) return rc;
    CombineParams p = {};
    p.rows = rows;
    p.inverse = inverse;
    p.last = offsets + groups;
    p.gates = gates;
    p.residual = residual;
    p.y = y;
    p.tokens = tokens;
    p.places = tokens * fan;
    p.fan = (int32_t)fan;
    p.n = (int32_t)n;
    p.rows_f32 = rows_f32;
    p.y_f32 = y_f32;
    return status(launch_combine(p, (hipStream_t)stream));
}

int gemm_f16_combine_rows_grad(int64_t tokens, int64_t fan, int64_t n, int64_t groups, const void *dy, int32_t dy_f32,
                               const void *rows, int32_t rows_f32, const int32_t *inverse, const int32_t *offsets,
                               const float *gates, void *drows, int32_t drows_f32, float *dgates, void *stream) {
    int rc = check_combine(tokens, fan, n);
    if (rc != GEMM_F16_OK) return rc;
    if (groups < 1 || groups >= kMaxSide || dy_f32 < 0 || dy_f32 > 1 || rows_f32 < 0 || rows_f32 > 1 || drows_f32 < 0 ||
        drows_f32 > 1)
        return GEMM_F16_EINVAL;
    if (tokens == 0 || (!drows && !dgates) || (n == 0 && !dgates)) return GEMM_F16_OK;
    const int rs = rows_f32 ? 4 : 2, ys = dy_f32 ? 4 : 2, ds = drows_f32 ? 4 : 2;
    const Buffer bufs[] = {{drows, drows ? tokens * fan * n * ds : 0, ds, true},
                           {dgates, dgates ? tokens * fan * 4 : 0, 4, true},
                           {dy, tokens * n * ys, ys, false},
                           {rows, dgates ? tokens * fan * n * rs : 0, rs, false},
                           {inverse, tokens * fan * 4, 4, false},
                           {offsets, (groups + 1) * 4, 4, false},
                           {gates, gates ? tokens * fan * 4 : 0, 4, false}};
    rc = check_buffers(bufs);
    if (rc != GEMM_F16_OK) return rc;
    int cus;
    rc = current_device(&cus);
    if (rc != GEMM_F16_OK) return rc;
    CombineParams p = {};
    p.rows = rows;
    p.inverse = inverse;
    p.last = offsets + groups;
    p.gates = gates;
    p.y = const_cast<void *>(dy);
    p.drows = drows;
    p.dgates = dgates;
    p.tokens = tokens;
    p.places = tokens * fan;
    p.fan = (int32_t)fan;
    p.n = (int32_t)n;
    p.rows_f32 = rows_f32;
    p.y_f32 = dy_f32;
    p.drows_f32 = drows_f32;
    return status(launch_combine_grad(p, (hipStream_t)stream));
}

}  // extern "C"
