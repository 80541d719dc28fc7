/*
 * gemm_f16.h - C ABI of the MI355X (gfx950) fp16 GEMM library libgemm_f16.so.
 *
 * The operation is the tiled dense GEMM of the Tilus Hopper matmul tutorial,
 * "1. WGMMA: Hopper's Asynchronous Tensor Core", section "The Full Kernel":
 *
 *     C[m][n] = fp16( sum_{k<K} A[m][k] * B[n][k] )      0 <= m < M, 0 <= n < N
 *
 * with A viewed as [M,K] and B as [N,K] (the product uses B transposed), an
 * fp32 accumulator that starts at zero, and one cast of the accumulator to
 * fp16 (round to nearest, ties to even) before C is stored.  C is
 * overwritten; there is no alpha/beta.
 *
 * Layouts (all dense, no strides):
 *   a  fp16 [M,K] row-major      element (m,k) at a[m*K + k]
 *   b  fp16 [N,K] row-major      element (n,k) at b[n*K + k]   ("K-major")
 *   c  fp16 [M,N] row-major      element (m,n) at c[m*N + n]
 * fp16 is IEEE 754 binary16.  Pointers are device pointers (memory the HIP
 * runtime allocated on the current device, e.g. through PyTorch).
 *
 * Ownership: the caller owns every buffer.  The library allocates no device
 * memory and keeps no pointer after the call returns; the dense products need
 * no workspace, the segmented ones (at the end of this file) take the
 * caller's.  c must not overlap a or b.
 *
 * Asynchrony: the work is enqueued on `stream` (a hipStream_t passed as
 * void*; NULL is the null stream) and the call returns without waiting.
 * Completion is the caller's business (stream or event synchronisation).
 *
 * Threads: every entry point may be called from several host threads at
 * once.  The only state the library keeps is a per-device cache of the
 * device's architecture and compute-unit count, filled on first use, and
 * per host thread the XCD setting of the last grid of one tile per CU
 * (gemm_f16_select_xcd).
 *
 * Errors: every entry point returns 0 on success or one of the negative
 * GEMM_F16_E* codes below; gemm_f16_status_string() names them.  Argument
 * checks run before any HIP call, so an invalid call has no effect.  The
 * library never exits the process.
 */
#ifndef GEMM_F16_H
#define GEMM_F16_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
    GEMM_F16_OK = 0,
    GEMM_F16_EINVAL = -1,     /* negative size, M or N >= 2^30, M*N >= 2^47, K >= 2^22, bad option */
    GEMM_F16_ENULL = -2,      /* null pointer with a non-empty extent */
    GEMM_F16_EALIGN = -3,     /* pointer not aligned to its element size (2 or 4 bytes) */
    GEMM_F16_EDEVICE = -4,    /* current device is not gfx950 */
    GEMM_F16_EHIP = -5,       /* a HIP runtime call or the kernel launch failed */
    GEMM_F16_EOVERLAP = -6    /* the output overlaps a or b */
};

/*
 * C = fp16(A * B^T) with fp32 accumulation (see the top of this file).
 *
 * m, n, k >= 0; m, n < 2^30; m*n < 2^47; k < 2^22.
 * m == 0 or n == 0: returns GEMM_F16_OK and launches nothing.
 * k == 0: C is filled with +0 (the zero accumulator is stored).
 * Sizes that are not multiples of the block tile are handled: elements of A
 * and B outside [M,K] / [N,K] are read as zero and elements of C outside
 * [M,N] are never written.
 * Speed: K % 8 == 0 with 16-byte aligned A and B loads the operands straight
 * into LDS; any other K or alignment goes through registers, at roughly
 * 0.55-0.7 of that speed on large shapes.
 */
int gemm_f16_nt(int64_t m, int64_t n, int64_t k, const void *a, const void *b,
                void *c, void *stream);

/*
 * Launch options for gemm_f16_nt_ex (tuning, determinism tests).
 *   tile     0 = automatic choice by shape; otherwise one of the
 *            GEMM_F16_TILE_* block-tile configurations.
 *   swizzle  tile-columns per rasterization group (the swizzle_size of
 *            "4. Pipeline Abstraction and Two Consumer Warp Groups", section
 *            "Tile Rasterization"); 0 = library default, 1 = plain grid.
 *   xcd      1 = give each of the 8 XCDs a contiguous run of tiles,
 *            0 = hardware dispatch order, -1 = library default
 *            (gemm_f16_select_xcd).
 *   variant  0 = the library's kernels.  1..7 = a kernel whose K-tile width
 *            (block_k), LDS ring depth and wave roles are those of the
 *            GEMM_F16_VARIANT_* below, one tile per workgroup (the tuning
 *            sweep's axes; "4. Pipeline Abstraction and Two Consumer Warp
 *            Groups", sections "Pipeline Depth" and "Two Consumer Warp
 *            Groups").  A variant needs C = A B^T, an explicit block tile of
 *            256x256 (variants 1, 3, 4, 5 only), 256x128 or 128x256 (not
 *            variant 7), or 128x128, K a positive multiple of its block_k,
 *            and 16-byte aligned A and B; otherwise the call returns
 *            GEMM_F16_EINVAL.
 * Every option but the variant changes only the schedule: the fp32 sum of
 * each output is taken in the same order, so results are bitwise identical
 * across options that select the same block tile.
 */
typedef struct {
    int32_t tile;
    int32_t swizzle;
    int32_t xcd;
    int32_t variant;
} gemm_f16_options;

enum {
    GEMM_F16_VARIANT_DEFAULT = 0,
    GEMM_F16_VARIANT_BK64_S2 = 1,      /* block_k 64, 2 LDS stages, every wave loads */
    GEMM_F16_VARIANT_BK64_S3 = 2,      /* block_k 64, 3 stages */
    GEMM_F16_VARIANT_BK32_S2 = 3,      /* block_k 32, 2 stages */
    GEMM_F16_VARIANT_BK32_S3 = 4,      /* block_k 32, 3 stages */
    GEMM_F16_VARIANT_BK32_S4 = 5,      /* block_k 32, 4 stages */
    GEMM_F16_VARIANT_PRODUCER_S2 = 6,  /* block_k 64, 2 stages, 4 loader waves + 4 MFMA waves */
    GEMM_F16_VARIANT_PRODUCER_S3 = 7,  /* block_k 64, 3 stages, 4 loader waves + 4 MFMA waves */
    GEMM_F16_VARIANT_LAST = 7
};

enum {
    GEMM_F16_TILE_AUTO = 0,
    GEMM_F16_TILE_256x256 = 1,     /* 4 waves, each 128x128 of C */
    GEMM_F16_TILE_128x128 = 2,     /* 4 waves, each 64x64 of C */
    GEMM_F16_TILE_64x64 = 3,       /* 4 waves, each 32x32 of C */
    GEMM_F16_TILE_256x256_W8 = 4,  /* 8 waves, each 64x128 of C */
    GEMM_F16_TILE_256x128 = 5,     /* 4 waves, each 128x64 of C */
    GEMM_F16_TILE_128x256 = 6,     /* 4 waves, each 64x128 of C */
    GEMM_F16_TILE_128x128_M16 = 7, /* 4 waves, each 64x64 of C, on v_mfma_f32_16x16x32_f16 */
    GEMM_F16_TILE_64x128 = 8,      /* 4 waves, each 32x64 of C */
    GEMM_F16_TILE_128x64 = 9,      /* 4 waves, each 64x32 of C */
    GEMM_F16_TILE_LAST = 9
};

/* gemm_f16_nt with explicit options; opt == NULL means all defaults. */
int gemm_f16_nt_ex(int64_t m, int64_t n, int64_t k, const void *a, const void *b,
                   void *c, void *stream, const gemm_f16_options *opt);

/*
 * The second contract, that of the day-78 listing "wgmma_gemm.cu" (its
 * kernel, its B layout and its fp32 output):
 *
 *     D[m][n] = sum_{k<K} A[m][k] * B[k][n]      fp32 accumulation, fp32 out
 *
 *   a  fp16 [M,K] row-major      element (m,k) at a[m*K + k]
 *   b  fp16 [K,N] row-major      element (k,n) at b[k*N + n]
 *   d  fp32 [M,N] row-major      element (m,n) at d[m*N + n], 4-byte aligned
 *
 * D is the fp32 accumulator itself (no rounding to fp16).  Same sizes,
 * ownership, asynchrony and error rules as gemm_f16_nt, plus n < 2^25;
 * k == 0 fills D with +0.  Options as for gemm_f16_nt_ex, except that
 * GEMM_F16_TILE_128x128_M16 is not available (GEMM_F16_EINVAL).
 */
int gemm_f16_nn_f32(int64_t m, int64_t n, int64_t k, const void *a, const void *b,
                    void *d, void *stream);
int gemm_f16_nn_f32_ex(int64_t m, int64_t n, int64_t k, const void *a, const void *b,
                       void *d, void *stream, const gemm_f16_options *opt);

/* Static message for a status code (never NULL). */
const char *gemm_f16_status_string(int status);

/*
 * Host-side copy of the block-tile scheduler the kernels run (same source):
 * workgroup index `pid` of a grid of num_m*num_n tiles -> (m_block, n_block).
 * With xcd != 0 the dispatch index is first remapped so each of the 8 XCDs
 * gets a contiguous run of tiles; the tiles are then grouped `swizzle`
 * tile-columns wide and handed out row-major inside a group ("4. Pipeline
 * Abstraction and Two Consumer Warp Groups", section "Tile Rasterization").
 * Returns GEMM_F16_EINVAL for num_m or num_n below 1, a grid of 2^63
 * tiles or more, pid outside the grid or swizzle < 1.
 * Pure host function: no HIP call.
 */
int gemm_f16_tile_coord(int64_t pid, int64_t num_m, int64_t num_n, int32_t swizzle,
                        int32_t xcd, int64_t *m_block, int64_t *n_block);

/*
 * Block tile the automatic choice would use for (m, n, k) on the current
 * device: one of GEMM_F16_TILE_*, or a negative status for invalid sizes.
 * Asks HIP for the device's compute-unit count (once per device); with no
 * device it assumes 256.
 */
int gemm_f16_select_tile(int64_t m, int64_t n, int64_t k);

/*
 * The xcd option that xcd = -1 stands for, on a grid of num_m x num_n
 * block tiles rasterized `swizzle` tile-columns wide, on a device of `cus`
 * compute units: 1 (remap) except on a grid of exactly `cus` tiles whose
 * dispatch order leaves no XCD more operand panels (distinct tile rows
 * plus tile columns) than the remap does; then 0.  Returns
 * GEMM_F16_EINVAL for num_m, num_n or swizzle below 1, cus below 0, or a
 * grid of 2^31 tiles or more.  Pure host function: no HIP call.
 */
int gemm_f16_select_xcd(int64_t num_m, int64_t num_n, int32_t swizzle, int32_t cus);

/* ---- segmented products ------------------------------------------------------
 *
 * Matrix products over rows that fall into consecutive segments of ragged
 * sizes: the tokens of each expert of a routed layer, or the requests of
 * each low-rank adapter.  Segment g holds rows offsets[g] .. offsets[g+1]-1
 * of `rows`; the sizes live on the GPU only and the host never waits for
 * them.
 *
 * Common rules: device pointers, row-major dense operands, asynchronous on
 * `stream`, the errors above; int32 arrays are 4-byte aligned.  offsets is
 * int32 [groups+1], non-decreasing, offsets[0] read as 0, other values
 * clamped to [0, rows].  Offsets, ids, indices and orders that break these
 * rules give unspecified outputs but no access out of range.  An output
 * must not overlap any input or the workspace (GEMM_F16_EOVERLAP).
 * workspace (where a call has one): device memory of at least the bytes that the matching
 * *_workspace function returns (0: may be NULL), 16-byte aligned, its
 * content free to be overwritten until the call's work is done; too few
 * bytes give GEMM_F16_EINVAL.
 * Sums run in fp32, in an order that depends on the sizes alone: the same
 * call gives the same bits.
 */

/*
 * The plan of a routed batch: a stable sort of row numbers by group.
 *   ids      int32 (id_bytes 4) or int64 (id_bytes 8) [rows]: the group of
 *            each row; an id outside [0, groups) belongs to no group and
 *            sorts behind all of them
 *   order    int32 [rows]      row at each place of the sorted order
 *   inverse  int32 [rows]      place of each row: order[inverse[r]] == r
 *   offsets  int32 [groups+1]  first place of each group; offsets[groups]
 *            is where the rows of no group begin
 * 0 <= rows < 2^30, 1 <= groups <= 2048.
 */
int gemm_f16_group_rows(int64_t rows, int64_t groups, const void *ids, int32_t id_bytes,
                        int32_t *order, int32_t *inverse, int32_t *offsets,
                        void *workspace, int64_t workspace_bytes, void *stream);
int64_t gemm_f16_group_rows_workspace(int64_t rows, int64_t groups);

/*
 * Products grouped by segment, with the segment g of row r:
 *
 *   grouped_nt   C[r][n] = sum_k A[src(r)][k] * B[g][n][k]      B [groups,N,K]
 *   grouped_nn   C[r][n] = sum_k A[r][k] * B[g][k][n]           B [groups,K,N]
 *   grouped_tn   C[g][k][n] = sum_{r in g} A[r][k] * B[r][n]    A [rows,K], B [rows,N]
 *
 * A and B are fp16, C is fp16 (out_f32 0; rounded once, to nearest even) or
 * fp32 (out_f32 1).  grouped_nt reads A [a_rows,K] at src(r) = index[r] / fan
 * (index NULL: r): with `order` of gemm_f16_group_rows as the index, row
 * order[r] / fan is the token of the r-th routed row when each token has
 * `fan` of them.  A row whose src lies outside [0, a_rows) is taken as
 * zeros.  grouped_nn and grouped_tn with C's fp16 gradient in A give the
 * gradients of grouped_nt by its input rows and by its weights.
 * Rows behind offsets[groups] come out as zeros; so does C[g] of an empty
 * segment (grouped_tn).
 *
 * rows, a_rows < 2^30; n < 2^30 (nn, tn: 2^25); k < 2^22; 1 <= groups <=
 * 2^20; 1 <= fan; rows*n, groups*n*k < 2^47.
 */
int gemm_f16_grouped_nt(int64_t rows, int64_t groups, int64_t n, int64_t k, const void *a,
                        int64_t a_rows, const void *b, const int32_t *offsets,
                        const int32_t *index, int64_t fan, void *c, int32_t out_f32,
                        void *stream);
int gemm_f16_grouped_nn(int64_t rows, int64_t groups, int64_t n, int64_t k, const void *a,
                        const void *b, const int32_t *offsets, void *c, int32_t out_f32,
                        void *stream);
int gemm_f16_grouped_tn(int64_t rows, int64_t groups, int64_t n, int64_t k, const void *a,
                        const void *b, const int32_t *offsets, void *c, int32_t out_f32,
                        void *stream);

/*
 * grouped_tn with a workspace: where C has few tiles and the segments many
 * rows, each segment's rows are split among workgroups, whose fp32 sums meet
 * in the workspace and are added in their order.  The workspace is at most
 * 512 tiles of 64 KB; where its size is 0, the call is gemm_f16_grouped_tn.
 */
int gemm_f16_grouped_tn_ws(int64_t rows, int64_t groups, int64_t n, int64_t k, const void *a,
                           const void *b, const int32_t *offsets, void *c, int32_t out_f32,
                           void *workspace, int64_t workspace_bytes, void *stream);
int64_t gemm_f16_grouped_tn_workspace(int64_t rows, int64_t groups, int64_t n, int64_t k);

/*
 * A projection shared by requests that each have a low-rank adapter of
 * their own (or none):
 *
 *   Y[r][n] = fp16( sum_k X[r][k] W[n][k]
 *                   + scale[s] * sum_j (sum_k X[r][k] D[s][j][k]) * U[s][n][j] ),  s = ids[r]
 *
 *   x        fp16 [rows,K]            w   fp16 [N,K]
 *   down     fp16 [adapters,rank,K]   up  fp16 [adapters,N,rank]
 *   ids      int32 [rows]: the adapter of each row; outside [0, adapters): none
 *   order, offsets   of gemm_f16_group_rows(rows, adapters, ids, ...)
 *            (past its 2048 groups: any stable sort of the rows by adapter)
 *   scale    fp32 [adapters], or NULL for ones
 *   y        fp16 [rows,N]
 *
 * The inner product is kept in fp32 (past 64 rows its second product takes it
 * as three bf16 parts, which hold it exactly) and Y is rounded once.
 * rows, n < 2^30; k < 2^22; 1 <= rank <= 4096; 1 <= adapters <= 2^20;
 * rows*n, n*k, adapters*rank*(n+k) < 2^47.
 */
int gemm_f16_lora_nt(int64_t rows, int64_t n, int64_t k, int64_t adapters, int64_t rank,
                     const void *x, const void *w, const void *down, const void *up,
                     const int32_t *ids, const int32_t *order, const int32_t *offsets,
                     const float *scale, void *y, void *workspace, int64_t workspace_bytes,
                     void *stream);
int64_t gemm_f16_lora_workspace(int64_t rows, int64_t n, int64_t k, int64_t adapters,
                                int64_t rank);

/* ---- the feed-forward layer around the products --------------------------------
 *
 * What a transformer's feed-forward layer, dense or routed, needs between its
 * products: a product with bias, activation and residual in its epilogue, the
 * routing of tokens to experts and the way back from them, each with its
 * gradient.  The common rules of the segmented products above hold here too.
 */

enum {
    GEMM_F16_ACT_NONE = 0,
    GEMM_F16_ACT_RELU = 1,       /* max(z, 0) */
    GEMM_F16_ACT_GELU = 2,       /* z Phi(z), Phi the normal distribution (erf) */
    GEMM_F16_ACT_GELU_TANH = 3,  /* z / 2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
    GEMM_F16_ACT_SILU = 4,       /* z / (1 + exp(-z)) */
    GEMM_F16_ACT_LAST = 4
};

/*
 * The epilogue of gemm_f16_fused_nt.  Null pointers leave their part out; all
 * zeros is the plain product.
 */
typedef struct {
    int32_t act;          /* GEMM_F16_ACT_* */
    int32_t bias_f32;     /* type of bias: fp16 (0) or fp32 (1) */
    int32_t out_f32;      /* type of c and residual: fp16 (0) or fp32 (1) */
    const void *bias;     /* [n] */
    const void *residual; /* [m,n]; may be c itself, else must not overlap it */
    void *pre;            /* fp16 [m,n]: z, for the gradient; past fp16's range an infinity */
} gemm_f16_epilogue;

/*
 *   z = A B^T + bias,   c = act(z) + residual,   pre = fp16(z)
 *
 *   a  fp16 [m,k]    b  fp16 [n,k]    c  fp16 or fp32 [m,n]
 *
 * Everything is summed in fp32 and c rounded once; act takes the unrounded z.
 * m, n < 2^30; m*n < 2^47; k < 2^22; any size and alignment; k == 0: z is the
 * bias.  epilogue == NULL: the plain product.  Where z is -inf, the
 * activations but relu give what their formulas give, a NaN.
 */
int gemm_f16_fused_nt(int64_t m, int64_t n, int64_t k, const void *a, const void *b, void *c,
                      const gemm_f16_epilogue *epilogue, void *workspace, int64_t workspace_bytes,
                      void *stream);
int64_t gemm_f16_fused_workspace(int64_t m, int64_t n, int64_t k);

/*
 * The elementwise part of its gradient:
 *
 *   dz[m][n] = dy[m][n] act'(pre[m][n])        dbias[n] = sum_m dz[m][n]
 *
 *   dy   fp16 or fp32 [m,n]: the gradient of c
 *   pre  fp16 [m,n]: of the forward call; not read without an activation.  At
 *        an infinity (z past fp16's range) act' is its limit, 0 or 1
 *   dz   fp16 [m,n] or NULL; may be dy itself where that is fp16
 *   dbias  fp32 [n] or NULL: sums in fp32 of dz before it is rounded
 *
 * The residual's gradient is dy; A's is dz B and B's dz^T A (gemm_f16_nn_f32
 * or gemm_f16_grouped_nn, and gemm_f16_grouped_tn, with one segment).  The
 * workspace is needed with dbias only.
 */
int gemm_f16_fused_grad(int64_t m, int64_t n, const void *dy, int32_t dy_f32, const void *pre,
                        int32_t act, void *dz, float *dbias, void *workspace,
                        int64_t workspace_bytes, void *stream);
int64_t gemm_f16_fused_grad_workspace(int64_t m, int64_t n);

enum { GEMM_F16_SCORE_SOFTMAX = 0, GEMM_F16_SCORE_SIGMOID = 1 };

/* How tokens are routed (see gemm_f16_route). */
typedef struct {
    int32_t score;        /* GEMM_F16_SCORE_* */
    int32_t groups;       /* groups of experts / groups neighbours each; 1: none */
    int32_t top_groups;   /* groups that a token may use */
    int32_t group_top;    /* a group's value: its largest key (1), or the sum of its two largest (2) */
    int32_t renormalize;  /* 1: a token's gates sum to scale */
    float scale;          /* finite */
} gemm_f16_routing;

/*
 * The experts of each token and their gates.
 *
 *   s = softmax(logits) over a token's experts, or sigmoid(logits)
 *   key = s + bias; without a bias, the logit (whose order is that of s)
 *   ids = the `fan` largest keys among the top_groups groups of largest value,
 *         in falling order, ties to the lowest index (of groups, too); a
 *         group's sum is that of keys, without a bias of scores
 *   gates = scale * s[ids], renormalised: scale * s[ids] / sum(s[ids])
 *
 *   logits  fp16 or fp32 [tokens,experts]     bias  fp32 [experts] or NULL
 *   ids     int32 [tokens,fan]                gates fp32 [tokens,fan]
 *
 * The choice is that of the formula in 64 bits (keys that differ by less than
 * their rounding in fp32 are told apart in 64).  An expert whose logit or key
 * is -inf or NaN is never chosen; where too few are left, the remaining ids
 * are -1, which gemm_f16_group_rows sorts behind all experts, with gates of 0.
 * In the softmax a logit of -inf or NaN counts as 0; the bias, which is for the
 * choice alone, takes no expert out of it.
 * 0 <= tokens < 2^30; 1 <= experts <= 2048; 1 <= fan <= 32; fan <= experts /
 * groups * top_groups; 1 <= groups <= 64, a divisor of experts.
 */
int gemm_f16_route(int64_t tokens, int64_t experts, int64_t fan, const void *logits,
                   int32_t logits_f32, const float *bias, const gemm_f16_routing *routing,
                   int32_t *ids, float *gates, void *stream);

/*
 * dlogits [tokens,experts], of the logits' type, from dgates fp32 [tokens,fan]:
 * the gates' gradient with the choice held fixed.  Zeros for what has no part
 * in the gates; ids outside [0, experts) have none.  Of `routing`, score,
 * renormalize and scale are used.
 */
int gemm_f16_route_grad(int64_t tokens, int64_t experts, int64_t fan, const void *logits,
                        int32_t logits_f32, const int32_t *ids, const float *dgates,
                        const gemm_f16_routing *routing, void *dlogits, void *stream);

/*
 * Rows that were routed by gemm_f16_group_rows(tokens * fan, groups, ids)
 * back to their tokens:
 *
 *   y[t][n] = residual[t][n] + sum_f gates[t][f] * rows[inverse[t*fan + f]][n]
 *
 *   rows      fp16 or fp32 [tokens*fan, n], in the plan's order
 *   inverse, offsets   of the plan; places from offsets[groups] on belong to
 *             no group and add nothing, whatever they hold
 *   gates     fp32 [tokens,fan], or NULL for ones: the gradient of
 *             gemm_f16_grouped_nt's gathered tokens from that of its rows
 *   residual  [tokens,n] of y's type, or NULL; may be y itself, else must not overlap it
 *   y         fp16 or fp32 [tokens,n]: summed in fp32, rounded once
 *
 * tokens*fan, n < 2^30; fan >= 1; tokens*fan*n < 2^47.
 */
int gemm_f16_combine_rows(int64_t tokens, int64_t fan, int64_t n, int64_t groups, const void *rows,
                          int32_t rows_f32, const int32_t *inverse, const int32_t *offsets,
                          const float *gates, const void *residual, void *y, int32_t y_f32,
                          void *stream);

/*
 * Its gradient:
 *
 *   drows[inverse[t*fan + f]][n] = gates[t][f] * dy[t][n]
 *   dgates[t][f] = sum_n dy[t][n] * rows[inverse[t*fan + f]][n]
 *
 *   dy fp16 or fp32 [tokens,n]; drows fp16 or fp32 [tokens*fan, n] or NULL;
 *   dgates fp32 [tokens,fan] or NULL (then rows is not read)
 *
 * Rows behind offsets[groups] get zeros, and so do their gates.  The
 * residual's gradient is dy.
 */
int gemm_f16_combine_rows_grad(int64_t tokens, int64_t fan, int64_t n, int64_t groups,
                               const void *dy, int32_t dy_f32, const void *rows, int32_t rows_f32,
                               const int32_t *inverse, const int32_t *offsets, const float *gates,
                               void *drows, int32_t drows_f32, float *dgates, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_F16_H */
