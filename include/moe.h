/*
 * moe.h - C ABI of a deterministic MoE layer (forward and backward) for one AMD MI355X (gfx950).
 *
 * The layer is the mixture-of-experts step that the pages on Mixture-of-Kittens (MoK) describe.
 * Those pages are the MarkTechPost article "Cursor Open-Sources Mixture-of-Kittens (MoK): A
 * Deterministic MoE Training Megakernel for GB300 NVL72 Racks", the toknow.ai post
 * "Mixture-of-Kittens: Cursor's Open-Source Kernel Trains AI Up to 2.37x Faster" and the aiweekly.co
 * alert "Cursor open-sources MoE megakernel for GB300 NVL72 racks". This library takes one GPU's
 * share of it.
 *
 * Forward: the router, then an expert-grouped permute into a ring slot, then per-expert SwiGLU
 * MLPs, then a weighted combine. Backward: dgrad and wgrad of every GEMM, plus the router-weight
 * gradient, which is computed inside the SwiGLU backward (MarkTechPost, closing paragraph of
 * "Three design decisions that matter").
 *
 * Conventions for every entry point:
 *  - Every pointer argument is DEVICE memory of the current HIP device, owned by the caller. The
 *    library never allocates, frees or synchronises. Each call only enqueues kernels on `stream`
 *    (a hipStream_t; NULL means the null stream) and returns.
 *  - Row-major layouts throughout. bf16 is IEEE bfloat16 stored as uint16. Weights follow the
 *    [out, in] convention: W1 is [E, 2I, d] (rows 0..I-1 gate, I..2I-1 up), W2 is [E, d, I], and
 *    the router weight Wr is [E, d].
 *  - Return value: MOE_OK (0), or a negative moe_status. Arguments are checked on the host before
 *    anything is enqueued. A failed check enqueues nothing. Nothing prints and nothing throws.
 *  - Determinism: every result is a function of the inputs alone. No float atomics are used,
 *    and every reduction runs in a fixed order, so two runs are bitwise identical.
 *  - No host synchronisation: per-expert counts never leave the device. Buffers are sized for
 *    the worst case, so no token is ever dropped, whatever the expert imbalance (MarkTechPost,
 *    "Three design decisions that matter": ring token buffer; "Key Takeaways").
 */
#ifndef MOE_MI355X_H
#define MOE_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef void* moe_stream_t; /* hipStream_t */

typedef enum moe_status {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = -1,     /* null pointer, bad shape, misaligned pointer */
    MOE_ERR_RING_TOO_SMALL = -2,  /* ring_bytes < (slot + 1) * ring slot bytes */
    MOE_ERR_UNSUPPORTED = -3,     /* a mode the library does not provide */
    MOE_ERR_HIP = -4,             /* a HIP runtime error while enqueuing */
    MOE_ERR_WORKSPACE_TOO_SMALL = -5
} moe_status;

/* 3 is not in use. */
enum {
    MOE_PREC_BF16 = 0, MOE_PREC_MXFP8 = 1, MOE_PREC_MXFP4 = 2, MOE_PREC_FP8 = 4, MOE_PREC_INT8 = 5
};

/* cfg.flags bits */
enum {
    MOE_FLAG_PERSISTENT = 1,  /* grouped GEMMs as persistent grids walking the schedule table */
    MOE_FLAG_MXFP8_WGRAD = 2, /* MXFP8 mode only: the weight gradients in MXFP8 too (below) */
    MOE_FLAG_BF16_DW = 4      /* dw1 and dw2 are bf16 buffers instead of fp32 (below) */
};

/* Device status word (first 4 bytes of the workspace). moe_permute clears it and ORs bits into
 * it; the caller may read it after its own synchronisation. */
enum {
    MOE_DEVICE_BAD_EXPERT_INDEX = 1, /* a topk_idx entry outside [0, E): that row is skipped */
    MOE_DEVICE_BARRIER_TIMEOUT = 2   /* moe_forward_fused: a grid barrier waited ~2 s and gave up
                                        (the results of that call are not valid) */
};

/* Layer shape and mode. Constraints checked on the host: T >= 1; 1 <= k <= E <= 1024; k <= 64;
 * d % 256 == 0 (the GEMMs have no masked K tail: K steps of 64 and 256-wide tiles along d);
 * I % 128 == 0 (128-wide tiles along I); T * k < 2^31; T * E < 2^31; and, because the kernels
 * address rows with 32-bit offsets: T * d < 2^31, T * k * d < 2^31, T * k * 2I < 2^31 (an
 * expert may receive all T * k rows) and 4 * I * d < 2^31 (the bytes of one expert's W1).
 * precision MOE_PREC_BF16, MOE_PREC_MXFP8, MOE_PREC_FP8, MOE_PREC_INT8 or MOE_PREC_MXFP4 (MXFP4
 * also needs I % 256 == 0: its K steps along I are 256 deep).
 * Every entry point that enqueues work also checks that the current HIP device is a gfx950
 * (MOE_ERR_UNSUPPORTED otherwise, MOE_ERR_HIP when no device can be queried).
 *
 * MXFP8 mode (the pages name BF16 and MXFP8 modes: MarkTechPost, closing paragraph of "Three
 * design decisions that matter") follows the OCP MX v1.0 MXFP8 format. Elements are E4M3; every
 * 32 consecutive elements along a GEMM's reduction axis share one E8M0 scale 2^(code - 127),
 * code = floor(log2 amax) - 8 + 127 clamped to 0..254 (0 for an all-zero block). Elements round
 * to nearest even and saturate to +-448. The forward GEMMs read Xp and W1 quantised along d,
 * and A and W2 along I. The dgrad GEMMs read dY and W2 along d, and dH and W1 along 2I. The
 * weight gradients and dWr read bf16 operands, with Xp taken as the MXFP8 image the ring
 * holds. All accumulation is fp32; outputs are bf16 as in BF16 mode.
 * With MOE_FLAG_MXFP8_WGRAD the two weight gradients take MXFP8 operands as well, quantised
 * along their reduction axis, the positions of each expert: blocks of 32 consecutive positions
 * from the expert's first one, the last block holding what is left. dW2 reads w dY (the fp32
 * product, quantised directly) and A, dW1 reads dH and the ring's MXFP8 image of Xp, each
 * quantised so. dWr is unchanged.
 *
 * MXFP4 mode (the MarkTechPost page, section "MoE layer as the bottleneck", names the team's
 * earlier 4-bit NVFP4 training kernels; this mode takes the OCP MX 4-bit format instead, which
 * gfx950's scaled MFMA reads) follows the OCP MX v1.0 MXFP4 format on the same axes as MXFP8
 * mode: elements are E2M1 (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6), stored two to a byte
 * with element 2i in the low nibble; the scale code is floor(log2 amax) - 2 + 127 clamped to
 * 0..254; elements round to nearest even and saturate to +-6. The weight gradients and dWr read
 * bf16 operands, Xp taken as the exact bf16 image of the MXFP4 codes the ring holds.
 * MOE_FLAG_MXFP8_WGRAD is not accepted. Buffers: a ring slot holds Xp's codes [T*k, d/2 bytes]
 * then its scales; moe_quantize_weights writes the four weight copies in E2M1.
 *
 * FP8 mode takes the block-scaled FP8 format of the moe_fp8_ calls below: E4M3 with one fp32 scale
 * per 1 x 128 of the rows and per 128 x 128 of the weights, on the axes of the MX modes. The
 * forward products read Xp and W1 quantised along d, and A and W2 along I; the dgrad products dY
 * and W2 along d, and dH and W1 along 2I. The ring slot holds bf16 Xp as in BF16 mode, and the
 * weight gradients and dWr read bf16 operands. A is computed from the stored H, and dw and dH from
 * dA' rounded to bf16, each product's output. What is not finite stays so, as NaN. The call
 * moe_quantize_weights is needed as in the MX modes.
 * MOE_FLAG_PERSISTENT and MOE_FLAG_MXFP8_WGRAD are not accepted, moe_forward_fused not provided.
 *
 * INT8 mode is for inference: the experts' products in the 8-bit integers of the moe_i8_ calls below,
 * a scale for each token and output channel. The ring slot holds bf16 Xp as in BF16 mode;
 * moe_forward quantises its rows, forms A (bf16) from the exact integer products of the gate and up
 * projections, and quantises A's rows for the down product. H is not kept: `saved` holds A
 * alone (moe_sizes.saved_H means nothing). moe_quantize_weights is needed, and writes the forward's
 * two weights only; the bf16 weights are not needed behind it. No flag is accepted; moe_backward and moe_forward_fused return
 * MOE_ERR_UNSUPPORTED. Limits: d and I below 2^17; T * k, E * 2I and E * d below 2^24.
 *
 * Weight-gradient precision. The pages do not say in which precision the weight gradients are
 * kept. By default dw1 and dw2 are fp32 (the caller's main gradient, which microbatches
 * accumulate into). With MOE_FLAG_BF16_DW (any precision) they are bf16: each element is
 * the same fp32 sum rounded once to nearest even where it is stored; with accumulate the fp32
 * sum of the stored bf16 value and the new result is rounded once. dwr stays fp32. */
typedef struct moe_cfg {
    int32_t T;         /* tokens entering the layer */
    int32_t d;         /* hidden size */
    int32_t E;         /* experts on this GPU */
    int32_t k;         /* experts per token (top-k) */
    int32_t I;         /* SwiGLU intermediate size */
    int32_t precision; /* MOE_PREC_* */
    int32_t flags;     /* MOE_FLAG_* */
} moe_cfg;

/* Byte sizes of the caller-owned buffers, and the offsets of the intermediates inside them. */
typedef struct moe_sizes {
    size_t ring_slot;      /* one ring slot: the permuted tokens Xp, bf16 [T*k, d] */
    size_t saved;          /* forward activations kept for backward */
    size_t saved_H;        /* offset of H = [g | u], bf16 [T*k, 2I], rows in position order */
    size_t saved_A;        /* offset of A = silu(g) * u, bf16 [T*k, I] */
    size_t workspace;      /* scratch for route/permute/forward/backward (one buffer serves all) */
    size_t ws_O;           /* offset of the expert outputs O, bf16 [T*k, d], valid after forward */
    size_t ws_dH;          /* offset of dH, bf16 [T*k, 2I], valid after backward */
    size_t ws_dXp;         /* offset of dXp, bf16 [T*k, d], valid after backward */
    size_t wq;             /* MX, FP8 and INT8 modes: bytes of the quantised-weight buffer (else 0) */
} moe_sizes;

/* Sizes of every caller buffer for `cfg`. Host only; enqueues nothing. (Plumbing of this
 * library, defined by no passage of the pages. The schedule and task tables live inside the
 * workspace, so they have no size of their own here.)
 * In MXFP8 mode a ring slot holds the E4M3 codes of Xp [T*k, d] followed (at the next 256-byte
 * boundary) by their scales [T*k, d/32]; in MXFP4 mode the E2M1 codes [T*k, d/2 bytes] followed
 * by the scales. */
int moe_query(const moe_cfg* cfg, moe_sizes* out);

/*
 * moe_quantize_weights - MX, FP8 and INT8 modes: the quantised expert weights every such forward and
 * backward reads. Call it once per weight update; the result serves any number of batches.
 *
 *   w1  bf16 [E, 2I, d]   in
 *   w2  bf16 [E, d, I]    in
 *   wq  bytes [wq_bytes]  out, wq_bytes >= moe_sizes.wq. It receives four quantised tensors (in INT8
 *       mode the forward's two), each with its scales (per 32 in the MX modes): W1 along d [E, 2I, d] and W2 along I [E, d, I]
 *       (forward), and W2 along d stored transposed [E, I, d] and W1 along 2I stored transposed
 *       [E, d, 2I] (dgrad), in the mode's element format. The layout inside wq is private to the
 *       library.
 * Errors: MOE_ERR_INVALID_ARG in BF16 mode; MOE_ERR_WORKSPACE_TOO_SMALL for a short wq.
 */
int moe_quantize_weights(const moe_cfg* cfg, const void* w1, const void* w2, void* wq,
                         size_t wq_bytes, moe_stream_t stream);

/*
 * moe_route - router logits, top-k selection and renormalised softmax weights.
 *
 * The toknow.ai summary describes an MoE as sending each input to a few experts. The gate used
 * here is the plain top-k softmax:
 *   logits[t,e] = sum_i x[t,i] * w_router[e,i], in fp32. For each (t,e) one accumulator starts
 *       at +0 and gains the exact bf16 x bf16 products for i = 0,1,..,d-1 in ascending order,
 *       rounding after each addition.
 *   topk_idx[t,:] holds the k largest logits in descending order; equal logits go to the lower
 *       expert index. Selection compares logits numerically (-0 == +0; NaN unsupported).
 *   topk_w[t,j] = exp(l_j - l_0) / sum_{i<k} exp(l_i - l_0), in fp32 (l_0 = the largest),
 *       which equals softmax over all E followed by renormalisation over the k selected.
 *
 *   x        bf16 [T, d]    in
 *   w_router bf16 [E, d]    in
 *   logits   fp32 [T, E]    out
 *   topk_idx int32 [T, k]   out
 *   topk_w   fp32 [T, k]    out
 *   workspace bytes [ws_bytes]  scratch (the router weight widened to fp32), the same
 *                               workspace the other calls take
 */
int moe_route(const moe_cfg* cfg, const void* x, const void* w_router, float* logits,
              int32_t* topk_idx, float* topk_w, void* workspace, size_t ws_bytes,
              moe_stream_t stream);

/*
 * moe_permute - expert histogram, exclusive scan, and a stable grouping of the T*k rows by
 * expert into ring slot `slot`.
 *
 * The gather half of the pages' dispatch is the part that stays on one GPU (MarkTechPost, "Three
 * design decisions that matter": pull-based dispatch and the ring token buffer). Row r = t*k + j
 * goes to position pos = offsets[e] + (number of rows r' < r with the same expert e), so inside
 * an expert segment rows ascend by r.
 *
 *   topk_idx int32 [T, k]          in   (from moe_route, or given by the caller; a caller's row
 *                                       may name one expert twice: every row is its own
 *                                       position either way)
 *   x        bf16 [T, d]           in
 *   ring     bytes [ring_bytes]    out: slot `slot` (at slot * ring_slot bytes) receives
 *                                       Xp[pos] = x[row_src[pos] / k], bf16 [T*k, d]; in an MX
 *                                       mode its MX image (codes, then scales)
 *   counts   int32 [E]             out: rows per expert
 *   offsets  int32 [E+1]           out: exclusive scan of counts, offsets[E] = T*k
 *   row_src  int32 [T*k]           out: pos -> r
 *   tk_row   int32 [T*k]           out: r -> pos (-1 for a skipped bad-index row)
 *   workspace bytes [ws_bytes]     scratch; also holds the device status word
 * Errors: MOE_ERR_RING_TOO_SMALL when (slot + 1) * ring_slot > ring_bytes or slot < 0.
 */
int moe_permute(const moe_cfg* cfg, const int32_t* topk_idx, const void* x, void* ring,
                size_t ring_bytes, int32_t slot, int32_t* counts, int32_t* offsets,
                int32_t* row_src, int32_t* tk_row, void* workspace, size_t ws_bytes,
                moe_stream_t stream);

/*
 * moe_permute_static - moe_permute for callers that cannot allocate: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc. Same operation, arguments and
 * results as moe_permute, except that:
 *  - there is no workspace argument: the permutation's scratch (per-256-row-block expert counts,
 *    per-row ranks, per-block flags) lives in a fixed array of MOE_STATIC_SCRATCH_BYTES inside
 *    the library, one per GPU, held until the process ends;
 *  - the device status word is written to `device_status` (int32, caller device memory) instead
 *    of the workspace's first word.
 * The call allocates nothing and frees nothing. Its scratch needs 4 * (nb * E + nb + T * k)
 * bytes with nb = ceil(T * k / 256), each part 256-byte aligned; beyond MOE_STATIC_SCRATCH_BYTES
 * it returns MOE_ERR_WORKSPACE_TOO_SMALL and enqueues nothing. Every call on one GPU shares that
 * GPU's array: calls that overlap on one GPU (concurrent streams, or threads) race and give
 * undefined results. Calls in one stream order are safe; the array keeps the last call's
 * contents, and every word is written before it is read.
 */
#define MOE_STATIC_SCRATCH_BYTES ((size_t)4 << 20)
int moe_permute_static(const moe_cfg* cfg, const int32_t* topk_idx, const void* x, void* ring,
                       size_t ring_bytes, int32_t slot, int32_t* counts, int32_t* offsets,
                       int32_t* row_src, int32_t* tk_row, int32_t* device_status,
                       moe_stream_t stream);

/*
 * moe_forward - grouped SwiGLU expert MLPs over the ring slot, then the weighted combine.
 *
 * The expert-grouped GEMMs are in MarkTechPost, "Three design decisions that matter". For each
 * expert e and each of its positions:
 *   [g | u] = Xp[pos] W1[e]^T   (fp32 accumulate; stored bf16 as H)
 *   A       = silu(g) * u        (from the fp32 g, u; stored bf16)
 *   O[pos]  = A W2[e]^T          (fp32 accumulate; stored bf16 in the workspace)
 * Combine, which is atomic-free and fixed-order:
 *   y[t] = bf16( sum_{j=0..k-1} topk_w[t,j] * O[tk_row[t*k+j]] ), fp32 FMA with j ascending.
 *
 *   ring, ring_bytes, slot   in: the slot written by moe_permute
 *   offsets, tk_row          in: from moe_permute
 *   topk_w   fp32 [T, k]     in
 *   w1       bf16 [E, 2I, d] in (not read in INT8 mode, may be NULL)
 *   w2       bf16 [E, d, I]  in (likewise)
 *   wq, wq_bytes             in: MX, FP8 and INT8 modes, the buffer moe_quantize_weights filled
 *                                (ignored in BF16 mode, may be NULL)
 *   y        bf16 [T, d]     out
 *   saved    bytes [saved_bytes]   out: H and A at the offsets moe_query reports
 *   workspace bytes [ws_bytes]     scratch
 */
int moe_forward(const moe_cfg* cfg, const void* ring, size_t ring_bytes, int32_t slot,
                const int32_t* offsets, const int32_t* tk_row, const float* topk_w,
                const void* w1, const void* w2, const void* wq, size_t wq_bytes, void* y,
                void* saved, size_t saved_bytes, void* workspace, size_t ws_bytes,
                moe_stream_t stream);

/*
 * moe_forward_fused - moe_route, moe_permute and moe_forward in ONE kernel launch (BF16 mode).
 *
 * The pages' layer is one persistent kernel that fuses all of its steps (MarkTechPost, "Cursor
 * Open-Sources Mixture-of-Kittens (MoK)": introduction, and the closing paragraph of "Three
 * design decisions that matter"). This call runs the router, the permutation into ring slot
 * `slot`, both grouped GEMMs and the combine as phases of one cooperatively launched grid
 * (every workgroup resident) that meet at grid-wide barriers, so a small layer pays one launch
 * instead of about a dozen. It writes everything the three calls write (logits, topk_idx,
 * topk_w, counts, offsets, row_src, tk_row, the ring slot, H and A in `saved`, O in the
 * workspace, y, the device status word), with the same values: bit for bit when no expert
 * receives 256 rows or more; otherwise the down projection of those experts' rows sums its K
 * chunks from another start (the separate path gives such blocks a 256 x 256 tile), which
 * changes their O and y in the last bits only. Arguments and errors are those of the three
 * calls; the other modes return MOE_ERR_UNSUPPORTED. The grid barriers keep their state in a
 * device variable of the library, one per GPU: fused calls that overlap on one GPU race.
 */
int moe_forward_fused(const moe_cfg* cfg, const void* x, const void* w_router, float* logits,
                      int32_t* topk_idx, float* topk_w, void* ring, size_t ring_bytes,
                      int32_t slot, int32_t* counts, int32_t* offsets, int32_t* row_src,
                      int32_t* tk_row, const void* w1, const void* w2, void* y, void* saved,
                      size_t saved_bytes, void* workspace, size_t ws_bytes, moe_stream_t stream);

/*
 * moe_backward - gradients of L = <y, dy> with respect to x, the router weight, w1, w2 and the
 * routing weights.
 *
 * Per position pos (token t, slot j, expert e, weight w):
 *   dA'      = dy[t] W2[e]                           (fp32, never stored)
 *   dw       = <dA', A[pos]>, which equals <dy[t], A[pos] W2[e]^T>. This is the router-weight
 *              gradient, fused into the SwiGLU backward (MarkTechPost, closing paragraph of
 *              "Three design decisions that matter"). Per-tile partials are summed in
 *              ascending tile order.
 *   dA       = w * dA'
 *   dg, du   = dA * u * s * (1 + g (1 - s)),  dA * silu(g)   (s = sigmoid(g); g, u from H)
 *   dH[pos]  = bf16([dg | du]);  dXp[pos] = bf16(dH[pos] W1[e])
 *   dW2[e]   = sum over pos in e, ascending, of bf16(w dy[t]) (x) A[pos]   (fp32 sums)
 *   dW1[e]   = sum over pos in e, ascending, of dH[pos] (x) Xp[pos]       (fp32 sums)
 * Per token: d_topk_w[t,j] = dw of its row. When w_router is given (the layer routed itself):
 *   dlogit_j = w_j (dw_j - sum_i w_i dw_i), and 0 off the selected set;
 *   dx[t]    = bf16( sum_j dXp[tk_row[t*k+j]] + sum_j dlogit_j Wr[e_j] ), j ascending, fp32;
 *   dWr[e]   = sum over pos in e, ascending, of dlogit(pos) * Xp[pos]          (fp32).
 * When w_router is NULL (routing given), dx[t] = bf16(sum_j dXp[tk_row[t*k+j]]), and dwr is not
 * touched. Experts with no rows get zero dW1/dW2 blocks. With accumulate != 0, dw1, dw2 and dwr
 * are added to (read-modify-write, the sum in fp32) instead of overwritten.
 *
 *   ring, ring_bytes, slot        in: the slot holding this batch's Xp (written by moe_permute)
 *   offsets, row_src, tk_row      in: from moe_permute
 *   topk_idx int32 [T, k], topk_w fp32 [T, k]   in
 *   w_router bf16 [E, d] or NULL  in
 *   w1, w2, wq, wq_bytes          in (as in moe_forward)
 *   saved                         in: from moe_forward of the same batch
 *   dy       bf16 [T, d]          in
 *   dx       bf16 [T, d]          out
 *   dw1      fp32 [E, 2I, d]      out (or accumulated); bf16 with MOE_FLAG_BF16_DW
 *   dw2      fp32 [E, d, I]       out (or accumulated); bf16 with MOE_FLAG_BF16_DW
 *   dwr      fp32 [E, d]          out (or accumulated); ignored when w_router is NULL
 *   d_topk_w fp32 [T, k]          out
 *   workspace bytes [ws_bytes]    scratch (dH and dXp at the offsets moe_query reports)
 */
int moe_backward(const moe_cfg* cfg, const void* ring, size_t ring_bytes, int32_t slot,
                 const int32_t* offsets, const int32_t* row_src, const int32_t* tk_row,
                 const int32_t* topk_idx, const float* topk_w, const void* w_router,
                 const void* w1, const void* w2, const void* wq, size_t wq_bytes,
                 const void* saved, size_t saved_bytes, const void* dy, void* dx, void* dw1,
                 void* dw2, float* dwr, float* d_topk_w, int32_t accumulate, void* workspace,
                 size_t ws_bytes, moe_stream_t stream);

/*
 * The gate: a router beyond moe_route's renormalised top-k softmax. A call reads the router's
 * logits; moe_route_gated computes those first.
 *
 * Per token, over its row l of E logits (s, c in 64 bits):
 *   s_e = exp(l_e) / sum_i exp(l_i)  (MOE_SCORE_SOFTMAX)  or  1 / (1 + exp(-l_e))
 *         (MOE_SCORE_SIGMOID; 0 below l_e = -709);
 *   c_e = s_e + bias_e, the choice score (bias NULL: c_e = s_e). The bias, which a trainer moves
 *         to balance the experts' load, takes no part in the weights and has no gradient.
 *   groups > 1: the experts form `groups` equal runs of E / groups. A group scores its largest c
 *         (MOE_GROUP_MAX) or the sum of its two largest (MOE_GROUP_TOP2); the topk_groups best
 *         stay, equal ones by the lower index. groups 1 or topk_groups = groups: all stay.
 *   topk_idx[t,:] holds the k largest c of the groups that stay, in descending order; equal ones
 *         go to the lower index. Without a bias, and with groups 1 or MOE_GROUP_MAX, that is the
 *         order of the logits themselves.
 *   topk_w[t,j] = scale * s_j, or with renorm scale * s_j / sum_{i<k} s_i (0 where that sum is 0),
 *         rounded once to fp32.
 * A logit of -inf or NaN closes its expert: s_e = 0, c_e below every open expert's, and a closed
 * expert is chosen, with weight 0, only where fewer than k open ones stay (in index order). A
 * group's second-largest counts nothing if it is closed. Softmax entries equal to the row's
 * largest have exp 1, so several +inf share a row.
 */
enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 };
enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2 = 1 };
typedef struct moe_gate {
    int32_t score;       /* MOE_SCORE_* */
    int32_t groups;      /* >= 1, divides E */
    int32_t topk_groups; /* 1 .. groups; k <= topk_groups * (E / groups) */
    int32_t group_score; /* MOE_GROUP_* */
    int32_t renorm;      /* 0 or 1 */
    float scale;         /* finite */
} moe_gate;

/*
 * moe_gate_select - the choice and its weights from given logits. Needs no workspace.
 *
 *   logits   fp32 [T, E]    in
 *   bias     fp32 [E]       in, or NULL
 *   topk_idx int32 [T, k]   out
 *   topk_w   fp32 [T, k]    out
 * Errors (all the gate's calls): MOE_ERR_INVALID_ARG for a gate outside the ranges above.
 */
int moe_gate_select(const moe_cfg* cfg, const moe_gate* gate, const float* logits,
                    const float* bias, int32_t* topk_idx, float* topk_w, moe_stream_t stream);

/*
 * moe_route_gated - moe_route with the gate in place of its top-k softmax: the same logits, in
 * the same order of summation, then moe_gate_select. Arguments as in the two calls.
 */
int moe_route_gated(const moe_cfg* cfg, const moe_gate* gate, const void* x, const void* w_router,
                    const float* bias, float* logits, int32_t* topk_idx, float* topk_w,
                    void* workspace, size_t ws_bytes, moe_stream_t stream);

/*
 * moe_gate_backward - gradient of the logits from the gradient of the weights, the choice held.
 *
 * With g_j = scale * d_topk_w[t,j]:
 *   sigmoid            dl_j = g_j s_j (1 - s_j)
 *   sigmoid, renorm    dl_j = (g_j - sum_i g_i q_i) q_j (1 - s_j),  q_j = s_j / sum_i s_i
 *   softmax, renorm    dl_j = q_j (g_j - sum_i g_i q_i)
 *   softmax            dl_e = s_e ([e chosen] g_e - sum_i s_i g_i), for every expert e
 * and 0 for the experts not chosen in the first three. fp32, but for the sigmoids and their sum (64
 * bits, as in the choice); sums in a fixed order. The q of softmax come from the chosen logits
 * alone, and are not 0 where every chosen s_j underflows 64 bits (weights 0 in the forward). A
 * topk_idx entry outside [0, E) counts nothing; one expert named twice gets both slots' sum.
 *
 *   logits   fp32 [T, E]    in   (as given to the forward)
 *   topk_idx int32 [T, k]   in
 *   d_topk_w fp32 [T, k]    in   (from moe_backward)
 *   dlogits  fp32 [T, E]    out, or added to with accumulate != 0 (gradients of other losses of
 *                           the logits, a balance loss say, may be added before or after)
 * groups, topk_groups and group_score are checked, and change nothing here.
 */
int moe_gate_backward(const moe_cfg* cfg, const moe_gate* gate, const float* logits,
                      const int32_t* topk_idx, const float* d_topk_w, float* dlogits,
                      int32_t accumulate, moe_stream_t stream);

/*
 * moe_router_backward - gradients of the router's linear map logits = x w_router^T:
 *   dx[t]  = bf16( sum_e dlogits[t,e] w_router[e] )     (with acc_dx: that sum + dx[t], one
 *                                                        rounding of the fp32 total)
 *   dwr[e] = sum_t dlogits[t,e] x[t]                    (with acc_dwr: added to dwr[e])
 * Sums in fp32 in a fixed order (dlogits enters dwr with all its 24 bits, and dx, which is rounded
 * to bf16, with 17: an error of at most 2^-17 of each term). A dlogits value that is not finite
 * makes its token's dx and its expert's dwr NaN, and touches no other; for dx one that rounds to
 * an infinite bf16 (3.39e38 and above) counts as not finite.
 *
 *   x        bf16 [T, d]    in
 *   w_router bf16 [E, d]    in
 *   dlogits  fp32 [T, E]    in
 *   dx       bf16 [T, d]    out, or NULL (not wanted); not x itself
 *   dwr      fp32 [E, d]    out, or NULL (not wanted)
 */
int moe_router_backward(const moe_cfg* cfg, const void* x, const void* w_router,
                        const float* dlogits, void* dx, float* dwr, int32_t acc_dx,
                        int32_t acc_dwr, moe_stream_t stream);

/*
 * Block-scaled FP8: E4M3 codes with one fp32 scale per block of 128 along the reduction axis.
 * scale = amax / 448 and code = rne_e4m3(v * (448 / amax)), amax the block's largest magnitude
 * (a block of zeros: scale 1, codes 0; an amax below 2^-110 counts as 2^-110); the code stands for
 * code * scale. A value that is not finite gets the NaN code and takes no part in amax, so a
 * product is NaN where it reads one and nowhere else.
 *
 * moe_fp8_quantize_rows - rows of activations or gradients, a scale per 1 x 128.
 *   src    bf16 [rows, cols]          in, cols a multiple of 128
 *   codes  bytes [rows, cols]         out
 *   scales fp32 [cols / 128, rows]    out: one row of scales per 128 columns, so that the product
 *                                     reads a step's scales of consecutive rows together
 * rows 0 enqueues nothing; the three pointers may then be NULL.
 * Errors: MOE_ERR_INVALID_ARG, also where ceil(rows / 32) * ceil(cols / 512) >= 2^24.
 */
int moe_fp8_quantize_rows(const void* src, int32_t rows, int32_t cols, void* codes, float* scales,
                          moe_stream_t stream);

/*
 * moe_fp8_quantize_weights - weights, a scale per 128 x 128, in one pass over them; both
 * orientations if codes_t and scales_t are given (both or neither).
 *   src      bf16 [E, N, K]               in, N and K multiples of 128
 *   codes    bytes [E, N, K]              out
 *   scales   fp32 [E, N / 128, K / 128]   out
 *   codes_t  bytes [E, K, N]              out or NULL: the weights of the dgrad product
 *   scales_t fp32 [E, K / 128, N / 128]   out or NULL
 */
int moe_fp8_quantize_weights(const void* src, int32_t E, int32_t N, int32_t K, void* codes,
                             float* scales, void* codes_t, float* scales_t, moe_stream_t stream);

/*
 * moe_fp8_gemm - expert-grouped product of quantised rows and quantised weights:
 *   out[p, n] = sum_kb a_scales[kb, p] * b_scales[e, n / 128, kb] *
 *               sum_{k in block kb} a[p, k] * b[e, n, k]       for offsets[e] <= p < offsets[e+1]
 * Each block's sum leaves the matrix instruction in fp32 and is added, times its two scales, to
 * the fp32 total, which is rounded once to bf16. (Inside the instruction the products of eight
 * consecutive k are added on a grid of about 2^-13 of the largest of them, as gfx950 does for every
 * FP8 product.) No product of two scales may leave fp32's range. E = 1 with offsets {0, M} is a
 * plain product. The gradient of the rows is the same call on (d out quantised by rows, codes_t,
 * scales_t), N and K swapped. Needs no workspace.
 *
 *   offsets  int32 [E + 1]              in, ascending, within [0, M] (values outside are clamped).
 *                                       Rows of `out` before the first or behind the last expert's
 *                                       are left as they were.
 *   a        bytes [M, K]               in
 *   a_scales fp32 [K / 128, M]          in
 *   b        bytes [E, N, K]            in
 *   b_scales fp32 [E, N / 128, K / 128] in
 *   out      bf16 [M, N]                out
 * Shapes: 0 <= M < 2^31 (0 enqueues nothing; a, a_scales and out may then be NULL),
 * 1 <= E <= 1024, N and K multiples of 128, N * K < 2^31. Errors: MOE_ERR_INVALID_ARG.
 */
int moe_fp8_gemm(const int32_t* offsets, int32_t M, int32_t E, int32_t N, int32_t K, const void* a,
                 const float* a_scales, const void* b, const float* b_scales, void* out,
                 moe_stream_t stream);

/*
 * 8-bit integers: symmetric int8 codes with one fp32 scale a row - a token of the activations, an
 * output channel of the weights. scale = amax / 127 and code = rne(127 v / amax), amax the row's
 * largest magnitude (a row of zeros: scale 1, codes 0; an amax below 2^-110 counts as 2^-110); ties
 * are exact, so the codes are those of the quotient itself. A row that holds a value that is not
 * finite gets codes 0 and the scale NaN.
 *
 * moe_i8_quantize_rows - rows of activations, or weights [E, N, K] as their E * N rows.
 *   src    bf16 [rows, cols]   in, cols a multiple of 128
 *   codes  int8 [rows, cols]   out, -127 .. 127
 *   scales fp32 [rows]         out
 * rows 0 enqueues nothing; the three pointers may then be NULL.
 * Errors: MOE_ERR_INVALID_ARG, also for rows of 2^24 and more (a workgroup takes a row or four).
 */
int moe_i8_quantize_rows(const void* src, int32_t rows, int32_t cols, void* codes, float* scales,
                         moe_stream_t stream);

/*
 * moe_i8_gemm - expert-grouped product of int8 rows and weights:
 *   out[p, n] = bf16( a_scales[p] * (sum_k a[p, k] b[e, n, k]) * b_scales[e, n] )
 *                                                            for offsets[e] <= p < offsets[e + 1]
 * The sum is exact (32-bit integers), its two products are fp32, and the result is rounded once to
 * bf16. It does not depend on the other rows. E = 1 with offsets {0, M} is a plain product. Codes may
 * be -128 too. Needs no workspace.
 *
 *   offsets  int32 [E + 1]     in, ascending, within [0, M] (values outside are clamped). Rows of
 *                              `out` before the first or behind the last expert's are left as they
 *                              were.
 *   a        int8 [M, K]       in
 *   a_scales fp32 [M]          in
 *   b        int8 [E, N, K]    in
 *   b_scales fp32 [E, N]       in
 *   out      bf16 [M, N]       out
 * Shapes: 0 <= M < 2^31 (0 enqueues nothing; a, a_scales and out may then be NULL),
 * 1 <= E <= 1024, N and K multiples of 128, K < 2^17, N * K < 2^31, and (M / 128 + 2 E) * (N / 128)
 * below 2^24. Errors: MOE_ERR_INVALID_ARG.
 */
int moe_i8_gemm(const int32_t* offsets, int32_t M, int32_t E, int32_t N, int32_t K, const void* a,
                const float* a_scales, const void* b, const float* b_scales, void* out,
                moe_stream_t stream);

/* Activations of the gated products. In fp32; GELU by the error function or its tanh form. */
enum { MOE_ACT_SILU = 0, MOE_ACT_GELU = 1, MOE_ACT_GELU_TANH = 2, MOE_ACT_RELU = 3 };

/*
 * moe_i8_gemm_gated - moe_i8_gemm with the gate in its epilogue: with g and u the fp32 products of
 * a row and the weights' rows i and I + i,
 *   out[p, i] = bf16( act(g) * u )
 * so that neither projection is stored. The result is what moe_i8_quantize_rows takes before the
 * down product.
 *   b        int8 [E, 2I, K]   in: rows 0..I-1 gate, I..2I-1 up, as in W1
 *   b_scales fp32 [E, 2I]      in
 *   out      bf16 [M, I]       out
 * The rest, and the shapes with N = 2I (I a multiple of 128), are moe_i8_gemm's.
 */
int moe_i8_gemm_gated(const int32_t* offsets, int32_t M, int32_t E, int32_t I, int32_t K,
                      int32_t act, const void* a, const float* a_scales, const void* b,
                      const float* b_scales, void* out, moe_stream_t stream);

/*
 * The dense gated feed-forward block in bf16: the shared expert that every token passes beside its
 * routed ones, or a layer without experts. Shapes: T >= 1, d and I multiples of 128;
 * (T + 64) * max(d, 2I) < 2^31 and 4 * I * d < 2^31 (32-bit offsets).
 */
typedef struct moe_ffn {
    int32_t T;     /* tokens */
    int32_t d;     /* hidden size */
    int32_t I;     /* intermediate size */
    int32_t act;   /* MOE_ACT_* */
    int32_t flags; /* 0, or MOE_FLAG_BF16_DW: dw1 and dw2 are bf16 buffers instead of fp32 */
} moe_ffn;
typedef struct moe_ffn_sizes {
    size_t workspace; /* bytes of scratch that serve both calls (dH, partial sums) */
} moe_ffn_sizes;
int moe_ffn_query(const moe_ffn* ffn, moe_ffn_sizes* out);

/*
 * moe_ffn_forward
 *   [g | u] = x w1^T    A = act(g) * u    y = A w2^T    (with acc_y: y + A w2^T)
 * Sums are fp32 and outputs bf16, each rounded once; A is formed from the fp32 g and u, and y from
 * the rounded A. With acc_y the fp32 total of the stored y and the product is rounded once.
 *
 *   x   bf16 [T, d]     in
 *   w1  bf16 [2I, d]    in: rows 0..I-1 gate, I..2I-1 up
 *   w2  bf16 [d, I]     in
 *   H   bf16 [T, 2I]    out: [g | u], which moe_ffn_backward reads; or NULL (not wanted)
 *   A   bf16 [T, I]     out
 *   y   bf16 [T, d]     out (or added to); not x
 *   workspace bytes [ws_bytes]   scratch: calls that share one follow each other
 * H, A and y overlap neither one another nor an input.
 */
int moe_ffn_forward(const moe_ffn* ffn, const void* x, const void* w1, const void* w2, void* H,
                    void* A, void* y, int32_t acc_y, void* workspace, size_t ws_bytes,
                    moe_stream_t stream);

/*
 * moe_ffn_backward - gradients of <y, dy>:
 *   dA = dy w2    dH = bf16([dA * u * act'(g) | dA * act(g)])   (g, u from the stored H)
 *   dx  = dH w1      dw1 = dH^T x      dw2 = dy^T A
 * Sums are fp32. dx is rounded once to bf16, with acc_dx after the stored dx is added in fp32; dw1
 * and dw2 likewise with acc_dw (fp32, or bf16 with MOE_FLAG_BF16_DW). relu'(0) = 0.
 *
 *   x, w1, w2, H, A     in, as in moe_ffn_forward of the same batch
 *   dy  bf16 [T, d]     in
 *   dx  bf16 [T, d]     out (or added to); not x and not dy
 *   dw1 [2I, d]         out (or added to)
 *   dw2 [d, I]          out (or added to)
 *   workspace bytes [ws_bytes]   scratch
 * dx, dw1 and dw2 overlap neither one another nor an input.
 */
int moe_ffn_backward(const moe_ffn* ffn, const void* x, const void* w1, const void* w2,
                     const void* H, const void* A, const void* dy, void* dx, void* dw1, void* dw2,
                     int32_t acc_dx, int32_t acc_dw, void* workspace, size_t ws_bytes,
                     moe_stream_t stream);

/*
 * Launch tracing, for benchmarks and profilers; the layer never needs it.
 * moe_trace_begin: until moe_trace_end, every kernel the library enqueues is bracketed by two
 * hipEventRecord calls on the kernel's own stream: events[2i] before and events[2i+1] after the
 * i-th launch, for 2i+1 < capacity. names[i] receives the kernel's static name when names is
 * non-NULL. The caller creates the hipEvent_t handles (with timing enabled) and keeps them
 * alive. Not meant for concurrent use from several threads.
 *   events   hipEvent_t [capacity]   host array of caller-created events
 *   names    const char* [capacity/2] host array, or NULL
 * moe_trace_end stops tracing and returns the number of launches seen since moe_trace_begin
 * (launches beyond capacity/2 were counted but not timed).
 */
int moe_trace_begin(void* const* events, int capacity, const char** names);
int moe_trace_end(void);

/* A static string for a moe_status value (plumbing of this library, defined by no passage of
 * the pages). */
const char* moe_status_string(int status);

#ifdef __cplusplus
}
#endif
#endif /* MOE_MI355X_H */
