/*
 * libvloss: fused per-token losses over rows of vocabulary logits (GB300, sm_103a).
 *
 * One row of fp32 logits s (length V) per token.  Each row gets one
 * max / log-sum-exp reduction, m = max_j s_j, lnS = ln sum_j exp(s_j - m),
 * lse = m + lnS, from which the entry points below produce:
 *
 *   cross-entropy   loss = lse - s[label],  gradient scale * (softmax(s) - onehot(label))
 *                   (aprender-train 0.36.0, entrenar/autograd/wgpu_cross_entropy.rs:
 *                    module doc, forward_async, read_loss, backward);
 *   top-k KL        loss = sum_q p_q (ln p_q - (s[id_q] - lse)),
 *                   gradient coef * (softmax(s) - p_T), p_T the teacher's top-k
 *                   probabilities scattered onto their ids
 *                   (cortiq-engine 0.8.21, src/gpu_wgpu/train_head.rs: module doc, kl_rows);
 *   teacher top-k   the k largest logits, descending, ties to the lower id, with
 *                   probabilities renormalised over the k (train_head.rs: topk_rows);
 *   acc_add         a += b, the sum of per-slice partials (train_head.rs: acc_add, head_kl).
 *
 * Conventions shared by every entry point:
 *
 *  - Pointers are DEVICE pointers owned by the caller, except where a comment says
 *    otherwise.  The library allocates no memory and keeps no pointer after return.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy default
 *    stream).  They never synchronise and never read results back; argument errors
 *    are detected on the host and returned before anything is launched.
 *  - Logits are row-major fp32: row t starts at logits + t * ld; `ld >= V` is the
 *    row stride in elements.  Any alignment of `logits` and any `ld` is accepted
 *    (the kernels stream the 16-byte-aligned body of each row with bulk copies and
 *    handle up to 3 leading and 3 trailing elements with plain loads).
 *  - A vocabulary slice is the column range [col0, col0 + ncols) of every row;
 *    in-place entry points write exactly that range of rows [0, ntok) and nothing else.
 *  - The loss window [loss_start, loss_end), 0 <= loss_start <= loss_end <= ntok,
 *    selects the tokens that count (CEForwardParams / CEBackwardParams of the
 *    cross-entropy page).  Rows outside it get loss 0 and an all-zero gradient.
 *  - Labels and teacher ids are uint32.  A label or id >= V is a data error: it is
 *    counted into *err (when err is not NULL) with atomicAdd, its term is left out,
 *    and a CE loss with a bad label is NaN.  No kernel traps.
 *  - Row statistics `stats` are pairs (m, lnS) per row, [ntok][2] fp32.  They carry the
 *    log-sum-exp of a row between calls more precisely than lse itself: m is exact and
 *    lnS is small exactly when the row is peaked, so the softmax of a later sliced pass
 *    keeps full fp32 accuracy.  Passing only lse costs up to half an ulp of lse in the
 *    exponent of every softmax value.
 *  - A wait inside a kernel that exceeds about two seconds (a bug, never a normal
 *    condition) ends that kernel early with its outputs incomplete and sets a flag
 *    that vl_watchdog_flag() reports.
 */
#ifndef VLOSS_H
#define VLOSS_H

#include <stdint.h>

#if defined(__GNUC__)
#define VL_API __attribute__((visibility("default")))
#else
#define VL_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum vl_status {
    VL_OK = 0,
    VL_EINVAL = 1,        /* bad argument: NULL where required, size or window out of range */
    VL_ELAUNCH = 2,       /* a CUDA call failed; vl_last_error_string() says which */
    VL_EUNSUPPORTED = 3   /* valid request beyond this build's limits (e.g. k > VL_KL_KMAX) */
} vl_status;

/* Limits of this build. */
#define VL_KL_KMAX 1024      /* teacher support per row for vl_kl_topk_inplace */
#define VL_TOPK_KMAX 2048    /* k of vl_topk_rows (the page's bound for topk_rows) */
#define VL_MAX_COLS 0x7FFF0000LL   /* longest row V (2^31 - 2^16): rows are indexed with 32-bit ints */
#define VL_TOPK_NOALLOC_BYTES (32ll << 20)   /* fixed scratch of vl_topk_rows_noalloc (32 MiB a device) */

/* Library version, major * 10000 + minor * 100 + patch. */
VL_API int vl_version(void);

/* Static text for a status code. */
VL_API const char* vl_status_string(vl_status s);

/* Text of the last error raised on the calling host thread ("" if none). */
VL_API const char* vl_last_error_string(void);

/*
 * Cross-entropy forward (wgpu_cross_entropy.rs: module doc "loss = -logits[label] +
 * logsumexp(logits)", forward_async, read_loss).  Reads logits rows [0, ntok), columns
 * [0, V); writes for every row lse[t] (and stats[t] when not NULL), and loss[t] =
 * lse[t] - s_t[label_t] inside the window, 0 outside.  mean (nullable, one float) gets
 * sum of loss over the window / (loss_end - loss_start), 0 for an empty window, as
 * read_loss computes it.
 *   logits [ntok][ld] fp32 (read only)   labels [ntok] u32   loss [ntok] fp32
 *   lse [ntok] fp32 (nullable)           stats [ntok][2] fp32 (nullable)
 *   mean: one fp32 (nullable)            err: one int32 counter (nullable)
 */
VL_API vl_status vl_ce_fwd(const float* logits, int64_t ld, int64_t ntok, int64_t V,
                    const uint32_t* labels, int64_t loss_start, int64_t loss_end,
                    float* loss, float* lse, float* stats, float* mean,
                    int32_t* err, void* stream);

/*
 * Cross-entropy backward in place over a vocabulary slice (wgpu_cross_entropy.rs:
 * backward, "logits[i] = (softmax(logits)[i] - one_hot(label)[i]) * scale").  For rows in
 * the window, columns j in [col0, col0 + ncols):
 *     logits[t][j] = scale * (exp(s_t,j - lse_t) - [j == label_t]),
 * rows outside the window are zeroed.  The page fixes scale = 1 / max(1, window); here it
 * is the caller's argument.  The row statistics come from `stats` when not NULL, else from
 * `lse` (one of them is required).  loss_part (nullable) gets, per row, the slice's share
 * of the CE loss: lse - s[label] when the label lies in the slice and the row is in the
 * window, else 0.
 */
VL_API vl_status vl_ce_bwd_inplace(float* logits, int64_t ld, int64_t ntok, int64_t V,
                            int64_t col0, int64_t ncols, const uint32_t* labels,
                            const float* lse, const float* stats,
                            int64_t loss_start, int64_t loss_end, float scale,
                            float* loss_part, int32_t* err, void* stream);

/*
 * Cross-entropy forward and backward in one pass over each row: the row is read from
 * HBM once and the gradient written once.  Outputs as vl_ce_fwd, then logits rows are
 * overwritten as vl_ce_bwd_inplace does with col0 = 0, ncols = V.
 */
VL_API vl_status vl_ce_fused(float* logits, int64_t ld, int64_t ntok, int64_t V,
                      const uint32_t* labels, int64_t loss_start, int64_t loss_end,
                      float scale, float* loss, float* lse, float* stats, float* mean,
                      int32_t* err, void* stream);

/*
 * Top-k distillation KL with the gradient written in place (train_head.rs: module doc,
 * kl_rows; the float64 loop of head_kl_matches_host).  Per row t in the window:
 *     loss[t]     = sum over q with p_q > 0 and col0 <= id_q < col0 + ncols of
 *                   p_q * (ln p_q - (s[id_q] - lse_t))
 *     logits[t][j] = (coef + ce_coef) * exp(s_j - lse_t)
 *                    - coef * sum_{q: id_q = j} p_q - ce_coef * [j == label_t]
 * for j in [col0, col0 + ncols).  Rows outside the window: loss 0, slice zeroed.
 *   tid [ntok][k] u32, tp [ntok][k] fp32: the teacher's top-k ids and probabilities,
 *     taken as given (sum p = 1 is the caller's precondition; repeated ids add up).
 *   coef: the KL gradient coefficient (the page passes gscale / total).
 *   Row statistics: from stats_in when not NULL, else lse_in when not NULL, else
 *     computed here over the full row, which then requires col0 = 0 and ncols = V.
 *   labels (nullable) with ce_coef folds the CE gradient of the same row into this pass;
 *     the loss output stays the KL alone.  labels == NULL or ce_coef == 0: KL only.
 *   loss [ntok] fp32: the KL, or the slice's part of it for a slice (add the parts of
 *     all slices with vl_acc_add).
 * k must satisfy 1 <= k <= VL_KL_KMAX.
 */
VL_API vl_status vl_kl_topk_inplace(float* logits, int64_t ld, int64_t ntok, int64_t V,
                             int64_t col0, int64_t ncols,
                             const uint32_t* tid, const float* tp, int64_t k, float coef,
                             int64_t loss_start, int64_t loss_end,
                             const float* lse_in, const float* stats_in,
                             const uint32_t* labels, float ce_coef,
                             float* loss, int32_t* err, void* stream);

/*
 * Cross-entropy and top-k distillation KL of the same rows in one pass (the loss step of
 * train_head.rs head_kl -- one kl_rows over whole rows -- with the CE of
 * wgpu_cross_entropy.rs): each row is read from HBM once and its combined gradient is
 * written once, in place.  For rows t in the window:
 *     logits[t][j] = (coef + ce_coef) * exp(s_j - lse_t) - coef * sum_{q: id_q = j} p_q
 *                    - ce_coef * [j == label_t]
 *     kl_loss[t]   = sum over q with p_q > 0 of p_q * (ln p_q - (s[id_q] - lse_t))
 *     ce_loss[t]   = lse_t - s_t[label_t]  (NaN for a label >= V, counted in *err)
 * Rows outside the window: both losses 0, gradient row zeroed, lse and stats not written.
 * lse and stats (nullable) as vl_ce_fwd for the rows in the window; ce_mean (nullable) is
 * the mean of ce_loss over the window (as read_loss).  Long rows are split over a
 * thread-block cluster whose CTAs exchange their row statistics and loss parts through
 * distributed shared memory.
 *   labels [ntok] u32, tid [ntok][k] u32, tp [ntok][k] fp32 (as vl_kl_topk_inplace),
 *   kl_loss [ntok] fp32, ce_loss [ntok] fp32.  1 <= k <= VL_KL_KMAX.
 */
VL_API vl_status vl_ce_kl_fused(float* logits, int64_t ld, int64_t ntok, int64_t V,
                         const uint32_t* labels, const uint32_t* tid, const float* tp, int64_t k,
                         float coef, float ce_coef, int64_t loss_start, int64_t loss_end,
                         float* kl_loss, float* ce_loss, float* lse, float* stats, float* ce_mean,
                         int32_t* err, void* stream);

/*
 * bf16 logits (the page keeps f16 activations beside f32 logits, train_head.rs: Head,
 * head_kl's cvt / cvt_cols): the same five calls over rows of bf16 logits, given as
 * their 16-bit patterns (the upper half of an fp32).  Each row is read as bf16, every
 * maximum, sum, logarithm and exponential is taken in fp32, and each gradient element
 * is rounded to bf16 (nearest even) once, when it is written in place; losses, lse and
 * stats are fp32 as above.  Arguments, outputs and errors as in the fp32 calls; rows
 * may start at any 2-byte boundary, with any ld >= V.  Half the bytes of a row per pass.
 */
VL_API vl_status vl_ce_fwd_bf16(const uint16_t* logits, int64_t ld, int64_t ntok, int64_t V,
                    const uint32_t* labels, int64_t loss_start, int64_t loss_end,
                    float* loss, float* lse, float* stats, float* mean,
                    int32_t* err, void* stream);
VL_API vl_status vl_ce_bwd_inplace_bf16(uint16_t* logits, int64_t ld, int64_t ntok, int64_t V,
                            int64_t col0, int64_t ncols, const uint32_t* labels,
                            const float* lse, const float* stats,
                            int64_t loss_start, int64_t loss_end, float scale,
                            float* loss_part, int32_t* err, void* stream);
VL_API vl_status vl_ce_fused_bf16(uint16_t* logits, int64_t ld, int64_t ntok, int64_t V,
                      const uint32_t* labels, int64_t loss_start, int64_t loss_end,
                      float scale, float* loss, float* lse, float* stats, float* mean,
                      int32_t* err, void* stream);
VL_API vl_status vl_kl_topk_inplace_bf16(uint16_t* logits, int64_t ld, int64_t ntok, int64_t V,
                             int64_t col0, int64_t ncols,
                             const uint32_t* tid, const float* tp, int64_t k, float coef,
                             int64_t loss_start, int64_t loss_end,
                             const float* lse_in, const float* stats_in,
                             const uint32_t* labels, float ce_coef,
                             float* loss, int32_t* err, void* stream);
VL_API vl_status vl_ce_kl_fused_bf16(uint16_t* logits, int64_t ld, int64_t ntok, int64_t V,
                         const uint32_t* labels, const uint32_t* tid, const float* tp, int64_t k,
                         float coef, float ce_coef, int64_t loss_start, int64_t loss_end,
                         float* kl_loss, float* ce_loss, float* lse, float* stats, float* ce_mean,
                         int32_t* err, void* stream);

/*
 * Teacher top-k per row (train_head.rs: topk_rows): ids[t][q], q < k, are the columns of
 * the k largest logits of row t in descending order of value, ties broken by the lower
 * column (-0.0 equals +0.0); probs[t][q] = exp(s[ids[q]] - s[ids[0]]) / sum over the k.
 * The selection is exact (the page's per-thread best-8 is not).  Rows outside the window
 * are not written.  1 <= k <= min(V, VL_TOPK_KMAX).  NaN is a data error: a NaN value is
 * never selected, each row in the window that holds one adds 1 to *err (when err is not
 * NULL), and a row with fewer than k other values gets id 0xFFFFFFFF and probability 0
 * at the positions it cannot fill.  +-inf are ordinary values.
 * Time depends on the data: long rows are filtered with a threshold estimated from their
 * first 3840 columns, and a row for which fewer than k values reach it (one sorted in
 * descending order, for instance) is read a second time; the result is exact either way.
 *   ids [ntok][k] u32, probs [ntok][k] fp32, err: one int32 counter (nullable).
 *   workspace (nullable), workspace_bytes: device memory owned by the caller, 16-byte
 *     aligned, no initial contents needed.  Rows of 30720 to 2^20 columns with k up to
 *     about 6% of V are then streamed by one kernel whose filter warps write each row's
 *     candidates to the workspace while its finish warps order the previous row; the rare
 *     row it cannot settle goes to the exact kernel.  vl_topk_workspace_bytes gives the
 *     size for one CTA per SM of the current device; a smaller workspace that still holds
 *     one CTA's candidate regions runs fewer CTAs, and one below that (or none) has each
 *     row selected and ordered by the single exact kernel.  Same results either way.
 *     Calls that share a workspace must not overlap on the GPU.
 */
VL_API vl_status vl_topk_rows(const float* logits, int64_t ld, int64_t ntok, int64_t V, int64_t k,
                       int64_t loss_start, int64_t loss_end,
                       uint32_t* ids, float* probs, int32_t* err,
                       void* workspace, int64_t workspace_bytes, void* stream);

/*
 * vl_topk_rows for callers that cannot allocate device memory.  No counterpart on the
 * pages: it is the same selection, with its scratch taken from a fixed array in the
 * library instead of a workspace the caller passes.  It serves code that has no way to
 * get device memory at the point of the call: a custom memory pool or allocator hook that
 * calls into this library and must not re-enter the allocator, a latency-bound path that
 * may not risk an allocation (or its failure) there, or an embedded runtime with no device
 * allocator.  Results equal those of vl_topk_rows.
 *   The scratch is one array of VL_TOPK_NOALLOC_BYTES (32 MiB) that every device which
 *   loads the library holds until the process exits.  Rows of 30720 to 2^20 columns use
 *   it (shorter or longer rows need no scratch).  A call takes at most as many rows of
 *   the window as the array holds candidate regions and row list for (millions at
 *   V = 128256; 97 at V = 2^20 and k = 2048 on a 152-SM device); a larger window is
 *   rejected with VL_EUNSUPPORTED and a message that gives the limit (split it into calls).
 *   The first call on a device looks up the array's device address there (with that
 *   device current); make that first call before any stream capture.
 *   Every call shares the one array, which keeps the last call's contents (what must start
 *   at zero is cleared on the stream by each call); calls that overlap on the GPU -- on
 *   two streams, or from two host threads -- race on it and give wrong results.
 */
VL_API vl_status vl_topk_rows_noalloc(const float* logits, int64_t ld, int64_t ntok, int64_t V, int64_t k,
                               int64_t loss_start, int64_t loss_end,
                               uint32_t* ids, float* probs, int32_t* err, void* stream);

/*
 * Bytes of workspace with which vl_topk_rows streams ntok rows of V columns on one CTA per
 * SM of the current device (256 CTAs when no device is present): two sets of candidate
 * regions per CTA (about 60 KB at k = 256, 130 KB at k = 2048 for V = 128256) and 4 bytes a
 * row; 0 when rows of that length and k do not use a workspace (rows shorter than 30720 or
 * longer than 2^20 columns, or k above about 6% of V).
 */
VL_API int64_t vl_topk_workspace_bytes(int64_t ntok, int64_t V, int64_t k);

/*
 * Windowed mean of per-row losses (wgpu_cross_entropy.rs: read_loss, which sums the
 * losses and divides by loss_end - loss_start): *mean = sum of loss[loss_start, loss_end)
 * / (loss_end - loss_start), 0 for an empty window.  The same reduction as the mean
 * output of vl_ce_fwd / vl_ce_fused (a fixed-order double-float sum, so the result does
 * not depend on the launch), for losses produced piecewise, e.g. by calls over chunks of
 * the rows.  loss [ntok] fp32 (read only), mean: one fp32.
 */
VL_API vl_status vl_window_mean(const float* loss, int64_t ntok, int64_t loss_start, int64_t loss_end,
                                float* mean, void* stream);

/*
 * The frozen vocabulary head around the row losses, on chunks of rows so that the
 * [ntok][V] logits are never held whole (cortiq-engine train_head.rs: topk, head_kl).
 * hidden [ntok][hs] and w [V][hs] are bf16 (16-bit patterns), row-major, 16-byte
 * aligned, hs a multiple of 8.  Per chunk, logits = hidden . w^T with bf16 inputs and
 * fp32 accumulation and output (cuBLASLt: a plain dense GEMM), then this library's
 * kernels.  Everything stays on the stream: no host readback between chunks.
 * workspace: caller-owned device memory, 16-byte aligned, no initial contents needed;
 * the call takes as many rows per chunk as it holds (at least one row:
 * vl_*_workspace_bytes(1, ...)).  Calls that share a workspace must not overlap.
 *
 * vl_teacher_topk: ids/probs of the rows [loss_start, loss_end) as vl_topk_rows over the
 *   logits (the teacher's top-k, train_head.rs topk).
 * vl_head_kl: the student's head step (train_head.rs head_kl): per row, the CE + top-k
 *   KL losses and gradient of vl_ce_kl_fused over the logits (window, coef, ce_coef as
 *   there), the gradient rounded to bf16 (the page's cvt_cols), and
 *   dx[t] = dx_scale * sum_j g[t][j] * w[j]  (the page's mm(wt, ..., 1/gscale)),
 *   fp32 [ntok][hs], 16-byte aligned; rows outside the window get dx = 0.  ce_mean
 *   (nullable): the windowed mean of ce_loss.  wt (nullable): the transposed weight
 *   plane [hs][V] bf16, 16-byte aligned, as the page keeps for this GEMM; with it (and V
 *   a multiple of 8) both GEMMs run on the tensor-core kernel of vl_gemm_bf16_tn, without
 *   it the dx GEMM reads w through cuBLASLt.
 */
/*
 * The head's GEMM on the 5th-generation tensor cores: D[M][N] = alpha * A[M][K] . B[N][K]^T,
 * A and B bf16 (16-bit patterns), row-major, 16-byte aligned, K a multiple of 8; D fp32,
 * row-major with stride ldd >= N.  fp32 accumulation in tensor memory (tcgen05.mma fed by
 * TMA).  Logits are hidden . W^T; the backward dlogits . wt^T with the transposed weight
 * plane wt (train_head.rs keeps one per slice for that GEMM).
 */
VL_API vl_status vl_gemm_bf16_tn(const uint16_t* A, const uint16_t* B, float* D, int64_t M, int64_t N, int64_t K,
                          int64_t ldd, float alpha, void* stream);

VL_API int64_t vl_teacher_topk_workspace_bytes(int64_t rows, int64_t V, int64_t k);
VL_API vl_status vl_teacher_topk(const uint16_t* hidden, int64_t hs, const uint16_t* w, int64_t V, int64_t ntok,
                          int64_t k, int64_t loss_start, int64_t loss_end, uint32_t* ids, float* probs,
                          int32_t* err, void* workspace, int64_t workspace_bytes, void* stream);
VL_API int64_t vl_head_kl_workspace_bytes(int64_t rows, int64_t V);
VL_API vl_status vl_head_kl(const uint16_t* hidden, int64_t hs, const uint16_t* w, const uint16_t* wt, int64_t V,
                     int64_t ntok,
                     const uint32_t* labels, const uint32_t* tid, const float* tp, int64_t k, float coef,
                     float ce_coef, float dx_scale, int64_t loss_start, int64_t loss_end, float* dx,
                     float* kl_loss, float* ce_loss, float* ce_mean, int32_t* err, void* workspace,
                     int64_t workspace_bytes, void* stream);

/*
 * a[i] = a[i] + b[i] for 0 <= i < n, fp32, bit-exact (train_head.rs: acc_add, which adds a
 * later vocabulary slice's partial to the first one's).  a and b may not overlap unless
 * a == b.
 */
VL_API vl_status vl_acc_add(float* a, const float* b, int64_t n, void* stream);

/*
 * ---------------------------------------------------------------- post-training
 *
 * Policy and preference training over the same rows of logits, the layer norm in front of
 * the head, and the head's product in 8-bit floating point.  No counterpart on the pages;
 * the formulas stand with each call.  The conventions above hold; in these calls:
 *  - `weight` [ntok] fp32 takes the place of the loss window: a row of weight 0 (a prompt
 *    or padding token) is not read at all (its logits may be anything, NaN included), has
 *    loss, log-probability and KL 0 and a zero gradient row.
 *  - `grad` [ntok][ldg] receives the gradient of the logits, in the logits' type; it may be
 *    `logits` itself (then ldg == ld: in place), must not overlap it otherwise (rows of the same
 *    stride may lie between its rows, as the halves of a wider buffer do), and may be NULL
 *    where no gradient is wanted.  Writes are 16 bytes wide when grad and logits rows
 *    agree in their alignment modulo 16 bytes, else narrower (same results).
 *  - a logit of -inf is an ordinary value (probability 0).
 *  - scaling logits by a temperature belongs to the head's product (its alpha).
 */

/*
 * Clipped policy loss with a KL term, forward and backward, over rows of logits.  Per row t
 * with weight w != 0 (a = actions[t], A = adv[t]):
 *     logp  = s[a] - lse                      r  = exp(logp - old_logp[t])
 *     pg    = -min(r A, clip(r, 1 - clip_lo, 1 + clip_hi) A)
 *     kl    = exp(q) - q - 1, q = ref_logp[t] - logp     (0 when ref_logp is NULL)
 *     loss  = w (pg + kl_coef kl)
 *     G     = d loss / d logp = w (-[r A not above its clipped value] r A + kl_coef (1 - exp(q)))
 *     grad[t][j] = scale G ([j == a] - softmax(s)_j)
 * The weights carry the mask and the averaging (over tokens, sequences or groups alike).
 *   actions [ntok] u32; old_logp, adv, weight [ntok] fp32; ref_logp [ntok] fp32 (nullable);
 *   0 <= clip_lo <= 1, clip_hi >= 0 (a positive infinity switches that side's clip off).
 *   loss [ntok] fp32; logp, kl [ntok] fp32 (nullable); total: one fp32, the sum of loss
 *   (nullable); err: one int32 (nullable).
 * A row whose factor scale * G is 0 (a clipped one) has a gradient row of zeros.  An action
 * >= V is counted in *err; its loss and logp are NaN, its gradient row is zero.
 * Rows of up to VL_POLICY_ONEPASS_COLS columns are read from HBM once; longer ones twice.
 */
#define VL_POLICY_ONEPASS_COLS 245760
VL_API vl_status vl_policy_loss(const float* logits, int64_t ld, int64_t ntok, int64_t V,
                         const uint32_t* actions, const float* old_logp, const float* ref_logp,
                         const float* adv, const float* weight, float clip_lo, float clip_hi, float kl_coef,
                         float scale, float* grad, int64_t ldg, float* loss, float* logp, float* kl,
                         float* total, int32_t* err, void* stream);
VL_API vl_status vl_policy_loss_bf16(const uint16_t* logits, int64_t ld, int64_t ntok, int64_t V,
                         const uint32_t* actions, const float* old_logp, const float* ref_logp,
                         const float* adv, const float* weight, float clip_lo, float clip_hi, float kl_coef,
                         float scale, uint16_t* grad, int64_t ldg, float* loss, float* logp, float* kl,
                         float* total, int32_t* err, void* stream);

/*
 * Preference loss over pairs of sequences, forward and backward.  The rows of sequence s,
 * s < 2 npairs, are [seq_start[s], seq_start[s + 1]); pair i prefers sequence i (chosen) to
 * sequence npairs + i (rejected), as a concatenated batch lays them.  With logp_t the
 * log-probability of labels[t]:
 *     pi_s  = sum over its rows of weight_t logp_t      (weights 1, or 1 / length for a mean)
 *     gap_i = (pi_i - ref_i) - (pi_{npairs+i} - ref_{npairs+i}),   h = beta gap
 *     VL_PREF_SIGMOID  loss = -(1 - smooth) ln sigmoid(h) - smooth ln sigmoid(-h)
 *     VL_PREF_IPO      loss = (gap - 1 / (2 beta))^2                  (smooth is not used)
 *     VL_PREF_HINGE    loss = max(0, 1 - h)                           (smooth is not used)
 *     grad[t][j] = scale (d loss_i / d pi_s) weight_t ([j == labels[t]] - softmax(s_t)_j)
 * (scale = 1 / npairs gives the gradient of the mean.)  Sequence sums are taken in pairs of fp32 (about 48 bits) in
 * a fixed order.
 *   labels [ntok] u32; weight [ntok] fp32; seq_start [2 npairs + 1] int64, ascending, in
 *   [0, ntok] (values outside are clamped; rows of no sequence get a zero gradient);
 *   ref_logp [2 npairs] fp32, the reference model's pi_s (nullable: zeros).
 *   beta > 0, 0 <= smooth < 1.  npairs >= 1 unless ntok == 0.
 *   loss, margin (= h) [npairs] fp32; seq_logp (pi_s) [2 npairs] fp32 (nullable); mean: one
 *   fp32, the mean of loss (nullable); err: one int32 (nullable).
 *   workspace: vl_preference_workspace_bytes(ntok, npairs) bytes of device memory, 16-byte
 *   aligned, no initial contents needed; calls that share one must not overlap on the GPU.
 * A pair with a label >= V (in a row of weight != 0) has loss, margin and pi_s NaN and zero
 * gradient rows; each such label is counted in *err.
 * A label of probability 0 (logit -inf) makes its pi_s -inf.  In the rejected sequence: margin +inf and, without
 * smoothing, loss 0 and no gradient; in the chosen one: loss +inf and the slope's limit in the gradient (the
 * squared loss has no limit: its gradient is not finite); in both: NaN.
 */
typedef enum vl_pref_kind { VL_PREF_SIGMOID = 0, VL_PREF_IPO = 1, VL_PREF_HINGE = 2 } vl_pref_kind;
VL_API int64_t vl_preference_workspace_bytes(int64_t ntok, int64_t npairs);
VL_API vl_status vl_preference_loss(const float* logits, int64_t ld, int64_t ntok, int64_t V,
                         const uint32_t* labels, const float* weight, const int64_t* seq_start, int64_t npairs,
                         const float* ref_logp, float beta, float smooth, int kind, float scale,
                         float* grad, int64_t ldg, float* loss, float* margin, float* seq_logp, float* mean,
                         int32_t* err, void* workspace, int64_t workspace_bytes, void* stream);
VL_API vl_status vl_preference_loss_bf16(const uint16_t* logits, int64_t ld, int64_t ntok, int64_t V,
                         const uint32_t* labels, const float* weight, const int64_t* seq_start, int64_t npairs,
                         const float* ref_logp, float beta, float smooth, int kind, float scale,
                         uint16_t* grad, int64_t ldg, float* loss, float* margin, float* seq_logp, float* mean,
                         int32_t* err, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Layer norm over rows of hs elements (the norm in front of the head):
 *     mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps), xh = (x - mu) rstd
 *     y  = xh gamma + beta
 *   x [rows][ldx], y [rows][ldy] fp32, or bf16 in the _bf16 calls (sums in fp32, each output
 *   rounded once); gamma, beta [hs] fp32 (nullable: 1 and 0); mu, rstd [rows] fp32 (nullable).
 *   y may be x itself (ldy == ldx), or lie between its rows.  1 <= hs <= VL_NORM_MAX_HS; any alignment and strides.
 * Backward, with t = dy gamma:
 *     dx = rstd (t - mean(t) - xh mean(t xh)),  dgamma = sum over rows of dy xh,  dbeta = sum of dy
 *   dy fp32 (in the _bf16 call: bf16, or fp32 when dy_f32 != 0, as the head's products hand
 *   it back); mu, rstd as the forward pass wrote them; dx in x's type, may be x itself, or dy
 *   when the types agree (then with the same stride); dgamma, dbeta [hs] fp32 (nullable), summed in a fixed
 *   order: the same bits on every call.  With rows == 0 they are set to 0.
 *   workspace: vl_layernorm_bwd_workspace_bytes(rows, hs) bytes, 16-byte aligned, needed when
 *   dgamma or dbeta is given; calls that share one must not overlap on the GPU.
 */
#define VL_NORM_MAX_HS 16384
VL_API vl_status vl_layernorm_fwd(const float* x, int64_t ldx, int64_t rows, int64_t hs, const float* gamma,
                         const float* beta, float eps, float* y, int64_t ldy, float* mu, float* rstd, void* stream);
VL_API vl_status vl_layernorm_fwd_bf16(const uint16_t* x, int64_t ldx, int64_t rows, int64_t hs, const float* gamma,
                         const float* beta, float eps, uint16_t* y, int64_t ldy, float* mu, float* rstd, void* stream);
VL_API int64_t vl_layernorm_bwd_workspace_bytes(int64_t rows, int64_t hs);
VL_API vl_status vl_layernorm_bwd(const float* dy, int64_t lddy, const float* x, int64_t ldx, int64_t rows, int64_t hs,
                         const float* gamma, const float* mu, const float* rstd, float* dx, int64_t lddx,
                         float* dgamma, float* dbeta, void* workspace, int64_t workspace_bytes, void* stream);
VL_API vl_status vl_layernorm_bwd_bf16(const void* dy, int dy_f32, int64_t lddy, const uint16_t* x, int64_t ldx,
                         int64_t rows, int64_t hs, const float* gamma, const float* mu, const float* rstd,
                         uint16_t* dx, int64_t lddx, float* dgamma, float* dbeta, void* workspace,
                         int64_t workspace_bytes, void* stream);

/*
 * The head's product in 8-bit floating point (e4m3) with a scale for each block of 128 of the
 * contraction: D[m][n] = alpha sum over k-blocks b of sa[b][m] sb[n / 128][b]
 * sum over k in b of A[m][k] B[n][k].  Each block's sum comes from the tensor cores; the
 * scaled sum over blocks is kept in fp32.
 *   A [M][K], B [N][K] e4m3 bytes, row-major, 16-byte aligned, K a multiple of 16;
 *   sa [ceil(K/128)][M], sb [ceil(N/128)][ceil(K/128)] fp32; D [M][ldd] fp32.
 * With a frozen head: logits = hidden . W^T; and dx = g . Wt^T over the transposed plane Wt
 * [hs][V], whose 128 x 128 blocks have the transposed scales.  On the way back V is the contraction: a
 * vocabulary that is no multiple of 16 is padded to Vp, the next one.  Logits and gradient get rows of
 * stride Vp whose columns past V are zeroed once (neither the product forward, N = V and ldd = Vp, nor the
 * losses write them), the gradient is quantised with K = Vp, and Wt is [hs][Vp] with zeros past V.
 *
 * The quantisers: over each block, scale = max(amax, 2^-100) * fp32(1 / 448), rounded to fp32,
 * and q = x / scale (an fp32 division) rounded to the nearest e4m3, ties to even, at most 448.  A NaN stays NaN, an infinity
 * makes its block's values 0 or NaN with an infinite scale, so that the product is NaN.
 * vl_quant_fp8_rows (fp32 x) / _bf16: blocks of 1 x 128, x [M][ldx] -> q [M][K], sa as above.
 * vl_quant_fp8_blocks_bf16: blocks of 128 x 128, w [N][K] bf16 (contiguous) -> q [N][K], sb.
 * K is at most 2^30 in all of them.
 */
VL_API vl_status vl_quant_fp8_rows(const float* x, int64_t ldx, int64_t M, int64_t K, uint8_t* q, float* sa,
                         void* stream);
VL_API vl_status vl_quant_fp8_rows_bf16(const uint16_t* x, int64_t ldx, int64_t M, int64_t K, uint8_t* q, float* sa,
                         void* stream);
VL_API vl_status vl_quant_fp8_blocks_bf16(const uint16_t* w, int64_t N, int64_t K, uint8_t* q, float* sb, void* stream);
VL_API vl_status vl_gemm_fp8_tn(const uint8_t* A, const float* sa, const uint8_t* B, const float* sb, float* D,
                         int64_t M, int64_t N, int64_t K, int64_t ldd, float alpha, void* stream);

/*
 * Rows in 4-bit floating point (e2m1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) with a scale for each small block
 * of columns, and the head's product over them.  Two formats:
 *   VL_FP4_NV   blocks of 16 columns with an e4m3 scale, and an fp32 scale rs[m] for each row;
 *   VL_FP4_MX   blocks of 32 columns with a power of two (e8m0); rs is NULL.
 * A value stands for q s r (r = 1 in MX).
 *   q   [M][Kp / 2] bytes, Kp the next multiple of 32 from K: two values a byte, the even column in the low half, columns
 *       past K zero; 16-byte aligned;
 *   sf  vl_fp4_scale_bytes(M, K, fmt) bytes, 16-byte aligned: tiles of 128 rows x 4 blocks, 512 bytes each, tile (m / 128,
 *       b / 4) the (m / 128) * ceil(ceil(K / block) / 4) + b / 4-th; in it row m, block b at byte
 *       16 (m % 32) + 4 (m % 128 / 32) + b % 4.  Blocks past K in the last tile are zero; rows past M are left as they are
 *       and never matter;
 *   rs  [M] fp32 (NV).
 *
 * vl_quant_fp4_rows (fp32 x) / _bf16, x [M][ldx]; every operation rounded to fp32 to nearest even:
 *   NV  r = max(amax of the row, 2^-100) * fp32(1 / 2688); s = e4m3((amax of the block * fp32(1 / 6)) * (1 / r)), nearest
 *       even; q = e2m1(x * (1 / (s * r))), nearest even, at most 6 (s = 0: 0).  A row that holds a NaN or an infinity gets
 *       r = NaN and zeros, so that its products are NaN.  A row's result does not depend on other rows.
 *   MX  s = 2^(floor(log2(amax of the block)) - 2), at least 2^-127 (amax = 0: 2^-127); q = e2m1(x / s), at most 6.  A
 *       block that holds a NaN or an infinity gets s = NaN and zeros.
 * vl_dequant_fp4_rows / _bf16: y [M][ldy] = (q s) r in fp32 (q s is exact), then rounded to bf16 there.  With the
 * quantiser before it: rows as a model trained for 4 bits sees them; states kept in 4 bits read back.
 * M is at most 2^31, K 2^30; buffers may not overlap.
 *
 * vl_gemm_fp4_tn: D[m][n] = alpha * ra[m] * rb[n] * sum over k of (qa sa)[m][k] (qb sb)[n][k], in fp32 (_bf16: rounded once
 * when written; the factors in an order that keeps what is between them in fp32 where the result is, for alpha 0 or of magnitude
 * 2^-100 upwards).  Products are exact, sums fp32 in the tensor cores; A [M][Kp/2], B [N][Kp/2] with scales as above,
 * D [M][ldd].  K is any length from 1.  Logits from hidden rows and a head plane W [V][hs]; and dx = g . Wt^T over the transposed
 * plane Wt [hs][V], quantised by itself (its blocks run along V).
 */
#define VL_FP4_NV 0
#define VL_FP4_MX 1
VL_API int64_t vl_fp4_scale_bytes(int64_t M, int64_t K, int fmt);
VL_API vl_status vl_quant_fp4_rows(const float* x, int64_t ldx, int64_t M, int64_t K, int fmt, uint8_t* q, uint8_t* sf,
                         float* rs, void* stream);
VL_API vl_status vl_quant_fp4_rows_bf16(const uint16_t* x, int64_t ldx, int64_t M, int64_t K, int fmt, uint8_t* q,
                         uint8_t* sf, float* rs, void* stream);
VL_API vl_status vl_dequant_fp4_rows(const uint8_t* q, const uint8_t* sf, const float* rs, int64_t M, int64_t K, int fmt,
                         float* y, int64_t ldy, void* stream);
VL_API vl_status vl_dequant_fp4_rows_bf16(const uint8_t* q, const uint8_t* sf, const float* rs, int64_t M, int64_t K,
                         int fmt, uint16_t* y, int64_t ldy, void* stream);
VL_API vl_status vl_gemm_fp4_tn(const uint8_t* A, const uint8_t* sfa, const float* ra, const uint8_t* B,
                         const uint8_t* sfb, const float* rb, float* D, int64_t M, int64_t N, int64_t K, int64_t ldd,
                         int fmt, float alpha, void* stream);
VL_API vl_status vl_gemm_fp4_tn_bf16(const uint8_t* A, const uint8_t* sfa, const float* ra, const uint8_t* B,
                         const uint8_t* sfb, const float* rb, uint16_t* D, int64_t M, int64_t N, int64_t K, int64_t ldd,
                         int fmt, float alpha, void* stream);

/*
 * Verification of drafted tokens against the target's probabilities, from given random numbers.  Sequence i brings
 * k = seq_start[i + 1] - seq_start[i] drafted tokens (0 upwards), rows seq_start[i] .. of `drafted`, `u` and `draft`, and
 * k + 1 rows of the target's logits, from row seq_start[i] + i of `target` on: row j of them is what follows
 * the first j drafted tokens.  With p_j, q_j the softmax of target and draft row j at the sequence's temperature:
 *   token j is accepted, in order, while u[j] * q_j(token) < p_j(token);
 *   at the first token refused the next one is drawn from max(p_j - q_j, 0) (from p_j where that is nothing), after k
 *   accepted ones from p_k: the first column whose running sum exceeds pick[i] * (the sum over all columns).
 * Accepted and drawn tokens are then distributed as the target's own.  draft = NULL: the drafter proposes without
 * probabilities, q_j is 1 at its token.  temperature 0: greedy, a token is accepted if it is the target's largest
 * (the lowest column of equal ones), and the next one is that; u, pick and draft are not used.  k = 0 draws from the target.
 *   target [ndraft + nseq][ldt], draft [ndraft][ldd] (nullable) fp32 or bf16; -inf bans a column, as does any number far below
 *       the row's largest (-1e10, the type's lowest)
 *   seq_start [nseq + 1] int64 (device), 0 to ndraft, not falling       drafted [ndraft] u32    u [ndraft], pick [nseq] fp32 in [0, 1)
 *       (1 too, as rounding a number below it may give)
 *   temperature [nseq] fp32, 0 or in [1e-6, 1e6] (nullable: 1)
 *   tokens [ndraft + nseq] u32: from place seq_start[i] + i the accepted tokens, the next one, then 0xFFFFFFFF
 *   accepted [nseq] int32: how many were accepted
 *   logp [ndraft + nseq] fp32 (nullable): ln p of each of these tokens (greedy: at temperature 1), 0 past the last
 * Data errors, counted into *err (nullable) once a sequence: a drafted token >= V is refused; a row of target or draft
 * that is reached and has no softmax (a NaN, +inf, or no column that is not banned), or a temperature out of range, ends the
 * sequence there with 0xFFFFFFFF as its next token.  Rows after the first refused token, with their tokens and random numbers,
 * never matter, but may be read (two to eight positions at once): they have to be readable memory that nothing writes meanwhile.
 * A sequence's result does not depend on the others, bit for bit where its rows begin at 16 bytes, or at the same place within
 * 16; at another place (rows of another number of bytes) the sums are taken in another order.
 * V is at most 2^30; the magnitude of a row's largest logit 2^30 times the temperature (beyond it a row may have no softmax).
 * Outputs may not overlap inputs.
 */
#define VL_VERIFY_MAX_SEQS (1LL << 24)
VL_API vl_status vl_verify_draft(const float* target, int64_t ldt, const float* draft, int64_t ldd, int64_t V,
                         const int64_t* seq_start, int64_t nseq, int64_t ndraft, const uint32_t* drafted,
                         const float* temperature, const float* u, const float* pick, uint32_t* tokens, int32_t* accepted,
                         float* logp, int32_t* err, void* stream);
VL_API vl_status vl_verify_draft_bf16(const uint16_t* target, int64_t ldt, const uint16_t* draft, int64_t ldd, int64_t V,
                         const int64_t* seq_start, int64_t nseq, int64_t ndraft, const uint32_t* drafted,
                         const float* temperature, const float* u, const float* pick, uint32_t* tokens, int32_t* accepted,
                         float* logp, int32_t* err, void* stream);

/*
 * Test hook for the failure path (no counterpart on the pages).  Arms the next row-engine
 * launch (vl_ce_fwd, vl_ce_bwd_inplace, vl_ce_fused, vl_kl_topk_inplace) made from the
 * calling host thread: CTA 0 of that launch stops issuing its row tiles at body tile
 * number withhold_tile (counted over the CTA's tiles in issue order), and every wait of
 * the launch gives up after wait_cycles SM cycles instead of about two seconds.  The
 * consumers' wait for the missing tile then runs out: the kernel raises the watchdog
 * flag, lets the copies already issued land, and returns with that CTA's outputs
 * incomplete; the other CTAs' rows are unaffected.  Nothing faults or hangs.
 * 1000 <= wait_cycles <= 4e9.  The setting is used once, then cleared.
 */
VL_API vl_status vl_test_inject_wait_timeout(int64_t withhold_tile, int64_t wait_cycles);

/*
 * Reads (and with clear != 0 resets) the flag that a kernel wait timed out on `device`.
 * Synchronous: it waits for the device to finish its work.  Returns -1 if the read fails.
 */
VL_API int vl_watchdog_flag(int device, int clear);

#ifdef __cplusplus
}
#endif

#endif /* VLOSS_H */
