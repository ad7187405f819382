/*
 * moe_layer.h -- C ABI of the steps around the routed-expert product of
 * moe_prefill.h, for MI355X (gfx950):
 *
 *   moe_route             router logits -> topk expert ids and routing weights
 *                         (what moe_prefill_plan_device and moe_combine take)
 *   moe_route_balance     the same with the batch's balance statistics and loss
 *   moe_route_backward    the router's gradient: routing weights and loss -> logits
 *   moe_combine_backward  the combine's gradient: output -> routing weights, expert rows
 *   moe_adapters          low-rank adapters of many requests beside a shared projection
 *
 * The conventions are moe_prefill.h's: device pointers on the current device,
 * caller-owned buffers, host checks before anything is enqueued, a negative
 * moe_status with nothing launched on error, asynchronous work on `stream`,
 * no exception across the ABI, no device allocation, and results that do not
 * depend on scheduling (no floating-point atomics).  Every call may be
 * captured into a HIP graph (kernels only: no copies, no fills).  Every base
 * pointer is 16-byte aligned (MOE_EALIGN); a call over zero tokens does
 * nothing and accepts NULL buffers, but for the statistics of
 * moe_route_balance, which it writes as zeros.  Offsets inside a tensor are
 * 64-bit.  Two calls that may run at the same time need workspaces of their
 * own; a captured graph holds the workspace it was captured with.
 */
#ifndef MOE_LAYER_H
#define MOE_LAYER_H

#include "moe_prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of logits, activations and adapter matrices. */
typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_F16 = 2 } moe_dtype;

/* moe_route flag: the chosen experts' weights are renormalised to sum 1. */
enum { MOE_ROUTE_RENORM = 1 };

#define MOE_ROUTE_MAX_EXPERTS 2048 /* as moe_prefill_plan_device */
#define MOE_ROUTE_MAX_TOPK 64
#define MOE_ADAPTER_MAX_RANK 256
#define MOE_ADAPTER_MAX_TOKENS (1 << 24)

/* The router's choice.  With p[t] the softmax of logits row t,
 *   ids[t*topk + k]  the expert of the k-th largest logit (equal logits: the
 *                    lower expert first),
 *   w[t*topk + k]    scale * p[t][id], or with MOE_ROUTE_RENORM
 *                    scale * p[t][id] / sum over the chosen of p.
 *   logits   device [tokens x n_expert] of `dtype`, row t at element t*ld
 *            (ld >= n_expert)
 *   ids      device int32 [tokens x topk]; w: device fp32 [tokens x topk]
 *   flags    0 or MOE_ROUTE_RENORM
 * 1 <= topk <= min(n_expert, 64), n_expert <= 2048.
 * A logit of -inf closes its expert for the token: p = 0, and it is chosen
 * (lowest index first, weight 0) only when fewer than topk are open; with all
 * closed every weight is 0.  A row holding +inf or NaN gets NaN weights where
 * the softmax has none (NaN orders above +inf).  ids are distinct and in
 * range whatever the logits.  Sums are held in fp32. */
int moe_route(const void *logits, int64_t ld, int dtype, int tokens, int n_expert, int topk,
              int flags, float scale, int32_t *ids, float *w, void *stream);

/* Workspace of moe_route_balance (0 on invalid sizes).  It does not shrink as
 * tokens or n_seq grow: that of the largest batch serves every smaller one of
 * the same n_expert. */
size_t moe_balance_bytes(int tokens, int n_expert, int n_seq);

/* moe_route with the balance statistics of the batch's n_seq sequences.
 * Sequence s is rows [seq_off[s], seq_off[s+1]), n_s of them (seq_off: device
 * int32 [n_seq+1], non-decreasing, within [0, tokens]); rows outside are
 * padding: they are routed like the others but join no statistic.
 *   counts[s][e]  device int32 [n_seq x n_expert]: how often e was chosen in
 *                 sequence s, a choice of a closed expert not counted
 *   probs[s][e]   device fp32 [n_seq x n_expert]: the mean of p[t][e] over
 *                 the sequence's rows
 *   loss          device fp32 [1]: coef / n_seq * sum over s of
 *                 sum over e of (counts * n_expert / (topk * n_s)) * probs
 * (1 * coef when every expert is chosen equally often).  An empty sequence
 * has zero counts and probs and adds nothing.  n_seq >= 1.
 *   workspace     device, moe_balance_bytes(tokens, n_expert, n_seq) bytes
 *                 or more, 16-byte aligned, free again when the call's work has run */
int moe_route_balance(const void *logits, int64_t ld, int dtype, int tokens, int n_expert, int topk,
                      int flags, float scale, const int32_t *seq_off, int n_seq, float coef,
                      int32_t *ids, float *w, int32_t *counts, float *probs, float *loss,
                      void *workspace, size_t workspace_bytes, void *stream);

/* The gradient of moe_route / moe_route_balance with respect to the logits.
 * For token t of sequence s, with c[e] = dloss * coef * n_expert * counts[s][e]
 * / (n_seq * topk * n_s^2) (0 for padding rows, or without counts) and
 * g_k = dw[t][k] * scale (0 without dw):
 *   plain weights:  dlogits[e] = p[e] * (G[e] - sum p G), G = c + g at the chosen
 *   renormalised:   dlogits[e] = p[e] * (c[e] - sum p c)
 *                   + at the chosen q_k * (g_k - sum q g), q = p / sum chosen p
 * (the choice itself and the counts are constants, as usual).
 *   ids      device int32 [tokens x topk] from the forward call (an id named
 *            twice in a row adds twice; one out of range adds nothing)
 *   dw       device fp32 [tokens x topk], or NULL
 *   seq_off, counts  as moe_route_balance took and wrote them, or both NULL
 *            for no loss (n_seq is then ignored)
 *   dloss    device fp32 [1], the loss's own gradient; NULL means 1
 *   dlogits  device [tokens x n_expert] of the logits' type, row t at element
 *            t*ldd; may be the logits' own buffer (same pointer and stride)
 * Accumulated in fp32, rounded once. */
int moe_route_backward(const void *logits, int64_t ld, int dtype, int tokens, int n_expert, int topk,
                       int flags, float scale, const int32_t *ids, const float *dw,
                       const int32_t *seq_off, int n_seq, float coef, const int32_t *counts,
                       const float *dloss, void *dlogits, int64_t ldd, void *stream);

/* The gradient of moe_combine, out[t] = sum over k of w[t][k] * dm[t*topk+k]:
 *   dw[t][k]       = sum over n of dout[t][n] * dm[t*topk+k][n]   (fp32 sums)
 *   ddm[t*topk+k]  = w[t][k] * dout[t]
 * dm, ddm: device fp32 [tokens*topk x hidden]; w, dw: device fp32
 * [tokens x topk]; dout: device fp32 [tokens x hidden]; hidden % 4 == 0
 * (MOE_EFORMAT).  dw or ddm may be NULL (not both): without dw, dm may be
 * NULL; without ddm, w may be.  ddm may be dm itself (dw is that of the rows as
 * they were).  MOE_EINVAL if tokens * topk exceeds 2^30 or tokens *
 * ceil(topk / 8) exceeds 2^26 - 4 (the launch's thread count).  No plan is
 * needed, so the backward pass of a layer may run after its plan is gone. */
int moe_combine_backward(const float *dm, const float *w, const float *dout, int tokens, int topk,
                         int hidden, float *dw, float *ddm, void *stream);

/* A set of n_adapter low-rank adapters of one projection (all device memory,
 * read in place):
 *   dtype    MOE_BF16 or MOE_F16, of a and b
 *   rank     1..256 in steps of 8: rows of a, columns of b (an adapter of a
 *            smaller rank uses the first of them)
 *   n_in, n_out  the projection's sizes, multiples of 8
 *   a        [n_adapter][rank][n_in], b  [n_adapter][n_out][rank]
 *   scale    fp32 [n_adapter] (alpha / rank, as the user has it)
 *   ranks    int32 [n_adapter], each adapter's own rank, or NULL for `rank`
 *            everywhere; values are clamped to [0, rank] */
typedef struct {
    int dtype;
    int n_adapter;
    int rank;
    int n_in;
    int n_out;
    const void *a;
    const void *b;
    const float *scale;
    const int32_t *ranks;
} moe_adapter_set;

/* Workspace of moe_adapters over up to `tokens` rows (0 on invalid sizes): that
 * of the largest batch serves every smaller one of the same set. */
size_t moe_adapters_bytes(const moe_adapter_set *set, int tokens);

/* Low-rank adapters of many requests beside a projection all of them share
 * (2-bit expert weights cannot take an adapter in, so it runs beside them):
 *   out[t] = base[t] + scale[i] * b[i] * (a[i] * x[t]),   i = ids[t],
 * over the first ranks[i] rows of a[i] and columns of b[i]; a row whose id is
 * negative or >= n_adapter has no adapter: out[t] = base[t].
 *   tokens at most 2^24
 *   ids    device int32 [tokens], in any order (rows of one request usually
 *          stand together: prompts; or every row its own: new tokens)
 *   x      device [tokens x n_in], base and out: device [tokens x n_out], rows
 *          ldx, ldb, ldo elements apart (multiples of 8), all of `dtype`:
 *          MOE_F32, or the set's own 16-bit type (MOE_EFORMAT otherwise)
 *   out    base itself (same pointer and stride: rows without an adapter are
 *          then left as they are) or memory that shares no element with base;
 *          it shares none with x
 *   workspace  device, moe_adapters_bytes(set, tokens) bytes or more, 16-byte
 *          aligned, free again when the call's work has run
 * a * x is held in fp32, the result rounded once.  What a row holds reaches no
 * other row; an infinity in x, a, b or a * x may give NaN where the formula has
 * an infinity, and products below 2^-126 (also of the low bits of a value below
 * 2^-110) may count as 0.  A row's result does not depend on the rows beside it;
 * its last bits may on how many there are, by the order of its sums. */
int moe_adapters(const moe_adapter_set *set, const int32_t *ids, int tokens, int dtype,
                 const void *x, int64_t ldx, const void *base, int64_t ldb, void *out, int64_t ldo,
                 void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_LAYER_H */
