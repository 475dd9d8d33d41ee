/*
 * qstep.h - C ABI of what stands around the block-quantized products of
 * qgemv.h and the attention of qattn.h in a generation step: the norms before
 * and after a block with its gate and residual, and the choice of the next
 * tokens from the logits.
 *
 * The reference pages stop at the products; the operators here are defined by
 * the formulas at each call.
 *
 * Conventions (those of qgemv.h, and)
 *   - Status codes, the stream argument, qg_last_cuda_error and
 *     qg_device_error are qgemv.h's. Argument errors are returned before
 *     anything is enqueued; no call synchronizes or allocates.
 *   - Pointers are device pointers unless said otherwise. Strides are in
 *     elements, from row to row. Sizes, strides and alignments are free down
 *     to the type's own size (QG_ERR_ALIGN below that) unless a call says
 *     more; rows on 16-byte boundaries are read faster.
 *   - A kernel may start while the one enqueued before it finishes
 *     (programmatic dependent launch) but touches memory only after it.
 */
#ifndef GB300_QSTEP_H
#define GB300_QSTEP_H

#include "qgemv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Norms around a block -------------------------------------------------- */

/* Arguments of qnorm_residual (host struct). */
typedef struct {
    const void *h;        /* h_type [n][d], the residual stream               */
    const void *y;        /* y_type [n][d], a block's result, or NULL         */
    int64_t h_stride, y_stride;
    const float *post_w, *post_b; /* [d], the norm of y; post_w NULL: y is
                             taken as it is; post_b NULL: none                */
    const float *gate;    /* [n][d] with gate_stride, 0 for one row that all
                             share; NULL: 1                                   */
    int64_t gate_stride;
    const float *w, *b;   /* [d], the norm of the new h; NULL: 1 and none     */
    void *h_out;          /* h_type [n][d] with h_out_stride, or NULL         */
    int64_t h_out_stride;
    void *x_out;          /* x_type [n][d] contiguous, or NULL                */
    void *xq;             /* the rows of x in blocks of act_type, or NULL     */
    int64_t n, d;
    int32_t h_type, y_type, x_type; /* QG_F32 or QG_F16                       */
    int32_t act_type;     /* QG_Q8_0, QG_Q8_1 or QG_Q8_K (with xq)            */
    int32_t layer;        /* 0: N divides by the root mean square; not 0: the
                             mean is taken off first                          */
    float scale, eps;
} qnorm_args;

/* For each row
 *   h' = h + scale * gate * N(y; post_w, post_b)    (h' = h without y)
 *   x  = N(h'; w, b)
 *   N(v; w, b) = v / sqrt(mean(v^2) + eps) * w + b, or with layer
 *                (v - m) / sqrt(mean((v - m)^2) + eps) * w + b, m = mean(v)
 * computed in f32, each output rounded once: x follows from h' before its
 * rounding to h_type. xq holds what quantize_act(act_type) makes of x in f32,
 * byte for byte, for qgemv_xq: d is a multiple of its block then, every array that
 * is given lies on a 16-byte boundary, and its stride is a multiple of
 * 16 bytes. At least one of h_out, x_out and xq is given. h_out may be h
 * (same stride); x_out may be h or y where type and stride are the same and
 * h_out is not that one too. Infinities and NaN in a row stay in that row.
 * 1 <= d <= 16384, n <= 2^30. Deterministic. */
int qnorm_residual(const qnorm_args *args, qg_stream_t stream);

/* ---- The next tokens -------------------------------------------------------- */

/* Chooses one token for each of n rows of logits (type QG_F32 or QG_F16,
 * [n][vocab] with `stride`) from given random numbers. With m the row's largest
 * logit, T = temperature[r], the tokens' weights are w_i = exp((l_i - m) / T);
 * kept are
 *   of all tokens the top_k[r] of largest logit (<= 0: all),
 *   of those, by falling logit, the ones before which less than top_p[r] times
 *     their weights' sum has been passed (>= 1: all; the first always stays),
 *   of those, the ones with w_i >= min_p[r] (the first always stays);
 * equal logits count in the order of their indexes. The token is the first, in
 * the order of the indexes, at which the sum of the kept weights passes
 * uniform[r] times their whole sum (the last one kept if none does), prob its
 * weight's share of that sum.
 * A temperature below 2^-60 (0, negative, NaN) takes the largest logit, prob 1.
 * A logit of -inf or NaN is never chosen; a row of nothing else gives token -1
 * and prob 0. With logits of +inf only they have weight, 1 each. A top_p or
 * min_p that is NaN keeps all, a uniform outside [0, 1) or NaN counts as the
 * nearer end (NaN: 0).
 * Weights are computed to 2^-35 of themselves and rounded to whole units of 2^-44
 * of the largest or a little more (a token below half of that is not chosen),
 * their sums are 64-bit integers: results depend on no order of summing, and
 * agree with 64-bit arithmetic unless a border lies within 2^-35 of a sum and
 * 2^-45 of the largest weight for each token in it: where all tokens are as good
 * as alike they err alike, 2^19 of them by 2^-26 of the largest.
 * temperature, top_k, top_p, min_p and uniform are [n]; all but uniform may be
 * NULL (1, all, all, all). token int32 [n]; prob f32 [n] or NULL. 1 <= vocab <=
 * 524288, 0 <= n <= 2^24. */
int qsample(int type, const void *logits, int64_t stride, int64_t n, int64_t vocab, const float *temperature,
            const int32_t *top_k, const float *top_p, const float *min_p, const float *uniform, int32_t *token,
            float *prob, qg_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GB300_QSTEP_H */
