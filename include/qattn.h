/*
 * qattn.h - C ABI of the attention that stands between the block-quantized
 * products of qgemv.h: a paged cache that holds keys and values in 4 bits,
 * appending to it with the position rotation applied on the way, attention of
 * new tokens over it, and causal attention over whole packed prompts.
 *
 * The reference pages stop at the products; the operators here are defined by
 * the formulas at each call. The 4-bit rule is Q4_0's of quantize_rows.
 *
 * Conventions (those of qgemv.h, and)
 *   - Status codes, the stream argument, qg_last_cuda_error and
 *     qg_device_error are qgemv.h's. Argument errors are returned before
 *     anything is enqueued; no call synchronizes or allocates.
 *   - Pointers are device pointers unless said otherwise, 16-byte aligned
 *     (QG_ERR_ALIGN); index arrays (int32) need 4 bytes.
 *   - Indexes that lie on the device cannot be checked on the host. A kernel
 *     that meets a page, slot, position, length or offset outside its range
 *     records code 4 in the device error word, leaves the access out (what
 *     that means is said at each call) and goes on.
 *   - Sums, softmax statistics and accumulators are f32, scores too: rows
 *     with one of more than 2^23 in size, whose f32 steps come near 1, may be
 *     NaN.
 *   - Outputs overlap no input and no workspace, unless a call says so.
 *   - A kernel may start while the one enqueued before it finishes
 *     (programmatic dependent launch) but touches memory only after it.
 */
#ifndef GB300_QATTN_H
#define GB300_QATTN_H

#include "qgemv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- The cache ------------------------------------------------------------ */

/* A paged cache of keys and values held in 4 bits (host struct).
 *
 * data: qkv_cache_bytes() bytes, [n_pages][n_kv_heads][page_size / 16 groups].
 * A group holds 16 tokens of one key/value head, D = head_dim, in 18 D bytes:
 *   at 0      16 rows of D/2 bytes, the key codes
 *   at 8 D    16 rows of D/2 bytes, the value codes
 *   at 16 D   16 rows of D/32 f16, the key scales
 *   at 17 D   16 rows of D/32 f16, the value scales
 * Token `slot` lies in page slot / page_size, group (slot % page_size) / 16,
 * as the group's token i = slot % 16. Codes and scales are Q4_0's: per 32
 * elements one f16 d and 16 bytes, byte j holding element j in its low and
 * j + 16 in its high nibble, value (code - 8) d. Only the order of the code
 * bytes is the cache's own (it is the order in which the attention kernel's
 * tensor-core fragments take them), NB = D/32:
 *   keys: row i; byte j of block b at ((j / 4) NB + b) 4 + j % 4;
 *   values: row r(i) = (i & 8) | ((i & 1) << 2) | ((i >> 1) & 3); byte j of
 *     block b at (u NB + b) 2 + j % 2, u = j / 2 ^ (r(i) & 2 ? 4 : 0).
 * Scales: row i, block b at 2 (i NB + b).
 * head_dim is 64 or 128, page_size a multiple of 16. */
typedef struct {
    void *data;
    int64_t n_pages;
    int32_t n_kv_heads, head_dim, page_size;
} qkv_cache;

/* Bytes of a cache, n_pages * n_kv_heads * page_size * 9/8 head_dim; -1 on a
 * geometry outside the limits above (or n_pages * page_size > 2^31 - 1). */
int64_t qkv_cache_bytes(int64_t n_pages, int n_kv_heads, int head_dim, int page_size);

/* Arguments of qkv_append (host struct). */
typedef struct {
    const void *q;        /* in_type [n_tok][n_heads][D], or NULL             */
    const void *k, *v;    /* in_type [n_tok][n_kv_heads][D]                   */
    int64_t q_stride, k_stride, v_stride; /* elements from token to token, a
                             multiple of 16 bytes, so that q, k and v can lie
                             in one fused product                              */
    const int32_t *slots; /* [n_tok] where each token goes; < 0: not cached   */
    const int32_t *positions; /* [n_tok], row of `rope`; NULL without rope    */
    const float *rope;    /* f32 [n_pos][rot_dim / 2][2], cos and sin of each
                             position and pair; NULL: no rotation              */
    void *q_out;          /* out_type [n_tok][n_heads][D]; required with q    */
    void *k_out, *v_out;  /* out_type [n_tok][n_kv_heads][D], or NULL         */
    int64_t n_tok;
    int32_t n_heads;      /* query heads (ignored without q)                  */
    int32_t in_type, out_type; /* QG_F32 or QG_F16                            */
    int32_t n_pos, rot_dim;    /* rot_dim a multiple of 8, <= D               */
    int32_t rope_pairs;   /* 0: channels i and i + rot_dim/2 make pair i;
                             1: channels 2i and 2i + 1                        */
} qkv_append_args;

/* Rotates q and k (channels 0 .. rot_dim - 1 of every head; the others pass),
 * writes k and v to the cache in 4 bits, and the rotated q (and where asked
 * the rotated k, and v) to q_out, k_out, v_out, in one launch:
 *   y_a = x_a cos - x_b sin, y_b = x_a sin + x_b cos
 * with both products and their sum each rounded in f32, so that the codes,
 * which are results of a rounding, are reproducible; then the Q4_0 rule of
 * quantize_rows on the f32 rows. k_out and v_out are not quantized. Outputs
 * may be their inputs (same type, contiguous). Two tokens of one call with the
 * same slot leave that slot undefined. A slot past the cache is not written; a
 * position outside [0, n_pos) leaves all of its token's rows unwritten. */
int qkv_append(const qkv_cache *cache, const qkv_append_args *args, qg_stream_t stream);

/* The values of the rows `slots` of the cache, (code - 8) d, exact in f32:
 * k_out and v_out f32 [n][n_kv_heads][D], either may be NULL; at most 2^30
 * rows. A slot < 0 or past the cache gives zeros (past it, code 4 as well). */
int qkv_read(const qkv_cache *cache, const int32_t *slots, int64_t n, float *k_out, float *v_out, qg_stream_t stream);

/* ---- Attention over the cache ---------------------------------------------- */

/* Workspace bytes of qkv_attend: the partial results of sequences that are
 * split over several thread blocks. 0 on a bad argument. Depends on none of
 * the sequences' lengths. */
size_t qkv_attend_workspace_bytes(int head_dim, int n_kv_heads, int n_heads, int max_q_len);

/* Attention of the newest tokens of n_seq sequences over the cache.
 * Sequence s has lengths[s] tokens in the cache, token t in page
 * table[s * table_stride + t / page_size], row t % page_size (entries past
 * the last used page are not read; table_stride at most 2^31 - 1). Its queries are rows q_offsets[s] ..
 * q_offsets[s + 1] - 1 of q (q_offsets NULL: row s alone), for its last
 * tokens: query i of m sees cache tokens t < lengths[s] - m + i + 1. With
 * group g = n_heads / n_kv_heads, query head h reads key/value head h / g:
 *   s_t = scale q . k_t, out = sum_t exp(s_t - max s) v_t / sum_t exp(s_t - max s)
 * and zeros where no token is seen. What the cache holds at tokens that are
 * not seen has no influence, NaN and infinities included.
 *
 * type (QG_F32 or QG_F16) is q's and out's. Codes enter the products exactly;
 * with QG_F16 the softmax weights are rounded to f16 (relative 2^-11), with
 * QG_F32 q and the weights are split in two f16 parts each (about 2^-21). A
 * weight enters as its product with its token's value scale, whose f16 parts
 * end at 2^-31 of the row's largest such product: 32 channels whose values
 * are far smaller than the head's others are only as fine as that.
 * q: [n_tok][n_heads][D], q_stride elements from token to token (a multiple
 * of 16 bytes); out: [n_tok][n_heads][D] contiguous. max_q_len >= every
 * sequence's number of queries; a sequence with more, or with q_offsets
 * outside 0 .. n_tok or falling, is left out (code 4). Rows in no sequence,
 * or in one that is left out, are not written; a row in two (q_offsets that
 * fall and rise again) is undefined. A length outside
 * 0 .. table_stride * page_size is taken as the nearer end, a page outside the
 * cache as tokens that are not seen (both code 4). A value block whose scale
 * is not finite gives NaN in its 32 channels to the rows that see its token.
 * The result does not depend
 * on what other sequences a call has beyond rounding: a long sequence is split
 * where the thread blocks' shares end. Same inputs, same bits. */
int qkv_attend(const qkv_cache *cache, int type, const void *q, int64_t q_stride, void *out, const int32_t *table,
               int64_t table_stride, const int32_t *lengths, const int32_t *q_offsets, int64_t n_seq, int64_t n_tok,
               int n_heads, int max_q_len, float scale, void *workspace, size_t workspace_bytes, qg_stream_t stream);

/* ---- Attention of a batch that shares a prefix ------------------------------- */

/* Workspace bytes of qkv_attend_shared, for calls of up to n_tok query rows.
 * 0 on a bad argument. Depends on no length. */
size_t qkv_attend_shared_workspace_bytes(int head_dim, int n_kv_heads, int n_heads, int64_t n_tok, int max_q_len);

/* Attention of the newest tokens of n_seq sequences that begin with the same
 * tokens: the prefix's prefix_len[0] ones (device), token t in page
 * prefix_table[t / page_size] of prefix_pages entries, row t % page_size, and
 * then each sequence's own, given as qkv_attend's (lengths, table and the rule
 * of what a query sees count the own tokens alone). Every query sees the whole
 * prefix:
 *   s_t = scale q . k_t, out = sum_t exp(s_t - max s) v_t / sum_t exp(s_t - max s)
 * over the prefix's tokens and the own ones that it sees; the result is that of
 * qkv_attend on sequences that hold both, but the prefix is read and its products
 * are formed once for all of them. Where neither holds a token seen, zeros. A call
 * has one prefix. With 8 key/value heads it is faster than qkv_attend on whole tables
 * from about 8 sequences and 10^5 sequences times prefix tokens on.
 *
 * Everything said at qkv_attend holds here, with these differences. Keys and
 * values of the prefix enter the products as two f16 parts, which hold them
 * exactly beside the largest ones of their 128 tokens down to 2^-33 of those. Of
 * the prefix's weights those parts (with QG_F16 the one, whose rounding the sum
 * below the line does not have) end at 2^-38 of the row's largest: each may be off
 * by half of that, and what n tokens with weights below it have together, up to
 * n 2^-39, is missing from the values. A prefix length
 * outside 0 .. prefix_pages * page_size is taken as the nearer end, a page
 * outside the cache as tokens that are not seen (both code 4). A key block of
 * the prefix whose scale is not finite makes every row NaN. n_tok * n_heads is
 * at most 2^26. */
int qkv_attend_shared(const qkv_cache *cache, int type, const void *q, int64_t q_stride, void *out,
                      const int32_t *prefix_table, int64_t prefix_pages, const int32_t *prefix_len, const int32_t *table,
                      int64_t table_stride, const int32_t *lengths, const int32_t *q_offsets, int64_t n_seq,
                      int64_t n_tok, int n_heads, int max_q_len, float scale, void *workspace, size_t workspace_bytes,
                      qg_stream_t stream);

/* ---- Attention over whole prompts ------------------------------------------- */

/* Causal attention over n_seq packed sequences: sequence s is rows offsets[s]
 * .. offsets[s + 1] - 1 (int32 [n_seq + 1], device); row i of it sees its rows
 * j <= i:
 *   s_j = scale q_i . k_j, out_i = sum_j exp(s_j - max s) v_j / sum_j exp(s_j - max s)
 * Rows in no sequence are not written. q f16 [n_tok][n_heads][D], k and v f16
 * [n_tok][n_kv_heads][D], query head h with key/value head h / (n_heads /
 * n_kv_heads), D = 64 or 128; strides in elements from token to token, a
 * multiple of 8. out: out_type (QG_F16 or QG_F32) [n_tok][n_heads][D]
 * contiguous. The softmax weights are rounded to f16 for the tensor cores
 * (relative 2^-11), whatever out_type. Rows that are not seen have no
 * influence, NaN and infinities included. Offsets outside 0 .. n_tok or
 * falling: that sequence is left out (code 4), and so is one that begins
 * before the end of an earlier one that is not. Same inputs, same bits, and a
 * sequence's result does not depend on what others the call has. */
int qattn_prompt(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                 int out_type, void *out, const int32_t *offsets, int64_t n_seq, int64_t n_tok, int n_heads,
                 int n_kv_heads, int head_dim, float scale, qg_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GB300_QATTN_H */
