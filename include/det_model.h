/*
 * det_model.h -- operators of language models whose sums are taken in a fixed
 * order: log probabilities of given tokens (with entropy, top alternatives and
 * the gradient), the learned relative position bias (with its gradient), and
 * the attention of one new token over a paged key-value cache.
 *
 * The conventions of det.h hold (device pointers, caller-owned buffers and
 * workspace, a cudaStream_t as void*, return codes, nothing allocated and
 * nothing synchronized), with these differences:
 * - dtype is DET_F32, DET_BF16 or DET_F16 (the attention: DET_BF16 or
 *   DET_F16).  Sums, softmax statistics and accumulators are held in 32 bits
 *   whatever the dtype; a result in 16 bits is rounded once, at the end.
 * - Results of exponentials and logarithms are not those of a CPU statement
 *   bit for bit.  What is promised is that the bits of a row (a row of
 *   logits, a bucket of one head, a head of one sequence) are a function of
 *   that row's contents and sizes alone: not of the run, the number of other
 *   rows in the call, its place among them, its alignment, or the number of
 *   SMs.
 * - There is no block_threads argument: the launch shape is not the
 *   caller's.
 * - There is no device status word: what a kernel finds out of range it
 *   skips, by the rule stated at the call.
 */
#ifndef DET_MODEL_H
#define DET_MODEL_H

#include "det.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DET_BF16 2
#define DET_F16 3

/* Most alternatives det_token_logprobs reports. */
#define DET_MAX_TOP_K 32

/* ------------------------------------------------------------------------
 * det_token_logprobs -- for every row x[0..vocab) of the logits
 *   lse     = log sum_v exp(x[v])
 *   logprob = x[tokens[r]] - lse
 *   entropy = -sum_v p[v] log p[v],  p[v] = exp(x[v] - lse)
 *   top     = the top_k largest x[v] in falling order, the lowest index first
 *             among equals (NaN sorts as the largest), as x[v] - lse and v.
 * A token outside [0, vocab) is skipped: its logprob is +0.0.  A logit of
 * -inf is a masked one (probability 0).  A row with no logit above -inf has
 * lse = logprob = -inf and entropy 0.  A row that holds NaN or +inf has NaN
 * results (top_index_out still names the largest).  So does, as the only sign of
 * it, a row whose logits could not be copied into shared memory in time (2 s; the
 * kernel ends all the same); alternatives that were not found have index -1.
 *   logits       device, rows x vocab of dtype; row r starts at element
 *                r * row_stride, any alignment
 *   tokens       device, rows int32, or NULL when logprob_out is
 *   *_out        device, rows floats each; each may be NULL
 *   top_logprob_out, top_index_out  device, rows x top_k (float, int32); each
 *                may be NULL; not used when top_k is 0
 * Limits: rows < 2^31, vocab <= 2^30, top_k <= DET_MAX_TOP_K and <= vocab.
 */
int det_token_logprobs(const void* logits, int64_t rows, int64_t vocab, int64_t row_stride, const int32_t* tokens,
                       int dtype, float* logprob_out, float* entropy_out, float* lse_out, int top_k,
                       float* top_logprob_out, int32_t* top_index_out, void* stream);

/* ------------------------------------------------------------------------
 * det_token_logprobs_backward -- the gradient of sum_r grad_logprob[r] *
 * logprob[r] + grad_entropy[r] * entropy[r] for the logits:
 *   grad[v] = [v == token] g_l - p[v] (g_l + g_h (log p[v] + entropy)),
 * with log p[v] = x[v] - lse.  A skipped token has g_l = 0; masked logits and
 * rows without a logit above -inf get 0.
 *   lse, entropy   device, rows floats each: det_token_logprobs' results
 *                  (entropy may be NULL when grad_entropy is).  Where |lse| is
 *                  finite and 1024 or more, log p is taken from the row again
 *                  (up to ten times the time of such a row): 32 bits do not hold
 *                  lse well enough there
 *   grad_logprob, grad_entropy  device, rows floats each; either may be NULL (0)
 *   tokens         may be NULL when grad_logprob is
 *   grad_logits    device, rows x vocab of dtype (written), row r at element
 *                  r * grad_row_stride; must not overlap the inputs
 * Limits: vocab < 2^28, rows x (vocab rounded up to 8,192) below 2^42 (4,096
 * and 2^41 for DET_F32).
 */
int det_token_logprobs_backward(const void* logits, int64_t rows, int64_t vocab, int64_t row_stride,
                                const int32_t* tokens, int dtype, const float* lse, const float* entropy,
                                const float* grad_logprob, const float* grad_entropy, void* grad_logits,
                                int64_t grad_row_stride, void* stream);

/* ------------------------------------------------------------------------
 * det_relative_bias -- out[h][i][j] = table[bucket(j - i - q_offset)][h], the
 * learned bias of key j for query i, whose position is q_offset + i.
 * bounds[0..num_bounds) are distances in rising order and
 *   bucket(r) = the number of bounds <= max(-r, 0)           (one direction:
 *               keys after the query count as distance 0)
 *   bucket(r) = the number of bounds <= |r|, plus num_bounds + 1 when r > 0
 *               (bidirectional)
 * so the table has num_bounds + 1 rows, or 2 (num_bounds + 1).
 *   table   device, buckets x heads of table_dtype, contiguous
 *   bounds  device, num_bounds int32 (NULL when num_bounds is 0)
 *   out     device, heads x q_len x k_len of dtype, contiguous (written); a
 *           table entry is converted to dtype once, to nearest
 * Limits: |q_offset| + q_len + k_len <= 2^30, q_len < 2^20, num_bounds <=
 * DET_MAX_BOUNDS, heads <= 65,535.
 */
#define DET_MAX_BOUNDS 2047
int det_relative_bias(const void* table, int table_dtype, int64_t heads, const int32_t* bounds, int64_t num_bounds,
                      int bidirectional, int64_t q_len, int64_t k_len, int64_t q_offset, void* out, int dtype,
                      void* stream);

/* ------------------------------------------------------------------------
 * det_relative_bias_backward -- grad_table[k][h] = sum of grad[b][h][i][j]
 * over every b, i, j whose bucket is k: the scatter-add of the output's
 * gradient on the table, without bins in memory and without a sort.  A bucket
 * that no pair falls into gets +0.0.
 *   grad        device, batch x heads x q_len x k_len of dtype, any strides
 *               (in elements) but 1 along j; any alignment
 *   grad_table  device, buckets x heads of table_dtype, contiguous (written)
 * Limits: |q_offset| + q_len + k_len <= 2^30, num_bounds <= DET_MAX_BOUNDS,
 * heads <= 65,535, batch x (q_len / 64 + 1) x (k_len / 248 + 2) below 2^31;
 * strides are not negative.  The workspace is heads x buckets x (the tiles of that
 * product) floats: 4.7 MB for 8 x 16 x 2,048 x 2,048 and 32 buckets, 604 MB with
 * 4,096 of them.
 */
size_t det_relative_bias_backward_workspace_bytes(int64_t batch, int64_t heads, int64_t q_len, int64_t k_len,
                                                  int64_t num_bounds, int bidirectional);
int det_relative_bias_backward(const void* grad, int dtype, int64_t batch, int64_t heads, int64_t q_len,
                               int64_t k_len, int64_t stride_b, int64_t stride_h, int64_t stride_q,
                               const int32_t* bounds, int64_t num_bounds, int bidirectional, int64_t q_offset,
                               void* grad_table, int table_dtype, void* workspace, size_t workspace_bytes,
                               void* stream);

/* ------------------------------------------------------------------------
 * det_paged_attention -- for each sequence b and query head h, with the
 * length n = lengths[b] and the key-value head g = h / (heads / kv_heads)
 *   x[j] = scale * q[b][h] . k[j][g] + bias[j],  j = 0..n-1
 *   out[b][h] = sum_j softmax(x)[j] v[j][g],   lse[b][h] = log sum_j exp(x[j])
 * where token j lies in slot j % page_size of page block_table[b][j /
 * page_size].  The query is the sequence's last token (position n - 1), so
 * bias[j] = bias_table[number of bounds <= n - 1 - j][h] (see
 * det_relative_bias), or 0 without a table.
 * Scores are 32-bit values in units of the natural logarithm: a finite bias,
 * the types' lowest values included, is a finite score (what q . k adds to it is
 * lost in the rounding), and -inf masks the token.
 * A length below 0 counts as 0, one above min(max_len, max_pages * page_size)
 * counts as that.  Tokens whose page is outside [0, num_pages) are skipped.
 * Slots past a sequence's length are not read.  Without a token, out is 0 and
 * lse -inf.
 *   q         device, batch x heads x head_dim of dtype; strides in elements,
 *             1 along head_dim
 *   k_cache, v_cache  device, of dtype, element (page, slot, g, d) at page *
 *             stride_page + slot * stride_token + g * stride_head + d;
 *             16-byte aligned, with strides that are multiples of 8
 *   block_table  device, batch x max_pages int32, rows table_stride apart
 *   lengths   device, batch int32
 *   bias_table  device, (num_bounds + 1) x heads of bias_dtype, or NULL; for a
 *             bidirectional bias its first num_bounds + 1 rows
 *   out       device, batch x heads x head_dim of dtype, contiguous (written)
 *   lse_out   device, batch x heads floats (written), or NULL
 *   max_len   a bound on the lengths known to the host
 * head_dim is 64, 128 or 256; heads is a multiple of kv_heads; batch and
 * kv_heads are at most 65,535, max_len below 2^31.
 */
size_t det_paged_attention_workspace_bytes(int64_t batch, int64_t heads, int64_t head_dim, int64_t max_len);
int det_paged_attention(const void* q, int64_t q_stride_b, int64_t q_stride_h, const void* k_cache,
                        int64_t k_stride_page, int64_t k_stride_token, int64_t k_stride_head, const void* v_cache,
                        int64_t v_stride_page, int64_t v_stride_token, int64_t v_stride_head, int64_t num_pages,
                        int64_t page_size, const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                        const int32_t* lengths, int64_t batch, int64_t heads, int64_t kv_heads, int64_t head_dim,
                        int dtype, float scale, const void* bias_table, int bias_dtype, const int32_t* bias_bounds,
                        int64_t num_bounds, int64_t max_len, void* out, float* lse_out, void* workspace,
                        size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif
