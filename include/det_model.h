/*
 * det_model.h -- operators of language models whose sums are taken in a fixed
 * order: log probabilities of given tokens (with entropy, top alternatives and
 * the gradient), the learned relative position bias (with its gradient), the
 * attention of one new token over a paged key-value cache, and the token
 * embedding, the layer norm and the gated linear recurrence, each with its
 * gradient.
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
 * - "Not read" is said of values.  A row that starts inside an aligned 16-byte
 *   vector may be fetched by the vectors, or 4-byte words, that hold it; what else
 *   they hold, before the row and after it, is discarded.
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

/* ------------------------------------------------------------------------
 * det_embedding -- out[i][0..dim) = scale * table[tokens[i]][0..dim), the
 * product in 32 bits, rounded once to dtype.  A token outside [0, vocab) gives a
 * row of +0.0.
 *   table   device, vocab x dim of table_dtype; row v starts at element
 *           v * table_stride
 *   tokens  device, n int32
 *   out     device, n x dim of dtype, contiguous (written)
 * Limits: n < 2^31, vocab < 2^31, dim <= 2^21.
 */
int det_embedding(const void* table, int table_dtype, int64_t vocab, int64_t dim, int64_t table_stride,
                  const int32_t* tokens, int64_t n, float scale, void* out, int dtype, void* stream);

/* ------------------------------------------------------------------------
 * det_embedding_backward -- the gradient of det_embedding's table:
 *   grad_table[v] = old + scale * PT(grad[i] : tokens[i] = v, i rising), per column,
 * the canonical pairwise tree of det_scatter_add_rows in 32 bits, times scale,
 * plus +0.0 or, with accumulate, what the row holds (in 32 bits), rounded once to
 * table_dtype: with DET_F32 and a scale of 1 the bits of det_scatter_add_rows, with
 * accumulate on the same table, without on one of zeros.  Rows of no token are +0.0;
 * with accumulate they are neither read nor written.
 *   grad        device, n x dim of dtype; row i starts at element i * grad_stride.
 *               Rows of tokens outside [0, vocab) are not read
 *   grad_table  device, vocab x dim of table_dtype, contiguous (written); must
 *               not overlap the inputs
 * Limits: n < 2^31, vocab < 2^31, dim <= 2^21.  The workspace is that of a sort of n
 * records and up to n / 16 rows of dim floats.
 */
size_t det_embedding_backward_workspace_bytes(int64_t n, int64_t vocab, int64_t dim);
int det_embedding_backward(const void* grad, int dtype, int64_t n, int64_t dim, int64_t grad_stride,
                           const int32_t* tokens, float scale, void* grad_table, int table_dtype, int64_t vocab,
                           int accumulate, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * det_layer_norm -- for every row x[0..cols)
 *   mean = sum x / cols,  rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps)
 *   out[c] = (x[c] - mean) * rstd * weight[c] + bias[c]
 *   x       device, rows x cols of dtype; row r starts at element r * x_stride
 *   weight, bias  device, cols of param_dtype; either may be NULL (1, 0)
 *   out     device, rows x cols of dtype, contiguous (written); may be x where
 *           x_stride is cols
 *   mean_out, rstd_out  device, rows floats each; either may be NULL
 * A row that holds NaN or an infinity has NaN in out.  So has one whose sum, or whose
 * sum of squares of x - mean (plus eps), passes the range of 32 bits.
 * Limits: rows < 2^31, 1 <= cols <= DET_MAX_NORM_COLS (rows of no columns are
 * refused unless there is no row), eps finite and not negative.
 */
#define DET_MAX_NORM_COLS 16384
int det_layer_norm(const void* x, int dtype, int64_t rows, int64_t cols, int64_t x_stride, const void* weight,
                   const void* bias, int param_dtype, float eps, void* out, float* mean_out, float* rstd_out,
                   void* stream);

/* ------------------------------------------------------------------------
 * det_layer_norm_backward -- with xh = (x - mean) * rstd and gw = grad * weight
 *   grad_x = rstd * (gw - sum(gw) / cols - xh * sum(gw * xh) / cols)
 *   grad_weight[c] = sum_r grad[r][c] * xh[r][c],  grad_bias[c] = sum_r grad[r][c]
 * The sums over rows are taken in an order that rows and cols alone decide.
 *   grad, x     device, rows x cols of dtype, rows at their strides
 *   mean, rstd  device, rows floats: det_layer_norm's
 *   weight      device, cols of param_dtype, or NULL (1)
 *   grad_x      device, rows x cols of dtype, contiguous (written), or NULL; may be grad where grad_stride is cols
 *   grad_weight, grad_bias  device, cols of param_dtype (written); either may be
 *               NULL.  Without rows they are +0.0
 * Limits: as det_layer_norm's.
 */
size_t det_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols);
int det_layer_norm_backward(const void* grad, int64_t grad_stride, const void* x, int64_t x_stride, int dtype,
                            int64_t rows, int64_t cols, const float* mean, const float* rstd, const void* weight,
                            int param_dtype, void* grad_x, void* grad_weight, void* grad_bias, void* workspace,
                            size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * det_linear_recurrence -- for every sequence b and channel c, with h = the
 * initial state,
 *   h = a[t] * h + u[t],  out[t] = h,   t = 0..length-1
 *   DET_GATE_DECAY:    a = gate[t], u = x[t]
 *   DET_GATE_SIGMOID:  a = 1 / (1 + exp(-gate[t])), u = (1 - a) * x[t]
 * in 32 bits; out is rounded once.  The bits of out[t] are a function of the initial
 * state and of the steps up to t alone: a sequence gives the same bits whatever
 * follows.  (One that is cut and resumed from its final state gives other roundings.)
 * a and 1 - a of the sigmoid form are off by at most 8 units of 2^-24 of their size
 * for DET_F32.  For 16-bit gates, whose own steps move them by far more, the
 * exponential and the reciprocal are the hardware's: 8 + 1.22 |gate| units, and a is
 * less by 2^-125 (0 from a gate of -87 down), in final_out and states_out too.
 *   x, gate   device, batch x time x channels of dtype; strides in elements, 1
 *             along channels
 *   initial   device, batch x channels floats, contiguous, or NULL (0)
 *   lengths   device, batch int32, or NULL (time).  One below 0 counts as 0, one above
 *             time as time.  Steps from a sequence's length on are not read, and
 *             their outputs are +0.0
 *   out       device, batch x time x channels of dtype, contiguous (written); must
 *             not overlap the inputs
 *   final_out device, batch x channels floats: the states at the sequences' ends,
 *             or NULL; may be initial
 *   states_out  device, batch x ceil(time / DET_RECURRENCE_KEEP) x channels floats:
 *             the state before every DET_RECURRENCE_KEEP-th step, for the gradient
 *             (past a sequence's end: its final state), or NULL
 * Products of up to DET_RECURRENCE_SPAN decays are formed, here and in the gradient: where
 * one passes the range of 32 bits (decays well above 1), results may become infinite or NaN
 * before they would step by step, and where one falls below it and decays well above 1
 * follow, what came before is lost early.  A state that is infinite or NaN leaves later
 * states infinite or NaN.
 * So does, as the only sign of it, a part of a sequence that was not told the states of the parts
 * before it in time (2 s; the kernel ends all the same), here and in the gradient.
 * Limits: batch <= 65,535, time < 2^31 - 2^16, channels < 2^31 - 2^16; strides are not negative.
 */
#define DET_GATE_DECAY 0
#define DET_GATE_SIGMOID 1
#define DET_RECURRENCE_KEEP 128
#define DET_RECURRENCE_SPAN 128
int det_linear_recurrence(const void* x, int64_t x_stride_b, int64_t x_stride_t, const void* gate,
                          int64_t gate_stride_b, int64_t gate_stride_t, int dtype, int form, int64_t batch,
                          int64_t time, int64_t channels, const float* initial, const int32_t* lengths, void* out,
                          float* final_out, float* states_out, void* stream);

/* ------------------------------------------------------------------------
 * det_linear_recurrence_backward -- the gradient of sum grad * out +
 * grad_final * final.  With l = grad_final at a sequence's end and from its last step
 * back l = grad[t] + a[t + 1] * l (a = 1 after the end):
 *   DET_GATE_DECAY:    grad_gate[t] = l * h[t - 1],  grad_x[t] = l
 *   DET_GATE_SIGMOID:  grad_gate[t] = l * (h[t - 1] - x[t]) * a * (1 - a),
 *                      grad_x[t] = l * (1 - a)
 * and grad_initial = a[0] * l of the first step.
 *   grad      device, batch x time x channels of dtype, strided as x is, or NULL (0)
 *   states    device: det_linear_recurrence's states_out
 *   grad_final  device, batch x channels floats, or NULL (0)
 *   grad_x, grad_gate  device, batch x time x channels of dtype, contiguous (written; +0.0
 *             from a sequence's length on); must not overlap the inputs
 *   grad_initial  device, batch x channels floats (written), or NULL
 */
int det_linear_recurrence_backward(const void* grad, int64_t grad_stride_b, int64_t grad_stride_t, const void* x,
                                   int64_t x_stride_b, int64_t x_stride_t, const void* gate, int64_t gate_stride_b,
                                   int64_t gate_stride_t, int dtype, int form, int64_t batch, int64_t time,
                                   int64_t channels, const float* states, const float* grad_final,
                                   const int32_t* lengths, void* grad_x, void* grad_gate, float* grad_initial,
                                   void* stream);

#ifdef __cplusplus
}
#endif
#endif
