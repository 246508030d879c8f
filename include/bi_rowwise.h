/*
 * bi_rowwise.h -- batch-invariant row-wise reductions beyond RMSNorm, in libbi: the
 * log-softmax of a logits row, the mean of a row, the log-probabilities of given tokens
 * with entropy, top alternatives and gradient, and the verification of drafted tokens.
 *
 * Source: book chapter "Batch-invariant kernels: why temperature-0 decoding is still
 * nondeterministic", Sources (the companion library overrides RMSNorm, matmul, mean and
 * log-softmax; log-probabilities are what the chapter's on-policy RL case compares between
 * sampler and trainer, The trap) and Case 6 / The boring rule item 1 (one strategy at
 * every batch size; data-parallel rows).  The pages give no formula beyond the names;
 * these follow the textbook definitions.
 *
 * Construction (bi_log_softmax and bi_mean): one CTA of 1024 threads per row.  Thread t owns the
 * 4-element groups t, t + 1024, t + 2048, ... of its row and folds them in ascending
 * order (elements within a group in ascending order), whether it reads a group as one
 * 128-bit load (16-byte aligned rows) or as scalars; the 1024 per-thread values are then
 * combined by a fixed butterfly within each warp and a fixed butterfly over the 32 warp
 * results.  The tree therefore depends on n only: a row's bits do not depend on the
 * number of rows, the row's position, its alignment or the stride.
 *
 * Conventions are those of bi.h: caller-owned device pointers, asynchronous launches on
 * `stream`, argument errors returned before any launch.  fp32 arithmetic.
 */
#ifndef BI_ROWWISE_H_
#define BI_ROWWISE_H_

#include "bi.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Log-softmax of each row:
 *   m_r = max_i x[r, i]   (exact),   s_r = sum_i exp(x[r, i] - m_r)   (fp32, tree above),
 *   y[r, i] = (x[r, i] - m_r) - log(s_r).
 *   x  fp32 [rows, n], row stride ldx >= n;  y  fp32 [rows, n], row stride ldy >= n;
 *   y may be x itself (ldy == ldx).  1 <= n < 2^31.  Pointers 4-byte aligned.
 *   A -inf entry gives y = -inf; a row containing NaN, or +inf, or only -inf gives NaN
 *   everywhere in the row (as the definition does). */
bi_status bi_log_softmax(const float* x, int64_t ldx, float* y, int64_t ldy, int64_t rows,
                         int64_t n, bi_stream_t stream);

/* Mean of each row: out[r] = (sum_i x[r, i]) / n, the sum in fp32 by the tree above, the
 * division correctly rounded.
 *   x      [rows, n], dtype x_dtype (BI_BF16 or BI_F32), row stride ldx >= n, aligned to
 *          its element size.  1 <= n < 2^31.
 *   out    fp32 [rows]. */
bi_status bi_mean(const void* x, int64_t ldx, int x_dtype, int64_t rows, int64_t n, float* out,
                  bi_stream_t stream);

/* Log-probabilities of given tokens, without writing the [rows, n] log-softmax: what a
 * sampler reports for the tokens it chose and a trainer recomputes for the same tokens.
 *   x        [rows, n] logits, dtype x_dtype (BI_BF16, BI_F16 or BI_F32), row stride
 *            ldx >= n, aligned to its element size (rows that are 16-byte aligned are read
 *            128 bits at a time; the arithmetic is the same either way).
 *            1 <= n <= BI_LOGPROBS_MAX_N.
 *   tokens   int32 [rows]: the scored token of each row.  -1 scores nothing (padding): its
 *            logp is 0.  Any other id outside [0, n) gives NaN and sets BI_ERR_DEVICE_ARG
 *            in the device error word.
 *   With m the row's largest entry, s = sum_i exp(x_i - m) and p_i = exp(x_i - m) / s:
 *   logp     fp32 [rows]: (x[token] - m) - log s.
 *   entropy  fp32 [rows] or NULL: -sum_i p_i log p_i = log s - (sum_i exp(x_i - m)
 *            (x_i - m)) / s  (a -inf entry adds 0).
 *   lse      fp32 [rows] or NULL: m + log s (bi_token_logprobs_backward takes it).
 *   top      0 .. min(n, BI_LOGPROBS_MAX_TOP): top_logp, top_ids [rows, top] get the row's
 *            largest entries in descending order as log-probabilities and indices; the
 *            lowest index first among equal entries, NaN below every number.
 *   fp32 sums over a tree that depends on n and x_dtype alone: a row's outputs do not depend on
 *   the number of rows, on the other rows, on top, or on alignment and stride.  No sum has more
 *   than 264 terms in a row, so s is within 2^-15 of itself at any n.  A row with a NaN
 *   or +inf, or of nothing but -inf, gives NaN (ids are still ranked). */
#define BI_LOGPROBS_MAX_TOP 32
#define BI_LOGPROBS_MAX_N (0x7fffffff - 0x3fff) /* 2^31 - 2^14 */
bi_status bi_token_logprobs(const void* x, int64_t ldx, int x_dtype, const int32_t* tokens,
                            int64_t rows, int64_t n, float* logp, float* entropy, float* lse,
                            int64_t top, float* top_logp, int32_t* top_ids, bi_stream_t stream);

/* Gradient of sum_r g_logp[r] * logp[r] + g_entropy[r] * entropy[r] with respect to x:
 *   dx[r, i] = g_logp[r] * ([i == tokens[r]] - p_i) - g_entropy[r] * p_i * (log p_i + entropy[r]),
 *   p_i = exp(x_i - lse[r]); an entry with p_i = 0 gets 0 (plus g_logp at the token).  The
 *   fp32 lse is off by up to 2^-24 of itself, which p_i takes over as a factor.
 *   lse, entropy  fp32 [rows], as bi_token_logprobs gave them.
 *   g_logp, g_entropy  fp32 [rows]; either may be NULL (a gradient of 0), not both; entropy
 *            may be NULL when g_entropy is.
 *   A token of -1 has no g_logp term; one outside [0, n) neither, and sets
 *   BI_ERR_DEVICE_ARG.
 *   A row without a g_logp term, or with one of 0, and with g_entropy NULL or 0 gets zeros,
 *   whatever its logits, lse and entropy are (padding may hold NaN).
 *   dx       [rows, n] of x's dtype (fp32 arithmetic, rounded once to nearest even), row
 *            stride lddx >= n; may be x itself (lddx == ldx). */
bi_status bi_token_logprobs_backward(const void* x, int64_t ldx, int x_dtype,
                                     const int32_t* tokens, int64_t rows, int64_t n,
                                     const float* lse, const float* entropy, const float* g_logp,
                                     const float* g_entropy, void* dx, int64_t lddx,
                                     bi_stream_t stream);

/* Verification of drafted tokens from given random numbers: what a speculative step does with
 * the logits of its verify block at a temperature.  One row of logits per token of the block, as
 * bi_verify_block lays blocks out: rows cu_q[b] .. cu_q[b+1]-1 are sequence b's, the first for its
 * last input and one for each drafted token behind it; the row in front of a drafted token decides
 * it.  With p = softmax(row / T) of that row and q the distribution that the draft was drawn from:
 *   - draft j is kept while u_j * q(token_j) < p(token_j);
 *   - in place of the first that is not, the first token i is emitted for which the sum of
 *     max(p_k - q_k, 0) over k <= i exceeds u of the whole sum (where p and q are equal
 *     throughout: of p);
 *   - behind a block that is kept in full, the first i for which the sum of p_k exceeds u.
 *   The emitted tokens are distributed as p, whatever the drafts were.
 *   T = 0 (or below 2^-64): a draft is kept while it is the row's largest entry, and the largest
 *   entry is emitted at the end, ranked as bi_argmax ranks; draft rows take no part.
 *
 *   logits       [total_q, n], dtype BI_BF16, BI_F16 or BI_F32, row stride ldl >= n, aligned to
 *                its element size.  1 <= n <= BI_DRAFTS_MAX_N.
 *   draft_logits [num_drafts, n] of the same dtype, row stride ldd >= n: q = softmax(row / T); or
 *                NULL: each draft was chosen without chance, q is 1 at the token and 0 elsewhere.
 *   draft_tokens int32 [num_drafts]: the drafts of all sequences one after the other, a sequence
 *                of w rows having w - 1.  (Draft j of sequence b is entry cu_q[b] - b + j.)  -1 is
 *                no draft: the block ends in front of it, with a token drawn from p.  Any other id
 *                outside [0, n) does the same and sets BI_ERR_DEVICE_ARG.
 *   uniforms     fp32 [total_q], in [0, 1): row cu_q[b] + j decides draft j, and the sequence's
 *                last row draws its last token.  (Values outside are taken as the nearest inside
 *                for a draw, NaN as 0; as they are in the comparison.)
 *   temperatures fp32 [batch], or NULL: `temperature` for all.  A sequence whose temperature is
 *                negative, infinite or NaN gets no tokens and sets BI_ERR_DEVICE_ARG.
 *   cu_q         int32 [batch + 1], cu_q[0] = 0, 1 to max_q rows each, cu_q[batch] <= total_q and
 *                cu_q[batch] - batch <= num_drafts; else the whole call emits nothing and sets
 *                BI_ERR_DEVICE_ARG.  Rows behind the last sequence take no part.
 *   tokens       int32 [batch, max_q]: the kept drafts, then the drawn token, then -1.
 *   accepted     int32 [batch]: how many drafts were kept.
 *   logprobs     fp32 [batch, max_q] or NULL: log p of each emitted token (of the softmax at
 *                temperature 1 where T is 0), 0 behind them.
 *   A row that the block comes to, target or draft, with a NaN, +inf or nothing but -inf has no
 *   distribution, at any temperature: the block ends there with a token of -1 and a
 *   log-probability of NaN.
 *   workspace    bi_verify_drafts_workspace_size(total_q, num_drafts, n) bytes (num_drafts 0 where
 *                draft_logits is NULL), 16-byte aligned, contents scratch.
 *   Weights are whole numbers of 2^-60, within 2^-29 of themselves, so the drawn token does not
 *   depend on the order of any sum.  A sequence's outputs depend on its own rows, drafts, uniforms
 *   and temperature alone: not on the batch, max_q, alignment or strides. */
#define BI_DRAFTS_MAX_N (1 << 20)
size_t bi_verify_drafts_workspace_size(int64_t total_q, int64_t num_drafts, int64_t n);
bi_status bi_verify_drafts(const void* logits, int64_t ldl, const void* draft_logits, int64_t ldd,
                           int dtype, const int32_t* draft_tokens, int64_t num_drafts,
                           const float* uniforms, const float* temperatures, float temperature,
                           const int32_t* cu_q, int64_t batch, int64_t total_q, int64_t max_q,
                           int64_t n, int32_t* tokens, int32_t* accepted, float* logprobs,
                           void* workspace, size_t workspace_bytes, bi_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BI_ROWWISE_H_ */
