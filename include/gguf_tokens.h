/*
 * gguf_tokens.h -- C ABI of libgguf_qk.so, the steps of a pass over several new
 * tokens per sequence (a prompt, a chunk of one, drafted tokens, or the one token
 * of a decode step): the norms of queries and keys per head with the rotation by
 * position, the attention of the new tokens over the paged cache of gguf_kv.h,
 * and the verification of drafted tokens against the target's probabilities.
 *
 * The conventions are those of gguf_qk.h and gguf_kv.h: device pointers into
 * memory the caller owns, work enqueued on `stream` of the current device,
 * arguments validated before any HIP call (a failed call enqueues nothing), the
 * same status codes, nothing allocated, no pointer kept, a workspace of the size
 * the _workspace call names (uninitialized, 16-byte aligned, one per call that may
 * overlap another in time). All work is deterministic. These are inference steps
 * and have no gradient.
 */
#ifndef GGUF_TOKENS_H
#define GGUF_TOKENS_H

#include "gguf_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* --- norms of queries and keys, rotation by position ------------------------- */

/* How the elements of a head pair up: 2 i with 2 i + 1, or i with i + n_rot / 2. */
#define GGUF_ROPE_ADJACENT 0
#define GGUF_ROPE_HALVES 1

/* The rotation: pair i (0 .. n_rot / 2 - 1) of a token's heads turns by the angle
 * pos[axes[i]][token] * freqs[i]. */
typedef struct gguf_rope {
  const double* freqs;   /* device, n_rot / 2: radians per position (base, scaling and
                            frequency factors of the model folded in) */
  const int32_t* axes;   /* device, n_rot / 2: the position axis of each pair (time,
                            height, width of image and video tokens, in sections or by
                            turns), a value outside 0 .. n_axes - 1 leaves the pair
                            unturned (angle 0); NULL: axis 0 for all */
  const int32_t* pos;    /* device, [n_axes] rows of n_tokens positions */
  int64_t pos_stride;    /* from axis to axis, >= n_tokens */
  int32_t n_axes;        /* 1 .. 16 */
  int32_t n_rot;         /* even, 0 .. head_dim; the elements behind it are not turned */
  int32_t pairing;       /* GGUF_ROPE_ADJACENT or GGUF_ROPE_HALVES */
  float magnitude;       /* factor of every cosine and sine (1, or a context
                            extension's), finite */
} gguf_rope;

/* Per token and head x (head_dim values of a row of q or k):
 *   y = x, or with a norm weight x * w / sqrt(mean(x^2) + eps)
 *       ("GGUF Inferencer in R", section 5.2, RMSN, over one head)
 *   out: pair (a, b) of y -> m (a cos t - b sin t), m (a sin t + b cos t), t the
 *        pair's angle, m the magnitude; other elements y.
 * q [n_tokens][n_heads * head_dim] and k [n_tokens][n_kv_heads * head_dim], strides in
 * elements from row to row; type F32 (GEMV outputs) or BF16 (prefill outputs),
 * outputs of the same type, all sums and products fp32, rounded once. Angles are
 * reduced in fp64 with what its products round off: positions of any size lose nothing.
 * q_norm and k_norm: fp32 [head_dim], either may be NULL (not normed). rope NULL: norms
 * only. n_heads or n_kv_heads may be 0 (its pointers are then not looked at).
 * head_dim even, 2 .. 512; n_heads and n_kv_heads at most 65535. q_out may be q and k_out
 * may be k (same stride); otherwise outputs may not overlap inputs or each other. Rows of q
 * and k may lie interleaved in one buffer (slices of one product's output) where their
 * strides are equal. Pointers aligned to their elements; rows that are 16-byte aligned, with head_dim and n_rot
 * multiples of 16 (BF16) or 8 (F32), run two to four times faster than others (32 + 8 heads
 * of 128: 8192 tokens in BF16 28 us and 106, 4096 in F32 27 and 55). */
int gguf_qk_rope(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int64_t n_heads,
                 const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride, int64_t n_kv_heads,
                 int32_t type, int64_t n_tokens, int64_t head_dim, const float* q_norm,
                 const float* k_norm, float eps, const gguf_rope* rope, hipStream_t stream);

/* --- attention of new tokens --------------------------------------------------- */

/* The rows of sequence s are rows row_start[s] .. row_start[s + 1] - 1 of q and out
 * (int32 [n_seqs + 1] on the device, ascending; row_start NULL: one row per sequence,
 * n_rows = n_seqs). They are the sequence's newest tokens: with n = min(lengths[s],
 * max_len) slots held, the new ones appended already, row j of m stands at slot
 * p = n - m + j. Per row and query head h (kv head h / (n_heads / n_kv_heads)), over
 * the slots i that the row sees,
 *   i <= p  and  (window == 0  or  i > p - window  or  i < sinks):
 *   w_i = softmax_i(scale * q . k_i),  out = sum_i w_i v_i
 * ("GGUF Inferencer in R", section 5.2.1, attend): causal among the new tokens, a
 * sliding window that counts the row's own slot, and `sinks` first slots that stay
 * visible behind it. A row that sees nothing (p < 0: an idle sequence) is zero. Rows
 * that belong to no sequence are left as they were; of row_start entries outside
 * 0 .. n_rows the part within counts. Windows and sinks count slots, as in
 * gguf_attn_decode. What lies in the pages behind a sequence's length is not looked at;
 * pages with an id outside the cache are left out.
 *
 * q and out of one type: F32 for single and drafted tokens, BF16 for prompts;
 * [n_rows][n_heads * head_dim], strides in elements from row to row (rows 16-byte
 * aligned), out may not overlap an input. max_len (<= 2^25) bounds the lengths:
 * longer sequences are taken to end there, as at the table's row.
 *
 * Limits (GGUF_QK_ERR_LIMIT past them): 2^23 rows, 2^20 sequences, 65535 query heads, 2^25
 * first slots, and 65535 tiles of columns, that is (n_rows * g + n_seqs * (c - 1)) / c with g
 * query heads per kv head and c = 16 or 32, or 128 where many rows run (below).
 *
 * One call, one kernel. Which kernel runs and how positions are split goes by the call's
 * totals, not by each sequence: a sequence of few rows and many slots among enough rows of
 * others is read by one block per kv head. Such calls are better made apart, each with its own
 * rows and row_start: one token behind 131072 slots beside a prompt of 1024 rows (BF16, 16
 * heads of 128 over 4) takes 2060 us in one call, 57 + 30 in two.
 *
 * Accuracy. F32: that of gguf_attn_decode. BF16: scores and sums in fp32, and where a
 * sequence has on average over the call more than 32 rows times query heads per kv head (16
 * for F16 and BF16 caches of head dims from 96 on) many rows run, for all of its sequences, so
 * that a row's roundings depend on the others:
 *   scores from exact products of q with the cache's values (F16 and Q8_0 caches: q's
 *     elements below 2^-26 of their head's greatest within 2^-34 of that; Q8_0: the nearest
 *     fp16 of a value, or within 2^-18 of the greatest scale of the slots read);
 *   softmax weights rounded to the operand type of the second product: bf16 for a BF16
 *     cache (2^-8 of each weight), fp16 otherwise (2^-11 of each, or 2^-25 of the row's
 *     greatest).
 * Below that as F32; the output is rounded once.
 * q, and keys and values within the length, have to be finite, as have their scaled
 * scores.
 *
 * Workspace. The size named serves every call with at most as many sequences and rows and
 * at most as large a bound, and the same cache, type, n_heads, window and sinks. It holds
 * partial results, head_dim + 2 fp32 numbers per row, query head and part of the positions:
 * at most 34 MB for prompts (BF16), but few rows and all F32 rows are cut into parts of at
 * most 1024 slots of the bound (or of window and first slots) however many they are, so that
 * there it grows with rows times bound: 64 sequences of 5 rows of 16 heads of 128 under a
 * bound of 131072 341 MB, 4096 F32 rows under 32768 1.1 GB. Bounds near the lengths, BF16
 * queries for prompts and calls over parts of the rows keep it small. */
int64_t gguf_attn_extend_workspace(const gguf_kv_cache* cache, int32_t type, int64_t n_seqs,
                                   int64_t n_rows, int64_t n_heads, int64_t max_len, int64_t window,
                                   int64_t sinks);
int gguf_attn_extend(const gguf_kv_cache* cache, const void* q, int32_t type, int64_t q_stride, void* out,
                     int64_t out_stride, const int32_t* row_start, int64_t n_rows, int64_t n_seqs,
                     int64_t n_heads, const int32_t* page_table, int64_t table_stride,
                     const int32_t* lengths, int64_t max_len, float scale, int64_t window, int64_t sinks,
                     void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* --- verification of drafted tokens ---------------------------------------------- */

/* Speculative decoding's acceptance with given random numbers. Sequence s has rows
 * row_start[s] .. row_start[s + 1] - 1 (int32 [n_seqs + 1], device, ascending, as
 * above): one per drafted token and a last one for the token behind them. Row r has
 * the target's logits target[r], the drafted token tokens[r] that they judge, the
 * logits draft[r] it was drawn from and a uniform random number uniform[r] in [0, 1);
 * tokens, draft and uniform of a sequence's last row are not looked at. With T =
 * temperature[s] (NULL: 1), p = softmax(target[r] / T), q = softmax(draft[r] / T)
 * (draft NULL: q is 1 at the drafted token and 0 elsewhere), t = tokens[r]:
 *   row r is accepted where  uniform[r] * q[t] < p[t];
 *   accepted[s] = rows before the first that is not (the last row never is);
 *   next[s] is drawn at that row r: from p if it is the last one, else from
 *     max(p - q, 0): the lowest i whose running sum exceeds uniform_next[s] times
 *     the whole (from p where p - q is nowhere above 0).
 * T = 0: p is 1 at the greatest logit (of equal ones the lowest index) and q is 1 at
 * the drafted token. accept_prob[r] (may be NULL) = min(1, p[t] / q[t]), 0 where p[t] is
 * 0, 1 for a sequence's last row; 0 for a token outside 0 .. vocab - 1, which is never accepted.
 * A sequence without rows has accepted 0 and next -1. Logits of -inf (ruled out) have
 * probability 0; a row without a finite greatest logit (all -inf, NaN, +inf), of
 * target or draft, accepts nothing, has accept_prob 0, and draws -1. Rows of no sequence are left alone.
 *
 * target and draft of one type, F32 or BF16, [n_rows][vocab], strides in elements from
 * row to row (>= vocab), aligned to their elements. Exponentials (to 2^-43) and sums
 * are fp64: a draw differs from the exact one only where the sum that uniform_next names
 * falls within 1e-12 of a boundary, with p's whole as 1; the whole of max(p - q, 0) is less
 * (a draft within 1 % of its target: some 0.01), so that there uniform_next itself counts to
 * 1e-12 over it. T >= 0 and finite (a negative or NaN T is taken as 0).
 * vocab <= 2^30, n_seqs <= 65535, n_rows * ceil(vocab / 8192) < 2^23. */
int64_t gguf_verify_draft_workspace(int64_t n_rows, int64_t n_seqs, int64_t vocab, int32_t has_draft);
int gguf_verify_draft(const void* target, int64_t target_stride, const void* draft, int64_t draft_stride,
                      int32_t type, const int32_t* tokens, const float* uniform, const float* uniform_next,
                      const int32_t* row_start, int64_t n_rows, int64_t n_seqs, int64_t vocab,
                      const float* temperature, int32_t* accepted, int32_t* next, float* accept_prob,
                      void* workspace, int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GGUF_TOKENS_H */
