/*
 * gguf_kv.h -- C ABI of libgguf_qk.so, the steps of a decode pass that follow
 * the GEMVs of gguf_qk.h: a paged key-value cache, the attention of one new
 * token over it, eviction from it, and the log probabilities read from the
 * output head.
 *
 * The conventions are those of gguf_qk.h: device pointers into memory the
 * caller owns, work enqueued on `stream` of the current device, arguments
 * validated before any HIP call (a failed call enqueues nothing), the same
 * status codes, nothing allocated, no pointer kept. In place of the scratch
 * slots of gguf_qk.h these calls take a workspace: uninitialized device memory
 * of the size the _workspace call names, 16-byte aligned, which the call's
 * kernels write before they read it. Two calls whose work may overlap in time
 * (on two streams, or in two captured graphs replayed at once) need a
 * workspace each. All work is deterministic: no result depends on the order in
 * which blocks run.
 */
#ifndef GGUF_KV_H
#define GGUF_KV_H

#include "gguf_qk.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Cache and logit types besides GGUF_QK_TYPE_Q8_0 (GGUF's tensor type ids). */
#define GGUF_KV_TYPE_F32 0
#define GGUF_KV_TYPE_F16 1
#define GGUF_KV_TYPE_BF16 30

/* --- the cache -------------------------------------------------------------- */

/* Keys and values of one layer in pages of page_size positions ("GGUF
 * Inferencer in R", section 5.2.1: per head the K rows are appended and V is
 * stored transposed). Page g of K holds, per kv head, page_size rows of
 * head_dim values; page g of V holds, per kv head, head_dim rows of page_size
 * values (so eight consecutive positions of one dim are one 16-byte load, the
 * operand of the matrix instruction that multiplies by V):
 *   K [n_pages][n_kv_heads][page_size][head_dim]
 *   V [n_pages][n_kv_heads][head_dim][page_size]
 * F16 and BF16 store the values so. Q8_0 stores Q8_0's codes and scales (32
 * consecutive dims of one position share an fp16 scale d; value = code * d),
 * kept apart per page and kv head so that both load aligned: the int8 codes in
 * the order above, behind them the scales (K [page_size][head_dim / 32],
 * V [head_dim / 32][page_size]).
 *
 * weight (fp32) and pos (int32), [n_pages][n_kv_heads][page_size] each, are
 * optional (NULL): the attention weight a slot has received so far, and the
 * position its token had in the sequence. Eviction leaves slots in another
 * order than positions, in each kv head another; attention over all of them
 * (window 0) does not depend on the order, a window does.
 *
 * type: F16, BF16 or Q8_0. head_dim: 64, 96, 128, 192 or 256. page_size: a
 * power of two from 16 to 256. All pointers 16-byte aligned. */
typedef struct gguf_kv_cache {
  void* k;
  void* v;
  float* weight;
  int32_t* pos;
  int64_t n_pages;
  int32_t type;
  int32_t n_kv_heads;
  int32_t head_dim;
  int32_t page_size;
} gguf_kv_cache;

/* Every call below reads the page table: int32 [n_seqs][table_stride], row s
 * the page ids of sequence s in order (slot i of the sequence is slot
 * i % page_size of page table[s][i / page_size]). Ids outside 0 .. n_pages - 1
 * are never followed: a token appended there is dropped, positions there are
 * left out of the attention and of the eviction's moves. Entries past a
 * sequence's last page are not used. */

/* Bytes of one page of K, which are those of one page of V, or
 * GGUF_QK_ERR_SHAPE. */
int64_t gguf_kv_page_bytes(int type, int64_t n_kv_heads, int64_t head_dim, int64_t page_size);

/* Writes n_tokens tokens into the cache. Token t's key and value are rows t of
 * k and v, [n_tokens][n_kv_heads * head_dim] with row_stride elements from row
 * to row, src_type F32 (GEMV outputs) or BF16 (prefill outputs); they go to
 * slot[t] of sequence seq[t] (seq NULL: sequence t), rounded once to F16 or
 * BF16 (nearest-even; magnitudes past F16's range become infinities) or
 * quantized to Q8_0 (d = max|x| / 127 over 32 dims, stored as fp16; codes
 * round(x / d), ties to even, within +-127; zeros where d is 0; values have to
 * be finite and below 8.3e6, where d leaves fp16's range). Where the cache has
 * them, the slots' weight becomes 0 and pos becomes pos[t] (pos NULL: slot[t],
 * which is the position only while a sequence has not been evicted from: after an
 * eviction slots start again at the budget, and `recent` would take such a token
 * for an old one; pass pos).
 * A token whose seq is outside 0 .. n_seqs - 1 or whose slot is outside the
 * table's row (a padding row, marked -1) is dropped. No two tokens of a call may
 * name the same slot (its contents are then undefined).
 * k, v 16-byte aligned, rows a multiple of 16 bytes apart. */
int gguf_kv_append(const gguf_kv_cache* cache, const void* k, const void* v, int32_t src_type,
                   int64_t row_stride, int64_t n_tokens, const int32_t* seq, const int32_t* slot,
                   const int32_t* pos, const int32_t* page_table, int64_t table_stride, int64_t n_seqs,
                   hipStream_t stream);

/* --- attention of one new token --------------------------------------------- */

/* Per sequence s and query head h (kv head h / (n_heads / n_kv_heads)), over
 * the positions i of [first, n), n = min(lengths[s], max_len) and first =
 * n - window or 0 (window 0: all positions):
 *   p_i = softmax_i(scale * q . k_i),  out = sum_i p_i v_i
 * ("GGUF Inferencer in R", section 5.2.1, attend). q, out: fp32
 * [n_seqs][n_heads * head_dim], q_stride and out_stride floats from row to row
 * (multiples of 4; the range from out's first row to its last may not overlap an
 * input's). A row with no position left (lengths[s] <= 0: an idle slot of the
 * batch) is zero. What lies in the pages behind a sequence's length is not
 * looked at, whatever it holds; q, and keys and values within the length, have
 * to be finite, as have scale * log2(e) (|scale| up to 2.35e38, checked), its
 * products with q, and the scores times log2(e), in fp32.
 *
 * A window counts slots and does not look at cache->pos: it is the window's newest
 * tokens only where slots are in the order of positions, which they no longer are
 * once gguf_kv_evict has cut the sequence. Where both are wanted, let the eviction
 * keep the window: append, gguf_kv_evict with budget = recent = the window (it
 * leaves exactly the tokens with pos > max pos - window), then window 0 here.
 *
 * max_len (<= 2^25) is a bound on the lengths that the host knows (it sets the
 * grid and the workspace); longer sequences are cut at it, as at the table's
 * row. One captured call can serve growing sequences under a bound far above
 * them, at a price. For up to 64 sequences that together have fewer than 768 kv
 * heads (384 past head dim 128; Q8_0: 448) the positions are cut to the lengths on
 * the device: 4 sequences of 3000, 4 kv heads of 128, 13.4 us under 3000 and 14.6
 * under 131072; 16 of 1000, 14.6 and 17.7; 64 of 1000, 36 and 61, most of it empty
 * blocks. Beyond, the bound alone decides: 128 of 1000, 65 and 107. With track the
 * workspace holds 4 bytes per sequence, query head and position of the bound, and
 * the blocks that add the weights cover it: 64 of 1000, 16 heads, 6 MiB and 38 us
 * under 1000, 577 MiB and 100 us under 131072.
 *
 * With track, weight[slot] of the cache grows by p_i summed over the query heads of
 * the kv head (needs cache->weight; a page then belongs to one sequence of the
 * call). Without, sequences may share pages.
 *
 * The workspace serves every call with at most as many sequences and at most as
 * large a bound, any window, and the same cache, n_heads and track.
 *
 * Scores, maxima, sums and outputs are fp32. The matrix cores take the exact cache
 * values against fp32 operands in parts: three bf16 (BF16 cache), which hold their 24
 * bits, or two fp16 (F16 and Q8_0), which hold 22 bits of all but the smallest. Off by
 * 2^-22 of itself or, where that is more:
 *   an element of q by 2^-34 of its row's greatest,
 *   a softmax weight (F16) by 2^-39 of the greatest,
 *   a softmax weight times V's scale (Q8_0) by the greatest weight times 2^-39 of the
 *     32-dim block's greatest scale, 2^-54 of the head's greatest, or 2^-54
 * so that outputs lose digits only where values some 2^17 times larger than those of
 * the heavy positions lie under weights below 2^-17. The sums over the positions'
 * |v| have to stay within fp32. */
int64_t gguf_attn_decode_workspace(const gguf_kv_cache* cache, int64_t n_seqs, int64_t n_heads,
                                   int64_t max_len, int32_t track);
int gguf_attn_decode(const gguf_kv_cache* cache, const float* q, int64_t q_stride, float* out,
                     int64_t out_stride, int64_t n_seqs, int64_t n_heads, const int32_t* page_table,
                     int64_t table_stride, const int32_t* lengths, int64_t max_len, float scale,
                     int64_t window, int32_t track, void* workspace, int64_t workspace_bytes,
                     hipStream_t stream);

/* --- eviction ----------------------------------------------------------------- */

/* Cuts every sequence longer than budget to budget slots, per kv head: kept are
 * the budget slots of greatest accumulated weight, where the newest `recent`
 * tokens (pos > max pos - recent; needs cache->pos unless recent is 0) count as
 * greater than any weight, a NaN weight as greater than any number, and of
 * equal ones the lower slots are kept. The kept slots at or behind
 * budget then move, in order, into the vacated slots before it (K, V, weight
 * and pos), so a call moves no more than it has to, and lengths[s] becomes
 * budget. The slots from budget on are left as they were and their pages are
 * free. Sequences of at most budget slots are left alone.
 * max_len (<= 2^30) has to be a bound that no length exceeds, nor may a length pass
 * its table row: such a sequence is taken to end there, and as it is cut to budget
 * all the same, the slots behind (the newest tokens, with or without `recent`) are
 * lost without having been looked at; with max_len <= budget nothing is selected and
 * the first budget slots stay. A call captured into a graph needs the bound of its
 * last replay. budget >= 1, 0 <= recent <= budget; cache->weight is needed; a page
 * belongs to one sequence. */
int64_t gguf_kv_evict_workspace(const gguf_kv_cache* cache, int64_t n_seqs, int64_t max_len,
                                int64_t budget);
int gguf_kv_evict(const gguf_kv_cache* cache, int64_t n_seqs, const int32_t* page_table,
                  int64_t table_stride, int32_t* lengths, int64_t max_len, int64_t budget,
                  int64_t recent, void* workspace, int64_t workspace_bytes, hipStream_t stream);

/* --- log probabilities ---------------------------------------------------------- */

/* Per row of logits x (F32 or BF16, [n_rows][vocab] with row_stride elements
 * from row to row), with lse = log sum_i exp(x_i):
 *   token_lp[r][j] = x[tokens[r][j]] - lse     for the n_tokens given tokens
 *                    (-inf for a token outside 0 .. vocab - 1)
 *   entropy[r]     = -sum_i p_i log p_i,  p_i = exp(x_i - lse)
 *   top_id[r][j], top_lp[r][j]   the top_k greatest logits in order, of equal
 *                    ones the lowest index first (NaN greatest)
 * all outputs fp32 (top_id int32), rows back to back. Logits of -inf (ruled-out
 * tokens) have probability 0; a row of nothing else, or with NaN or +inf in
 * it, gives NaN. token_lp (with n_tokens 0), entropy or the top pair (with
 * top_k 0) may be NULL. top_k <= 64 and <= vocab; vocab <= 2^30. logits aligned
 * to their elements, row_stride >= vocab. Where 8192 consecutive logits hold no
 * more than about top_k values above -inf, they are read again for each of the
 * top_k: 64 rows of 128256 with the top 20 take 15 us with 99 % ruled out and 234
 * with 99.9 %. */
int64_t gguf_logprobs_workspace(int64_t n_rows, int64_t vocab, int32_t top_k);
int gguf_logprobs(const void* logits, int32_t type, int64_t n_rows, int64_t vocab, int64_t row_stride,
                  const int32_t* tokens, int64_t n_tokens, int32_t top_k, float* token_lp,
                  float* entropy, int32_t* top_id, float* top_lp, void* workspace,
                  int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GGUF_KV_H */
