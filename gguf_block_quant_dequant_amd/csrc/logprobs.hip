// Entry point of the log probabilities (include/gguf_kv.h).
#include "abi_check.hpp"
#include "logprobs.hpp"

using namespace gqk;

namespace gqk {

// Splits per row: the row's 16-byte words from the aligned address below its
// start (at most 15 bytes before it), 8192 values at a time.
static int64_t lp_splits(int64_t vocab) { return (vocab + 7 + kLpSplit - 1) / kLpSplit; }

static int lp_shape(int64_t n_rows, int64_t vocab, int32_t top_k) {
  if (n_rows < 0 || vocab < 1 || top_k < 0 || top_k > vocab) return GGUF_QK_ERR_SHAPE;
  if (top_k > kLpMaxTop || vocab > (int64_t(1) << 30)) return GGUF_QK_ERR_LIMIT;
  return GGUF_QK_OK;
}

// Partial sums, then candidate lists.
static int64_t lp_bytes(int64_t n_rows, int64_t splits, int32_t top_k, int64_t* part_bytes) {
  *part_bytes = abi_mul(abi_mul(n_rows, splits), 16);
  const int64_t lists = abi_mul(abi_mul(n_rows, splits), (int64_t)top_k * 8);
  if (*part_bytes < 0 || lists < 0 || lists > INT64_MAX - *part_bytes - 16) return -1;
  return splits == 1 ? 0 : *part_bytes + (lists + 15) / 16 * 16;
}

}  // namespace gqk

extern "C" {

int64_t gguf_logprobs_workspace(int64_t n_rows, int64_t vocab, int32_t top_k) {
  const int st = lp_shape(n_rows, vocab, top_k);
  if (st) return st;
  int64_t pb;
  const int64_t b = lp_bytes(n_rows, lp_splits(vocab), top_k, &pb);
  return b < 0 ? GGUF_QK_ERR_SHAPE : b;
}

int gguf_logprobs(const void* logits, int32_t type, int64_t n_rows, int64_t vocab, int64_t row_stride,
                  const int32_t* tokens, int64_t n_tokens, int32_t top_k, float* token_lp,
                  float* entropy, int32_t* top_id, float* top_lp, void* workspace,
                  int64_t workspace_bytes, hipStream_t stream) {
  if (!logits) return GGUF_QK_ERR_NULL;
  int st = lp_shape(n_rows, vocab, top_k);
  if (st) return st;
  if ((type != GGUF_KV_TYPE_F32 && type != GGUF_KV_TYPE_BF16) || n_tokens < 0 || n_tokens > INT32_MAX ||
      row_stride < vocab)
    return GGUF_QK_ERR_SHAPE;
  if ((n_tokens > 0 && (!tokens || !token_lp)) || (top_k > 0 && (!top_id || !top_lp))) return GGUF_QK_ERR_NULL;
  const int64_t es = type == GGUF_KV_TYPE_F32 ? 4 : 2;
  if (abi_mul(abi_mul(n_rows, row_stride), es) < 0 || abi_mul(abi_mul(n_rows, n_tokens), 4) < 0 ||
      abi_mul(abi_mul(n_rows, top_k), 4) < 0)
    return GGUF_QK_ERR_SHAPE;
  const int64_t splits = lp_splits(vocab);
  int64_t part_bytes;
  const int64_t need = lp_bytes(n_rows, splits, top_k, &part_bytes);
  if (need < 0) return GGUF_QK_ERR_SHAPE;
  if (!abi_aligned(logits, (uintptr_t)es) || !abi_aligned(tokens, 4) || !abi_aligned(token_lp, 4) ||
      !abi_aligned(entropy, 4) || !abi_aligned(top_id, 4) || !abi_aligned(top_lp, 4) || !abi_aligned(workspace, 16))
    return GGUF_QK_ERR_ALIGN;
  if (n_rows == 0) return GGUF_QK_OK;
  if (need > 0 && !workspace) return GGUF_QK_ERR_NULL;
  if (workspace_bytes < need) return GGUF_QK_ERR_LIMIT;
  const void* p[7] = {token_lp, entropy, top_id, top_lp, need > 0 ? workspace : nullptr, logits, tokens};
  const int64_t n[7] = {n_tokens > 0 ? n_rows * n_tokens * 4 : 0, n_rows * 4, top_k > 0 ? n_rows * top_k * 4 : 0,
                        top_k > 0 ? n_rows * top_k * 4 : 0, need, ((n_rows - 1) * row_stride + vocab) * es,
                        n_tokens > 0 ? n_rows * n_tokens * 4 : 0};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 7; ++j)
      if (abi_overlap(p[i], n[i], p[j], n[j])) return GGUF_QK_ERR_ALIAS;
  st = abi_device();
  if (st) return st;
  LogprobArgs a;
  a.x = static_cast<const uint8_t*>(logits);
  a.tokens = tokens;
  a.token_lp = token_lp;
  a.entropy = entropy;
  a.top_id = top_id;
  a.top_lp = top_lp;
  a.part = static_cast<float*>(workspace);
  a.cand = reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(workspace) + part_bytes);
  a.n_rows = n_rows;
  a.row_stride = row_stride;
  a.vocab = (int32_t)vocab;
  a.n_tokens = (int32_t)n_tokens;
  a.top_k = top_k;
  a.splits = (int32_t)splits;
  // rows over two grid axes
  const int64_t gy = n_rows < 32768 ? n_rows : 32768, gz = (n_rows + gy - 1) / gy;
  if (gz > 65535) return GGUF_QK_ERR_LIMIT;
  const dim3 grid((unsigned)splits, (unsigned)gy, (unsigned)gz), block(kLpThreads), rows((unsigned)gy, (unsigned)gz);
  if (type == GGUF_KV_TYPE_BF16) hipLaunchKernelGGL(logprobs_split_kernel<true>, grid, block, 0, stream, a);
  else hipLaunchKernelGGL(logprobs_split_kernel<false>, grid, block, 0, stream, a);
  st = abi_launched();
  if (st || splits == 1) return st;
  if (type == GGUF_KV_TYPE_BF16) hipLaunchKernelGGL(logprobs_join_kernel<true>, rows, block, 0, stream, a);
  else hipLaunchKernelGGL(logprobs_join_kernel<false>, rows, block, 0, stream, a);
  return abi_launched();
}

}  // extern "C"
