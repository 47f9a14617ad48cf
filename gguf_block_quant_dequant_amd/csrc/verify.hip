// Entry points of the verification of drafted tokens (include/gguf_tokens.h).
#include "../../include/gguf_tokens.h"
#include "abi_check.hpp"
#include "verify.hpp"

namespace gqk {

// The workspace's parts: splits' sums, choices, what is drawn from.
struct VerifyPlan {
  int64_t splits, part_bytes, choice_bytes, bytes;
};

static int verify_plan(int64_t n_rows, int64_t n_seqs, int64_t vocab, bool draft, VerifyPlan* p) {
  if (n_rows < 0 || n_seqs < 0 || vocab < 1) return GGUF_QK_ERR_SHAPE;
  if (vocab > (int64_t(1) << 30) || n_seqs > 65535) return GGUF_QK_ERR_LIMIT;
  p->splits = (vocab + kVerifySplit - 1) / kVerifySplit;
  if (p->splits > INT32_MAX / kDrawThreads) return GGUF_QK_ERR_LIMIT;
  const int64_t blocks = abi_mul(n_rows, p->splits);
  if (blocks < 0 || blocks > INT32_MAX / kVerifyThreads) return GGUF_QK_ERR_LIMIT;   // threads of a grid axis
  p->part_bytes = blocks * (draft ? 2 : 1) * (int64_t)sizeof(double2);
  p->choice_bytes = (n_seqs * (int64_t)sizeof(VerifyChoice) + 15) / 16 * 16;
  p->bytes = p->part_bytes + p->choice_bytes + n_seqs * p->splits * 8;
  return GGUF_QK_OK;
}

template <bool BF16, bool WIDE>
static int launch_verify(const VerifyArgs& a, hipStream_t stream) {
  const dim3 block(kVerifyThreads);
  if (a.n_rows > 0) {
    hipLaunchKernelGGL((verify_sums_kernel<BF16, WIDE>), dim3((unsigned)(a.n_rows * a.splits), a.x[1] ? 2 : 1), block, 0,
                       stream, a);
    const int st = abi_launched();
    if (st) return st;
  }
  hipLaunchKernelGGL((verify_choose_kernel<BF16, WIDE>), dim3((unsigned)a.splits, (unsigned)a.n_seqs), dim3(kChooseThreads),
                     0, stream, a);
  const int st = abi_launched();
  if (st || a.n_rows == 0) return st;
  hipLaunchKernelGGL((verify_draw_kernel<BF16, WIDE>), dim3((unsigned)a.n_seqs), dim3(kDrawThreads), 0, stream, a);
  return abi_launched();
}

}  // namespace gqk

using namespace gqk;

extern "C" {

int64_t gguf_verify_draft_workspace(int64_t n_rows, int64_t n_seqs, int64_t vocab, int32_t has_draft) {
  VerifyPlan p;
  const int st = verify_plan(n_rows, n_seqs, vocab, has_draft != 0, &p);
  return st ? st : p.bytes;
}

int gguf_verify_draft(const void* target, int64_t target_stride, const void* draft, int64_t draft_stride, int32_t type,
                      const int32_t* tokens, const float* uniform, const float* uniform_next, const int32_t* row_start,
                      int64_t n_rows, int64_t n_seqs, int64_t vocab, const float* temperature, int32_t* accepted,
                      int32_t* next, float* accept_prob, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  VerifyPlan p;
  int st = verify_plan(n_rows, n_seqs, vocab, draft != nullptr, &p);
  if (st) return st;
  if (type != GGUF_KV_TYPE_F32 && type != GGUF_KV_TYPE_BF16) return GGUF_QK_ERR_SHAPE;
  const int64_t es = type == GGUF_KV_TYPE_F32 ? 4 : 2;
  if (n_seqs == 0) return GGUF_QK_OK;
  if (!row_start || !uniform_next || !accepted || !next || !workspace || (n_rows > 0 && (!target || !tokens || !uniform)))
    return GGUF_QK_ERR_NULL;
  if (target_stride < vocab || (draft && draft_stride < vocab) || abi_mul(abi_mul(n_rows, target_stride), es) < 0 ||
      (draft && abi_mul(abi_mul(n_rows, draft_stride), es) < 0))
    return GGUF_QK_ERR_SHAPE;
  if (!abi_aligned(target, (uintptr_t)es) || !abi_aligned(draft, (uintptr_t)es) || !abi_aligned(tokens, 4) ||
      !abi_aligned(uniform, 4) || !abi_aligned(uniform_next, 4) || !abi_aligned(row_start, 4) ||
      !abi_aligned(temperature, 4) || !abi_aligned(accepted, 4) || !abi_aligned(next, 4) || !abi_aligned(accept_prob, 4) ||
      !abi_aligned(workspace, 16))
    return GGUF_QK_ERR_ALIGN;
  if (workspace_bytes < p.bytes) return GGUF_QK_ERR_LIMIT;
  const void* ptr[11] = {accepted, next, accept_prob, workspace, target, draft, tokens, uniform, uniform_next, row_start, temperature};
  const int64_t len[11] = {n_seqs * 4, n_seqs * 4, n_rows * 4, p.bytes,
                           n_rows > 0 ? ((n_rows - 1) * target_stride + vocab) * es : 0,
                           draft && n_rows > 0 ? ((n_rows - 1) * draft_stride + vocab) * es : 0, n_rows * 4, n_rows * 4,
                           n_seqs * 4, (n_seqs + 1) * 4, n_seqs * 4};
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 11; ++j)
      if (abi_overlap(ptr[i], len[i], ptr[j], len[j])) return GGUF_QK_ERR_ALIAS;
  st = abi_device();
  if (st) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  VerifyArgs a;
  a.x[0] = static_cast<const uint8_t*>(target);
  a.x[1] = static_cast<const uint8_t*>(draft);
  a.stride[0] = target_stride;
  a.stride[1] = draft ? draft_stride : 0;
  a.tokens = tokens;
  a.uniform = uniform;
  a.uniform_next = uniform_next;
  a.row_start = row_start;
  a.temperature = temperature;
  a.accepted = accepted;
  a.next = next;
  a.prob = accept_prob;
  a.part = reinterpret_cast<double2*>(ws);
  a.choice = reinterpret_cast<VerifyChoice*>(ws + p.part_bytes);
  a.rest = reinterpret_cast<double*>(ws + p.part_bytes + p.choice_bytes);
  a.n_rows = n_rows;
  a.n_seqs = (int32_t)n_seqs;
  a.vocab = (int32_t)vocab;
  a.splits = (int32_t)p.splits;
  const bool wide = abi_aligned(target, 16) && target_stride * es % 16 == 0 && abi_aligned(draft, 16) &&
                    (!draft || draft_stride * es % 16 == 0);
  if (type == GGUF_KV_TYPE_BF16) return wide ? launch_verify<true, true>(a, stream) : launch_verify<true, false>(a, stream);
  return wide ? launch_verify<false, true>(a, stream) : launch_verify<false, false>(a, stream);
}

}  // extern "C"
