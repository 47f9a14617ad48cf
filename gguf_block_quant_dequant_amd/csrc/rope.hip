// Entry point of the norms and the rotation of queries and keys
// (include/gguf_tokens.h).
#include "../../include/gguf_tokens.h"
#include "abi_check.hpp"
#include "rope.hpp"

namespace gqk {

// Rows of a matrix in memory.
struct RopeRows {
  const void* p;
  int64_t row, stride, n;   // bytes of a row, from row to row, rows
};

// Whether any rows of a and b overlap. Rows of one stride may lie interleaved.
static bool rows_overlap(const RopeRows& a, const RopeRows& b) {
  if (!abi_overlap(a.p, (a.n - 1) * a.stride + a.row, b.p, (b.n - 1) * b.stride + b.row)) return false;
  if (a.stride != b.stride || a.stride == 0) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const int64_t s = a.stride, d = y >= x ? (int64_t)((y - x) % (uintptr_t)s) : (s - (int64_t)((x - y) % (uintptr_t)s)) % s;
  return d < a.row || s - d < b.row;
}

template <bool BF16, int VEC>
static void launch_rope(const RopeArgs& a, bool halves, dim3 grid, hipStream_t stream) {
  if (halves) hipLaunchKernelGGL((rope_kernel<BF16, VEC, true>), grid, dim3(kRopeThreads), 0, stream, a);
  else hipLaunchKernelGGL((rope_kernel<BF16, VEC, false>), grid, dim3(kRopeThreads), 0, stream, a);
}

}  // namespace gqk

using namespace gqk;

extern "C" int gguf_qk_rope(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int64_t n_heads,
                            const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride, int64_t n_kv_heads,
                            int32_t type, int64_t n_tokens, int64_t head_dim, const float* q_norm,
                            const float* k_norm, float eps, const gguf_rope* rope, hipStream_t stream) {
  if (n_heads < 0 || n_kv_heads < 0 || n_tokens < 0 || head_dim < 2 || head_dim % 2 || head_dim > kRopeMaxDim ||
      (type != GGUF_KV_TYPE_F32 && type != GGUF_KV_TYPE_BF16))
    return GGUF_QK_ERR_SHAPE;
  if (n_heads > 65535 || n_kv_heads > 65535) return GGUF_QK_ERR_LIMIT;
  if ((n_heads > 0 && (!q || !q_out)) || (n_kv_heads > 0 && (!k || !k_out))) return GGUF_QK_ERR_NULL;
  const int64_t es = type == GGUF_KV_TYPE_F32 ? 4 : 2;
  const void* in[2] = {q, k};
  void* out[2] = {q_out, k_out};
  const int64_t heads[2] = {n_heads, n_kv_heads}, is[2] = {q_stride, k_stride}, os[2] = {q_out_stride, k_out_stride};
  const float* norm[2] = {q_norm, k_norm};
  if ((norm[0] || norm[1]) && !(eps >= 0.f && eps - eps == 0.f)) return GGUF_QK_ERR_SHAPE;
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    if (is[i] < heads[i] * head_dim || os[i] < heads[i] * head_dim) return GGUF_QK_ERR_SHAPE;
    if (abi_mul(abi_mul(n_tokens, is[i]), es) < 0 || abi_mul(abi_mul(n_tokens, os[i]), es) < 0) return GGUF_QK_ERR_SHAPE;
  }
  int64_t half = 0;
  if (rope) {
    if (rope->n_rot < 0 || rope->n_rot % 2 || rope->n_rot > head_dim || rope->n_axes < 1 || rope->n_axes > 16 ||
        rope->pos_stride < n_tokens || (rope->pairing != GGUF_ROPE_ADJACENT && rope->pairing != GGUF_ROPE_HALVES) ||
        !(rope->magnitude - rope->magnitude == 0.f) || abi_mul(abi_mul(rope->pos_stride, rope->n_axes), 4) < 0)
      return GGUF_QK_ERR_SHAPE;
    half = rope->n_rot / 2;
    if (half > 0 && (!rope->freqs || !rope->pos)) return GGUF_QK_ERR_NULL;
    if (half > 0 && (!abi_aligned(rope->freqs, 8) || !abi_aligned(rope->axes, 4) || !abi_aligned(rope->pos, 4)))
      return GGUF_QK_ERR_ALIGN;
  }
  // runs of 16 bytes where everything allows them
  const int64_t vec = 16 / es;
  bool wide = head_dim % (2 * vec) == 0 && half % vec == 0;
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    if (!abi_aligned(in[i], (uintptr_t)es) || !abi_aligned(out[i], (uintptr_t)es) || !abi_aligned(norm[i], 4))
      return GGUF_QK_ERR_ALIGN;
    wide = wide && abi_aligned(in[i], 16) && abi_aligned(out[i], 16) && is[i] % vec == 0 && os[i] % vec == 0;
  }
  if (n_tokens == 0 || n_heads + n_kv_heads == 0) return GGUF_QK_OK;
  for (int i = 0; i < 2; ++i) {
    if (heads[i] == 0) continue;
    const int64_t row = heads[i] * head_dim * es;
    const RopeRows o = {out[i], row, os[i] * es, n_tokens};
    const int64_t whole = (n_tokens - 1) * o.stride + row;
    for (int j = 0; j < 2; ++j) {
      if (heads[j] == 0) continue;
      const int64_t jrow = heads[j] * head_dim * es;
      const bool same = i == j && in[j] == out[i] && is[j] == os[i];
      if (!same && rows_overlap(o, RopeRows{in[j], jrow, is[j] * es, n_tokens})) return GGUF_QK_ERR_ALIAS;
      if (j > i && rows_overlap(o, RopeRows{out[j], jrow, os[j] * es, n_tokens})) return GGUF_QK_ERR_ALIAS;
      if (abi_overlap(out[i], whole, norm[j], head_dim * 4)) return GGUF_QK_ERR_ALIAS;
    }
    if (half > 0 && (abi_overlap(out[i], whole, rope->freqs, half * 8) || abi_overlap(out[i], whole, rope->axes, half * 4) ||
                     abi_overlap(out[i], whole, rope->pos, ((rope->n_axes - 1) * rope->pos_stride + n_tokens) * 4)))
      return GGUF_QK_ERR_ALIAS;
  }
  const int st = abi_device();
  if (st) return st;
  RopeArgs a;
  for (int i = 0; i < 2; ++i) {
    a.in[i] = static_cast<const uint8_t*>(in[i]);
    a.out[i] = static_cast<uint8_t*>(out[i]);
    a.in_stride[i] = is[i] * es;
    a.out_stride[i] = os[i] * es;
    a.norm[i] = norm[i];
    a.heads[i] = (int32_t)heads[i];
  }
  a.freqs = half > 0 ? rope->freqs : nullptr;
  a.axes = half > 0 ? rope->axes : nullptr;
  a.pos = half > 0 ? rope->pos : nullptr;
  a.pos_stride = half > 0 ? rope->pos_stride : 0;
  a.n_tokens = n_tokens;
  a.n_axes = half > 0 ? rope->n_axes : 0;
  a.n_rot = (int32_t)(2 * half);
  a.head_dim = (int32_t)head_dim;
  a.eps = eps;
  a.magnitude = half > 0 ? rope->magnitude : 1.f;
  const int64_t units = head_dim / 2 / (wide ? vec : 1);
  a.lanes = 1;
  while (a.lanes < 64 && a.lanes < units) a.lanes *= 2;
  // tokens per block: one while that fills the device, then as many as the angles' space and 8 allow
  int64_t tokens = n_tokens / 2048;
  const int64_t most = half > 0 ? kRopeAngles / half : 8;
  tokens = tokens < 1 ? 1 : tokens > 8 ? 8 : tokens;
  if (tokens > most) tokens = most;
  a.tokens = (int32_t)tokens;
  const int64_t blocks = (n_tokens + tokens - 1) / tokens;
  if (blocks > INT32_MAX / kRopeThreads) return GGUF_QK_ERR_LIMIT;
  const dim3 grid((unsigned)blocks);
  const bool halves = rope && rope->pairing == GGUF_ROPE_HALVES;
  if (type == GGUF_KV_TYPE_BF16) {
    if (wide) launch_rope<true, 8>(a, halves, grid, stream);
    else launch_rope<true, 1>(a, halves, grid, stream);
  } else {
    if (wide) launch_rope<false, 4>(a, halves, grid, stream);
    else launch_rope<false, 1>(a, halves, grid, stream);
  }
  return abi_launched();
}
