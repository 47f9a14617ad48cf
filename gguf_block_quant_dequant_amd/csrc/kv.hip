// Entry points of the paged key-value cache (include/gguf_kv.h): its checks,
// append and eviction. Host code validates, picks launch shapes and launches.
#include "abi_check.hpp"
#include "kv_cache.hpp"

namespace gqk {

int kv_view(const gguf_kv_cache* cache, KvView* view) {
  if (!cache || !cache->k || !cache->v) return GGUF_QK_ERR_NULL;
  const int64_t hb = gguf_kv_page_bytes(cache->type, 1, cache->head_dim, cache->page_size);
  if (hb < 0 || cache->n_kv_heads < 1 || cache->n_pages < 1) return GGUF_QK_ERR_SHAPE;
  if (cache->n_pages > INT32_MAX) return GGUF_QK_ERR_SHAPE;
  if (cache->n_kv_heads > 65535) return GGUF_QK_ERR_LIMIT;   // heads lie along a grid axis
  const int64_t heads = abi_mul(cache->n_pages, cache->n_kv_heads);
  if (heads < 0 || abi_mul(heads, hb) < 0 || abi_mul(heads, (int64_t)cache->page_size * 4) < 0)
    return GGUF_QK_ERR_SHAPE;
  if (!abi_aligned(cache->k, 16) || !abi_aligned(cache->v, 16) || !abi_aligned(cache->weight, 16) ||
      !abi_aligned(cache->pos, 16))
    return GGUF_QK_ERR_ALIGN;
  KvView c;
  c.k = static_cast<uint8_t*>(cache->k);
  c.v = static_cast<uint8_t*>(cache->v);
  c.weight = cache->weight;
  c.pos = cache->pos;
  c.n_pages = cache->n_pages;
  c.head_bytes = hb;
  c.hkv = cache->n_kv_heads;
  c.dim = cache->head_dim;
  c.ps = cache->page_size;
  c.shift = __builtin_ctz((unsigned)cache->page_size);
  const int64_t kb = kv_bytes(c), pb = kv_plane_bytes(c);
  if (abi_overlap(c.k, kb, c.v, kb) || abi_overlap(c.weight, pb, c.k, kb) || abi_overlap(c.weight, pb, c.v, kb) ||
      abi_overlap(c.pos, pb, c.k, kb) || abi_overlap(c.pos, pb, c.v, kb) || abi_overlap(c.weight, pb, c.pos, pb))
    return GGUF_QK_ERR_ALIAS;
  *view = c;
  return GGUF_QK_OK;
}

static KvKind kind_of(int32_t type) {
  return type == GGUF_KV_TYPE_F16 ? kKvF16 : type == GGUF_KV_TYPE_BF16 ? kKvBF16 : kKvQ80;
}

// Calls fn.template operator()<KIND, DIM>() for the cache's type and head dim.
template <int KIND, class Fn>
static void by_dim(int dim, Fn&& fn) {
  switch (dim) {
    case 64: return fn.template operator()<KIND, 64>();
    case 96: return fn.template operator()<KIND, 96>();
    case 128: return fn.template operator()<KIND, 128>();
    case 192: return fn.template operator()<KIND, 192>();
    default: return fn.template operator()<KIND, 256>();
  }
}
template <class Fn>
static void by_cache(KvKind kind, int dim, Fn&& fn) {
  if (kind == kKvF16) by_dim<kKvF16>(dim, fn);
  else if (kind == kKvBF16) by_dim<kKvBF16>(dim, fn);
  else by_dim<kKvQ80>(dim, fn);
}

struct LaunchAppend {
  const AppendArgs& a;
  dim3 grid;
  bool bf16;
  hipStream_t stream;
  template <int KIND, int DIM>
  void operator()() const {
    if (bf16)
      hipLaunchKernelGGL((kv_append_kernel<KIND, true, DIM>), grid, dim3(kAppendThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((kv_append_kernel<KIND, false, DIM>), grid, dim3(kAppendThreads), 0, stream, a);
  }
};

struct LaunchMove {
  const EvictArgs& a;
  dim3 grid;
  hipStream_t stream;
  template <int KIND, int DIM>
  void operator()() const {
    hipLaunchKernelGGL((kv_evict_move_kernel<KIND, DIM>), grid, dim3(kMoveThreads), 0, stream, a);
  }
};

constexpr int64_t kMaxLen = int64_t(1) << 30;   // slots of a sequence (32-bit slot arithmetic)

// Workspace of an eviction: counts, then both lists, each 16-byte aligned.
struct EvictPlan {
  int64_t pairs, moves, count_bytes, list_bytes, bytes;
};
static int evict_plan(const KvView& c, int64_t n_seqs, int64_t max_len, int64_t budget, EvictPlan* p) {
  if (n_seqs < 0 || max_len < 0 || budget < 1) return GGUF_QK_ERR_SHAPE;
  if (n_seqs > 65535 || max_len > kMaxLen) return GGUF_QK_ERR_LIMIT;
  p->pairs = n_seqs * c.hkv;
  const int64_t over = max_len > budget ? max_len - budget : 0;
  p->moves = over < budget ? over : budget;
  p->count_bytes = (p->pairs * 4 + 15) / 16 * 16;
  p->list_bytes = (p->pairs * p->moves * 4 + 15) / 16 * 16;   // < 2^32 * 2^30 * 4: fits
  p->bytes = p->count_bytes + 2 * p->list_bytes;
  return GGUF_QK_OK;
}

}  // namespace gqk

using namespace gqk;

extern "C" {

int64_t gguf_kv_page_bytes(int type, int64_t n_kv_heads, int64_t head_dim, int64_t page_size) {
  if (type != GGUF_KV_TYPE_F16 && type != GGUF_KV_TYPE_BF16 && type != GGUF_QK_TYPE_Q8_0) return GGUF_QK_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 96 && head_dim != 128 && head_dim != 192 && head_dim != 256)
    return GGUF_QK_ERR_SHAPE;
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1))) return GGUF_QK_ERR_SHAPE;
  if (n_kv_heads < 1) return GGUF_QK_ERR_SHAPE;
  const int64_t b = abi_mul(n_kv_heads, kv_head_bytes(type == GGUF_QK_TYPE_Q8_0, head_dim, page_size));
  return b < 0 ? GGUF_QK_ERR_SHAPE : b;
}

int gguf_kv_append(const gguf_kv_cache* cache, const void* k, const void* v, int32_t src_type,
                   int64_t row_stride, int64_t n_tokens, const int32_t* seq, const int32_t* slot,
                   const int32_t* pos, const int32_t* page_table, int64_t table_stride, int64_t n_seqs,
                   hipStream_t stream) {
  AppendArgs a;
  int st = kv_view(cache, &a.c);
  if (st) return st;
  if (!k || !v || !slot || !page_table) return GGUF_QK_ERR_NULL;
  if (src_type != GGUF_KV_TYPE_F32 && src_type != GGUF_KV_TYPE_BF16) return GGUF_QK_ERR_SHAPE;
  const int64_t es = src_type == GGUF_KV_TYPE_F32 ? 4 : 2;
  const int64_t row = (int64_t)a.c.hkv * a.c.dim;
  if (n_tokens < 0 || n_seqs < 0 || table_stride < 1 || row_stride < row) return GGUF_QK_ERR_SHAPE;
  if (abi_mul(abi_mul(n_tokens, row_stride), es) < 0 || abi_mul(abi_mul(n_seqs, table_stride), 4) < 0)
    return GGUF_QK_ERR_SHAPE;
  if (!abi_aligned(k, 16) || !abi_aligned(v, 16) || row_stride * es % 16) return GGUF_QK_ERR_ALIGN;
  if (!abi_aligned(seq, 4) || !abi_aligned(slot, 4) || !abi_aligned(pos, 4) || !abi_aligned(page_table, 4))
    return GGUF_QK_ERR_ALIGN;
  if (n_tokens == 0) return GGUF_QK_OK;
  const int64_t in = ((n_tokens - 1) * row_stride + row) * es;
  if (kv_touches(a.c, k, in) || kv_touches(a.c, v, in) || kv_touches(a.c, seq, n_tokens * 4) ||
      kv_touches(a.c, slot, n_tokens * 4) || kv_touches(a.c, pos, n_tokens * 4) ||
      kv_touches(a.c, page_table, n_seqs * table_stride * 4))
    return GGUF_QK_ERR_ALIAS;
  st = abi_device();
  if (st) return st;
  a.k = k;
  a.v = v;
  a.seq = seq;
  a.slot = slot;
  a.pos = pos;
  a.table = page_table;
  a.row_stride = row_stride;
  a.table_stride = table_stride;
  a.n_tokens = n_tokens;
  a.n_seqs = n_seqs;
  // few tokens: small tiles, so that more CUs work on them (64 tokens, 8 heads:
  // 3.7 us, 4.5 in tiles of 64; 2048 tokens 5.1 against 5.7)
  a.tile = kAppendTile;
  while (a.tile > 8 && (n_tokens + a.tile - 1) / a.tile * a.c.hkv < 512) a.tile /= 2;
  const int64_t blocks = (n_tokens + a.tile - 1) / a.tile;
  if (blocks > INT32_MAX / kAppendThreads) return GGUF_QK_ERR_LIMIT;   // threads of a grid axis
  by_cache(kind_of(cache->type), a.c.dim,
           LaunchAppend{a, dim3((unsigned)blocks, (unsigned)a.c.hkv), src_type == GGUF_KV_TYPE_BF16, stream});
  return abi_launched();
}

int64_t gguf_kv_evict_workspace(const gguf_kv_cache* cache, int64_t n_seqs, int64_t max_len, int64_t budget) {
  KvView c;
  int st = kv_view(cache, &c);
  if (st) return st;
  EvictPlan p;
  st = evict_plan(c, n_seqs, max_len, budget, &p);
  return st ? st : p.bytes;
}

int gguf_kv_evict(const gguf_kv_cache* cache, int64_t n_seqs, const int32_t* page_table,
                  int64_t table_stride, int32_t* lengths, int64_t max_len, int64_t budget,
                  int64_t recent, void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  EvictArgs a;
  int st = kv_view(cache, &a.c);
  if (st) return st;
  if (!page_table || !lengths || !a.c.weight || (recent != 0 && !a.c.pos)) return GGUF_QK_ERR_NULL;
  if (table_stride < 1 || recent < 0 || recent > budget) return GGUF_QK_ERR_SHAPE;
  EvictPlan p;
  st = evict_plan(a.c, n_seqs, max_len, budget, &p);
  if (st) return st;
  if (abi_mul(abi_mul(n_seqs, table_stride), 4) < 0) return GGUF_QK_ERR_SHAPE;
  if (!abi_aligned(page_table, 4) || !abi_aligned(lengths, 4) || !abi_aligned(workspace, 16))
    return GGUF_QK_ERR_ALIGN;
  if (n_seqs == 0) return GGUF_QK_OK;
  if (p.moves > 0 && !workspace) return GGUF_QK_ERR_NULL;
  if (p.moves > 0 && workspace_bytes < p.bytes) return GGUF_QK_ERR_LIMIT;
  const int64_t table_bytes = n_seqs * table_stride * 4, used = p.moves > 0 ? p.bytes : 0;
  if (kv_touches(a.c, lengths, n_seqs * 4) || kv_touches(a.c, page_table, table_bytes) ||
      kv_touches(a.c, workspace, used) || abi_overlap(lengths, n_seqs * 4, page_table, table_bytes) ||
      abi_overlap(workspace, used, lengths, n_seqs * 4) || abi_overlap(workspace, used, page_table, table_bytes))
    return GGUF_QK_ERR_ALIAS;
  st = abi_device();
  if (st) return st;
  a.table = page_table;
  a.lengths = lengths;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.count = reinterpret_cast<int32_t*>(w);
  a.src = reinterpret_cast<int32_t*>(w + p.count_bytes);
  a.dst = reinterpret_cast<int32_t*>(w + p.count_bytes + p.list_bytes);
  a.table_stride = table_stride;
  a.max_len = max_len;
  a.budget = budget;
  a.recent = recent;
  a.max_moves = p.moves;
  const dim3 block(kEvictThreads), grid((unsigned)a.c.hkv, (unsigned)n_seqs);
  if (p.moves > 0) {
    const int64_t per = ((max_len + kEvictThreads - 1) / kEvictThreads + 3) / 4 * 4;   // slots per thread
    if (per <= 4) hipLaunchKernelGGL(kv_evict_select_kernel<4>, grid, block, 0, stream, a);
    else if (per <= 8) hipLaunchKernelGGL(kv_evict_select_kernel<8>, grid, block, 0, stream, a);
    else if (per <= 16) hipLaunchKernelGGL(kv_evict_select_kernel<16>, grid, block, 0, stream, a);
    else if (per <= 32) hipLaunchKernelGGL(kv_evict_select_kernel<32>, grid, block, 0, stream, a);
    else hipLaunchKernelGGL(kv_evict_select_kernel<0>, grid, block, 0, stream, a);
    st = abi_launched();
    if (st) return st;
  }
  // heads fastest, tiles slowest: tiles past a sequence's moves are empty, and
  // consecutive blocks go to different XCDs
  int64_t tiles = p.moves > 0 ? (p.moves + kMoveTile - 1) / kMoveTile : 1;
  if (tiles > 1024) tiles = 1024;   // blocks step over the rest
  by_cache(kind_of(cache->type), a.c.dim,
           LaunchMove{a, dim3(p.moves > 0 ? (unsigned)a.c.hkv : 1u, (unsigned)n_seqs, (unsigned)tiles), stream});
  return abi_launched();
}

}  // extern "C"
