// Entry points of the attention over the paged cache (include/gguf_kv.h):
// checks, the split over the cache's length, launches; and the join kernels.
#include "abi_check.hpp"
#include "attn_launch.hpp"

namespace gqk {

constexpr int64_t kAttnMaxLen = int64_t(1) << 25;   // splits of at least 1024 positions lie along a grid axis of 65535
// Blocks a call aims for, and the longest chunk of positions. Long chunks spare
// prologues, short ones even out sequences of different lengths. A Q8_0 block's
// prologue weighs more (its steps read half the bytes): 512 blocks and 2048
// positions took 62 us against 66 with 1024 (8 sequences of 20001 .. 32768);
// 16-bit types 200 us with 1024 positions against 215 with 2048 (32 sequences of
// 1 .. 16384) and 67 us with 2048 blocks against 72 with 1024 (64 of 0 .. 4096);
// at head dim 256 half the blocks (143 us against 158 for 0.62 GB). Q8_0's two
// values come from 4 heads of 128 alone; other head dims run at 3.4 .. 4.4 TB/s with them.
constexpr int64_t kAttnBlocks = 2048, kAttnBlocksQ80 = 512;
constexpr int64_t kAttnChunk = 1024, kAttnChunkQ80 = 2048;

// How a call is cut and what its workspace holds.
struct AttnPlan {
  int32_t group, head_tiles, splits, chunk;
  int64_t span, score_stride, most_partials;
  int64_t ml_bytes, o_bytes, bytes;
  float share;
};

static int attn_plan(const KvView& c, int64_t n_seqs, int64_t n_heads, int64_t max_len, int64_t window, bool track,
                     AttnPlan* p) {
  if (n_seqs < 0 || n_heads < 1 || n_heads % c.hkv || max_len < 0 || window < 0) return GGUF_QK_ERR_SHAPE;
  if (n_seqs > 65535 || n_heads > 65535 || max_len > kAttnMaxLen) return GGUF_QK_ERR_LIMIT;
  p->group = (int32_t)(n_heads / c.hkv);
  p->head_tiles = (p->group + 15) / 16;
  // positions a sequence can cover, from a tile's start
  p->span = window > 0 && window < max_len - (kAttnTile - 1) ? window + kAttnTile - 1 : max_len;
  if (p->span < 1) p->span = 1;
  // Chunks of whole tiles; at least 256 positions, at most 64
  // pages (their ids lie one per lane).
  const int64_t round = kAttnTile * kAttnWaves;
  const bool q8 = c.head_bytes != kv_head_bytes(false, c.dim, c.ps);
  int64_t most = int64_t(64) << c.shift;
  if (most > (q8 ? kAttnChunkQ80 : kAttnChunk)) most = q8 ? kAttnChunkQ80 : kAttnChunk;
  const int64_t cells = n_seqs * c.hkv * p->head_tiles;
  const int64_t blocks = q8 ? kAttnBlocksQ80 : c.dim > 128 ? kAttnBlocks / 2 : kAttnBlocks;
  int64_t want = cells > 0 ? blocks / cells : 1;   // splits
  if (want < 1) want = 1;
  int64_t chunk = ((p->span + want - 1) / want + round - 1) / round * round;
  if (chunk < kAttnLeast) chunk = kAttnLeast;
  // short sequences in one launch: the join costs more than the longer chunk
  // (300 positions, in a graph: 8.7 us against 10.7; 512: 10.1 against 10.7)
  if (p->span <= 4 * round) chunk = 4 * round;
  if (chunk > most) chunk = most;
  p->chunk = (int32_t)chunk;
  p->splits = (int32_t)((p->span + chunk - 1) / chunk);   // <= 2^25 / 1024 past the first 1024 blocks
  // A bound above the lengths leaves few long chunks: those longer than the
  // shortest are cut on the device to the lengths there are (up to 64 sequences,
  // one per lane). 4 sequences of 3000 under a bound of
  // 131072, F16: 13.8 us, 22.7 with the host's chunks; Q8_0: 14.3, 33.4. The empty
  // blocks stay: 64 of 1000, 36 us under 1000 and 61 under 131072.
  const int64_t fill = (q8 ? blocks : blocks / 2) - cells;
  p->share = p->splits > 1 && chunk > kAttnLeast && n_seqs <= 64 && fill > blocks / 8
                 ? (float)((double)(c.hkv * p->head_tiles) / (double)fill) : 0.f;
  // Partial results (rows times splits) of the largest call with at most these
  // sequences, this bound and any window: a plan's splits are at most `want`
  // (rows * want <= n_heads * blocks / (hkv * head_tiles)) or, with the longest
  // chunks, span / most, and never more than the shortest chunks give. 0 where no
  // such call is split. It grows with n_seqs and max_len.
  const int64_t rows = n_seqs * n_heads, least = (p->span + kAttnLeast - 1) / kAttnLeast;
  p->most_partials = n_heads * blocks / (c.hkv * p->head_tiles);
  if (p->most_partials < rows * ((p->span + most - 1) / most)) p->most_partials = rows * ((p->span + most - 1) / most);
  if (p->most_partials > rows * least) p->most_partials = rows * least;
  if (least == 1) p->most_partials = 0;
  p->score_stride = track ? (max_len + kAttnTile - 1) / kAttnTile * kAttnTile : 0;
  return GGUF_QK_OK;
}

// Sets the workspace's parts for `partials` partial results (0: one split); -1
// where they do not fit.
static int64_t attn_bytes(const KvView& c, int64_t n_seqs, int64_t n_heads, int64_t partials, bool track, AttnPlan* p) {
  const int64_t rows = n_seqs * n_heads;
  p->ml_bytes = abi_mul(partials > 0 ? partials : track ? rows : 0, 8);
  p->o_bytes = abi_mul(partials, c.dim * 4);
  const int64_t score_bytes = track ? abi_mul(rows, p->score_stride * 4) : 0;
  if (p->ml_bytes < 0 || p->o_bytes < 0 || score_bytes < 0) return -1;
  p->ml_bytes = (p->ml_bytes + 15) / 16 * 16;
  return p->bytes = p->ml_bytes + p->o_bytes + score_bytes;
}

template <int DIM>
static void launch_join(const AttnArgs& a, int joins, int tiles, dim3 grid, hipStream_t stream) {
  hipLaunchKernelGGL(attn_join_kernel<DIM>, grid, dim3(kJoinThreads), 0, stream, a, joins, tiles);
}

}  // namespace gqk

using namespace gqk;

extern "C" {

int64_t gguf_attn_decode_workspace(const gguf_kv_cache* cache, int64_t n_seqs, int64_t n_heads,
                                   int64_t max_len, int32_t track) {
  KvView c;
  int st = kv_view(cache, &c);
  if (st) return st;
  AttnPlan p;
  st = attn_plan(c, n_seqs, n_heads, max_len, 0, track != 0, &p);
  if (st) return st;
  const int64_t b = attn_bytes(c, n_seqs, n_heads, p.most_partials, track != 0, &p);
  return b < 0 ? GGUF_QK_ERR_LIMIT : b;
}

int gguf_attn_decode(const gguf_kv_cache* cache, const float* q, int64_t q_stride, float* out,
                     int64_t out_stride, int64_t n_seqs, int64_t n_heads, const int32_t* page_table,
                     int64_t table_stride, const int32_t* lengths, int64_t max_len, float scale,
                     int64_t window, int32_t track, void* workspace, int64_t workspace_bytes,
                     hipStream_t stream) {
  AttnArgs a;
  int st = kv_view(cache, &a.c);
  if (st) return st;
  if (!q || !out || !page_table || !lengths || (track && !a.c.weight)) return GGUF_QK_ERR_NULL;
  AttnPlan p;
  st = attn_plan(a.c, n_seqs, n_heads, max_len, window, track != 0, &p);
  if (st) return st;
  const int64_t partials = p.splits > 1 ? n_seqs * n_heads * p.splits : 0;
  if (attn_bytes(a.c, n_seqs, n_heads, partials, track != 0, &p) < 0) return GGUF_QK_ERR_LIMIT;
  const int64_t row = n_heads * a.c.dim;
  const float qscale = scale * 1.44269504088896340736f;   // infinite past |scale| = 2.358e38
  if (table_stride < 1 || q_stride < row || out_stride < row || !(qscale - qscale == 0.f)) return GGUF_QK_ERR_SHAPE;
  if (abi_mul(abi_mul(n_seqs, q_stride), 4) < 0 || abi_mul(abi_mul(n_seqs, out_stride), 4) < 0 ||
      abi_mul(abi_mul(n_seqs, table_stride), 4) < 0)
    return GGUF_QK_ERR_SHAPE;
  if (!abi_aligned(q, 16) || !abi_aligned(out, 16) || q_stride % 4 || out_stride % 4 || !abi_aligned(page_table, 4) ||
      !abi_aligned(lengths, 4) || !abi_aligned(workspace, 16))
    return GGUF_QK_ERR_ALIGN;
  if (n_seqs == 0) return GGUF_QK_OK;
  if (p.bytes > 0 && !workspace) return GGUF_QK_ERR_NULL;
  if (workspace_bytes < p.bytes) return GGUF_QK_ERR_LIMIT;
  const int64_t qb = ((n_seqs - 1) * q_stride + row) * 4, ob = ((n_seqs - 1) * out_stride + row) * 4;
  const int64_t tb = n_seqs * table_stride * 4, lb = n_seqs * 4;
  const void* w = p.bytes > 0 ? workspace : nullptr;
  if (abi_overlap(out, ob, q, qb) || abi_overlap(out, ob, page_table, tb) || abi_overlap(out, ob, lengths, lb) ||
      kv_touches(a.c, out, ob) || abi_overlap(w, p.bytes, out, ob) || abi_overlap(w, p.bytes, q, qb) ||
      abi_overlap(w, p.bytes, page_table, tb) || abi_overlap(w, p.bytes, lengths, lb) || kv_touches(a.c, w, p.bytes))
    return GGUF_QK_ERR_ALIAS;
  if (track) {
    const int64_t wb = kv_plane_bytes(a.c);
    if (abi_overlap(a.c.weight, wb, q, qb) || abi_overlap(a.c.weight, wb, page_table, tb) ||
        abi_overlap(a.c.weight, wb, lengths, lb))
      return GGUF_QK_ERR_ALIAS;
  }
  st = abi_device();
  if (st) return st;
  const int64_t tiles = (p.span + kWeightTile - 1) / kWeightTile;
  const int64_t weight_blocks = track ? tiles * a.c.hkv : 0;
  const int64_t joins = p.splits > 1 ? n_heads : 0;
  if (joins + weight_blocks > INT32_MAX / kJoinThreads) return GGUF_QK_ERR_LIMIT;   // threads of a grid axis
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.table = page_table;
  a.lengths = lengths;
  a.q = q;
  a.out = out;
  a.part_ml = reinterpret_cast<float*>(ws);
  a.part_o = reinterpret_cast<float*>(ws + p.ml_bytes);
  a.scores = reinterpret_cast<float*>(ws + p.ml_bytes + p.o_bytes);
  a.table_stride = table_stride;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.max_len = max_len;
  a.window = window;
  a.score_stride = p.score_stride;
  a.n_heads = (int32_t)n_heads;
  a.group = p.group;
  a.head_tiles = p.head_tiles;
  a.splits = p.splits;
  a.chunk = p.chunk;
  a.chunk_pages = (p.chunk + a.c.ps - 1) / a.c.ps + 1 < 64 ? (p.chunk + a.c.ps - 1) / a.c.ps + 1 : 64;
  a.qscale = qscale;
  a.n_seqs = (int32_t)n_seqs;
  a.share = p.share;
  const dim3 grid((unsigned)(a.c.hkv * p.head_tiles), (unsigned)n_seqs, (unsigned)p.splits);
  if (cache->type == GGUF_KV_TYPE_F16) launch_attn_f16(a, track != 0, grid, stream);
  else if (cache->type == GGUF_KV_TYPE_BF16) launch_attn_bf16(a, track != 0, grid, stream);
  else launch_attn_q8_0(a, track != 0, grid, stream);
  st = abi_launched();
  if (st || joins + weight_blocks == 0) return st;
  const dim3 jgrid((unsigned)(joins + weight_blocks), (unsigned)n_seqs);
  switch (a.c.dim) {
    case 64: launch_join<64>(a, (int)joins, (int)tiles, jgrid, stream); break;
    case 96: launch_join<96>(a, (int)joins, (int)tiles, jgrid, stream); break;
    case 128: launch_join<128>(a, (int)joins, (int)tiles, jgrid, stream); break;
    case 192: launch_join<192>(a, (int)joins, (int)tiles, jgrid, stream); break;
    default: launch_join<256>(a, (int)joins, (int)tiles, jgrid, stream); break;
  }
  return abi_launched();
}

}  // extern "C"
