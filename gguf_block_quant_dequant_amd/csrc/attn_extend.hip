// Entry points of the attention of several new tokens per sequence
// (include/gguf_tokens.h): checks, the split over the positions, launches.
#include "../../include/gguf_tokens.h"
#include "abi_check.hpp"
#include "attn_launch.hpp"
#include "attn_prompt_launch.hpp"

namespace gqk {

constexpr int64_t kExtendMaxLen = int64_t(1) << 25;
// Blocks a call of the few-rows kernel aims for (8 sequences of 3 to 5 rows behind 5000 to
// 8187 slots, F16: 40 us with 512, 34.5 with 1024, 42 with 2048; the same of 5 behind 8000,
// BF16: 53, 54, 68).
constexpr int64_t kExtendBlocks = 1024;
constexpr int64_t kExtendChunk = 1024;    // longest chunk of positions of the few-rows kernel: 64 pages of 16
constexpr int64_t kExtendOnce = 4 * kAttnTile * kAttnWaves;   // positions that it does not split
constexpr int kFewColumns = 16;           // columns of its tiles
constexpr int64_t kTwoTileReads = 65536;  // slots of all sequences
constexpr int64_t kPromptBlocks = 256;    // blocks that run at once: one per CU, or two of one group of waves to head dim 128
// Blocks from which one group of waves each, two blocks at a time, does better: 8 prompts
// to 4096 (4680 blocks) 560 us against 685; one of 4096 (512) 110 against 104.
constexpr int64_t kPromptSingle = 1024;
// Shortest chunk of the prompt kernel, per group of waves: a block's start and end take as
// long as four to five steps of 64 slots (Q8_0, one sequence of 16 rows behind 8000 slots: 32
// us with 512, 22 with 256, 21 with 128; 64 rows behind 30000: 52, 54, 53. BF16, two groups,
// a prompt of 1024: 32 with 256 in all, 28 with 512; 512 rows behind 2000: 32, and 34 with
// 1024).
constexpr int64_t kPromptLeast = 256;

struct ExtendPlan {
  bool prompt;                // the kernel for many rows
  int32_t group, splits, chunk, unit, columns, groups, fill, least;
  int64_t tiles;              // tiles of columns, at most
  int64_t ml_bytes, bytes;    // where the partial outputs lie; the workspace named
};

// (row, query head) pairs per sequence up to which BF16 queries stay with the kernel for few
// rows (see extend_plan).
static int64_t few_pairs(const KvView& c, bool q8) {
  return q8 || c.dim < 96 ? 2 * kFewColumns : kFewColumns;
}

// Positions that the columns of a tile read, at most: the first slots, the window and the
// tile's rows, in whole units.
static int64_t tile_span(int64_t max_len, int64_t window, int64_t sinks, int64_t columns, int64_t group, int64_t unit) {
  int64_t span = max_len;
  if (window > 0 && window < max_len) {
    const int64_t pad = (sinks + unit - 1) / unit * unit;
    const int64_t seen = pad + window + (columns - 1) / group + 1 + unit;
    if (seen < span) span = seen;
  }
  return span < 1 ? 1 : span;
}

// Blocks that a call of the kernel for many rows aims for.
static int64_t prompt_blocks(int groups, int dim) {
  return groups == 2 || dim > 128 ? kPromptBlocks : 2 * kPromptBlocks;
}

// Partial results (rows times query heads times splits) of the largest call with at most
// these sequences and rows and this bound; 0 where no such call is split. Splits are at most
// the blocks aimed for over the cells (tiles times kv heads), so that rows * n_heads * splits <=
// columns * blocks; with the longest chunks of the few-rows kernel they are span / longest; and
// never more than the shortest chunks give. (rows * group <= columns * tiles.) Each of these
// grows with the sequences, the rows and the bound.
static int64_t most_partials(const KvView& c, int32_t type, bool q8, int64_t group, int64_t n_seqs, int64_t n_rows,
                             int64_t n_heads, int64_t max_len, int64_t window, int64_t sinks) {
  if (n_seqs == 0 || n_rows == 0) return 0;
  const bool bf16 = type == GGUF_KV_TYPE_BF16;
  const int64_t few = few_pairs(c, q8);
  const int64_t fewest = bf16 && few * n_seqs / group < n_rows ? few * n_seqs / group : n_rows;   // of the few-rows kernel
  const int columns = attn_most_columns(q8);
  int64_t most = 0;
  int64_t span = tile_span(max_len, window, sinks, columns, group, c.ps > kAttnTile ? c.ps : kAttnTile);
  if (span > kExtendOnce) {
    const int64_t rows = fewest * n_heads, least = rows * ((span + kAttnLeast - 1) / kAttnLeast);
    const int64_t longest = rows * ((span + kExtendChunk - 1) / kExtendChunk);
    most = columns * kExtendBlocks;
    if (most < longest) most = longest;
    if (most > least) most = least;
  }
  if (bf16 && n_rows * group > few) {
    span = tile_span(max_len, window, sinks, kPromptColumns, group, c.ps > kPromptSlots ? c.ps : kPromptSlots);
    const int groups = prompt_groups(q8, c.dim);   // where positions are split
    const int64_t shortest = kPromptLeast * groups;
    if (span > shortest) {
      int64_t partials = kPromptColumns * prompt_blocks(groups, c.dim);
      const int64_t least = n_rows * n_heads * ((span + shortest - 1) / shortest);
      if (partials > least) partials = least;
      if (most < partials) most = partials;
    }
  }
  return most;
}

static int extend_plan(const KvView& c, int32_t type, int64_t n_seqs, int64_t n_rows, int64_t n_heads, int64_t max_len,
                       int64_t window, int64_t sinks, ExtendPlan* p) {
  if ((type != GGUF_KV_TYPE_F32 && type != GGUF_KV_TYPE_BF16) || n_seqs < 0 || n_rows < 0 || n_heads < 1 ||
      n_heads % c.hkv || max_len < 0 || window < 0 || sinks < 0)
    return GGUF_QK_ERR_SHAPE;
  if (n_seqs > (1 << 20) || n_rows > (int64_t(1) << 23) || n_heads > 65535 || max_len > kExtendMaxLen ||
      sinks > kExtendMaxLen)
    return GGUF_QK_ERR_LIMIT;
  p->group = (int32_t)(n_heads / c.hkv);
  if (n_rows * p->group > INT32_MAX / 2) return GGUF_QK_ERR_LIMIT;
  // The kernel for many rows, whose tiles go straight to LDS, where a sequence's rows fill
  // more than a tile of 16 columns of the one for few; from head dim 96 on (64 sequences of 5
  // rows of 4 heads behind 1000 slots, BF16, 128: 62 us with the few-rows kernel, 32 with the
  // other; 192: 72, 44; 8 behind 8000: 55, 40; one behind 8000: 18, 21). More than two tiles at
  // head dim 64 (8 behind 8000, 8 kv heads: 46, 51; one: 14, 19) and for Q8_0 (64 behind 1000,
  // 128: 33, 49; one behind 8000: 16, 22), which it converts for all its columns.
  const bool q8 = c.head_bytes != kv_head_bytes(false, c.dim, c.ps);
  p->prompt = type == GGUF_KV_TYPE_BF16 && n_rows * p->group > few_pairs(c, q8) * n_seqs;
  // Two tiles of columns where a sequence has more than one on average (F16, 5 rows of 4 heads
  // of 128 behind 8000 slots: 8 sequences 54 us with one, which reads K and V twice, 45 with
  // two; 16 x 8 93 and 73). Past head dim 128 one wave per SIMD is left and one tile has twice
  // the blocks: two where the reads outweigh that (256, 64 sequences behind 4000 slots: 205,
  // 150; 16 x 8 behind 8000: 115, 105; 8 x 5 behind 8000: 69, 74; one: 22, 26).
  const int64_t reads = n_seqs * (window > 0 && window < max_len ? window : max_len);
  const bool two = n_rows * p->group > kFewColumns * n_seqs && (c.dim <= 128 || reads > kTwoTileReads);
  p->columns = p->prompt ? kPromptColumns : two ? attn_most_columns(q8) : kFewColumns;
  const int tile = p->prompt ? kPromptSlots : kAttnTile;
  p->unit = c.ps > tile ? c.ps : tile;
  p->tiles = (n_rows * p->group + n_seqs * (p->columns - 1)) / p->columns;
  if (p->tiles > 65535) return GGUF_QK_ERR_LIMIT;   // along a grid axis
  const int64_t span = tile_span(max_len, window, sinks, p->columns, p->group, p->unit);
  const int64_t cells = p->tiles * c.hkv;
  int64_t chunk;
  if (p->prompt) {
    p->groups = cells < kPromptSingle ? prompt_groups(q8, c.dim) : 1;
    const int64_t blocks = prompt_blocks(p->groups, c.dim);
    const int64_t want = cells > 0 && cells < blocks ? blocks / cells : 1;
    chunk = ((span + want - 1) / want + 63) / 64 * 64;
    p->least = (int32_t)kPromptLeast * p->groups;
    if (chunk < p->least) chunk = p->least;
    p->fill = (int32_t)blocks;
  } else {
    const int64_t round = kAttnTile * kAttnWaves;
    int64_t want = cells > 0 ? kExtendBlocks / cells : 1;
    if (want < 1) want = 1;
    chunk = ((span + want - 1) / want + round - 1) / round * round;
    if (chunk < kAttnLeast) chunk = kAttnLeast;
    if (span <= kExtendOnce) chunk = kExtendOnce;
    if (chunk > kExtendChunk) chunk = kExtendChunk;
    p->fill = p->least = 0;
  }
  p->chunk = (int32_t)chunk;
  p->splits = (int32_t)((span + chunk - 1) / chunk);
  // Under a bound above the lengths, the prompt kernel's chunks are cut to the lengths on
  // the device: 256 rows behind 8000 slots under a bound of 131072, 166 us with the host's
  // chunks, 41 so. (The kernel for few rows holds the page ids of 64 pages, so that its chunks
  // cannot grow with the lengths; cut to them, 8 x 5 rows behind 3000 slots under 131072 took
  // 67 us and 43 without, 30 since empty blocks end early.)
  if (p->splits == 1 || chunk <= p->least || n_seqs > 64) p->fill = 0;
  // (rows times heads below 2^39, splits at most 2^17)
  const int64_t partials = most_partials(c, type, q8, p->group, n_seqs, n_rows, n_heads, max_len, window, sinks);
  if (abi_mul(partials, c.dim * 4 + 16) < 0) return GGUF_QK_ERR_LIMIT;
  p->bytes = (partials * 8 + 15) / 16 * 16 + partials * c.dim * 4;
  p->ml_bytes = p->splits > 1 ? (n_rows * n_heads * p->splits * 8 + 15) / 16 * 16 : 0;
  return GGUF_QK_OK;
}

template <int DIM>
static void launch_join_rows(const AttnRowsArgs& a, hipStream_t stream) {
  constexpr int kItems = kJoinThreads / (DIM / 4);
  const int64_t items = a.n_rows * a.n_heads, blocks = (items + kItems - 1) / kItems;
  if (a.splits <= kJoinFew && blocks <= INT32_MAX / kJoinThreads)
    hipLaunchKernelGGL(attn_join_few_kernel<DIM>, dim3((unsigned)blocks), dim3(kJoinThreads), 0, stream, a);
  else   // rows <= 2^23: threads of a grid axis
    hipLaunchKernelGGL(attn_join_rows_kernel<DIM>, dim3((unsigned)a.n_rows, (unsigned)a.n_heads), dim3(kJoinThreads), 0,
                       stream, a);
}

}  // namespace gqk

using namespace gqk;

extern "C" {

int64_t gguf_attn_extend_workspace(const gguf_kv_cache* cache, int32_t type, int64_t n_seqs, int64_t n_rows,
                                   int64_t n_heads, int64_t max_len, int64_t window, int64_t sinks) {
  KvView c;
  int st = kv_view(cache, &c);
  if (st) return st;
  ExtendPlan p;
  st = extend_plan(c, type, n_seqs, n_rows, n_heads, max_len, window, sinks, &p);
  return st ? st : p.bytes;
}

int gguf_attn_extend(const gguf_kv_cache* cache, const void* q, int32_t type, int64_t q_stride, void* out,
                     int64_t out_stride, const int32_t* row_start, int64_t n_rows, int64_t n_seqs, int64_t n_heads,
                     const int32_t* page_table, int64_t table_stride, const int32_t* lengths, int64_t max_len,
                     float scale, int64_t window, int64_t sinks, void* workspace, int64_t workspace_bytes,
                     hipStream_t stream) {
  AttnPromptArgs a;
  int st = kv_view(cache, &a.c);
  if (st) return st;
  if (!q || !out || !page_table || !lengths) return GGUF_QK_ERR_NULL;
  ExtendPlan p;
  st = extend_plan(a.c, type, n_seqs, n_rows, n_heads, max_len, window, sinks, &p);
  if (st) return st;
  const int64_t row = n_heads * a.c.dim, es = type == GGUF_KV_TYPE_F32 ? 4 : 2;
  const float qscale = scale * 1.44269504088896340736f;
  if (table_stride < 1 || q_stride < row || out_stride < row || !(qscale - qscale == 0.f) ||
      (!row_start && n_rows != n_seqs))
    return GGUF_QK_ERR_SHAPE;
  if (abi_mul(abi_mul(n_rows, q_stride), es) < 0 || abi_mul(abi_mul(n_rows, out_stride), es) < 0 ||
      abi_mul(abi_mul(n_seqs, table_stride), 4) < 0)
    return GGUF_QK_ERR_SHAPE;
  if (!abi_aligned(q, 16) || !abi_aligned(out, 16) || q_stride * es % 16 || out_stride * es % 16 ||
      !abi_aligned(page_table, 4) || !abi_aligned(lengths, 4) || !abi_aligned(row_start, 4) || !abi_aligned(workspace, 16))
    return GGUF_QK_ERR_ALIGN;
  if (n_seqs == 0 || n_rows == 0) return GGUF_QK_OK;
  if (p.bytes > 0 && !workspace) return GGUF_QK_ERR_NULL;
  if (workspace_bytes < p.bytes) return GGUF_QK_ERR_LIMIT;
  const void* w = p.bytes > 0 ? workspace : nullptr;
  const int64_t ob = ((n_rows - 1) * out_stride + row) * es;
  const void* in[4] = {q, page_table, lengths, row_start};
  const int64_t in_bytes[4] = {((n_rows - 1) * q_stride + row) * es, n_seqs * table_stride * 4, n_seqs * 4,
                               (n_seqs + 1) * 4};
  for (int i = 0; i < 4; ++i)
    if (abi_overlap(out, ob, in[i], in_bytes[i]) || abi_overlap(w, p.bytes, in[i], in_bytes[i]))
      return GGUF_QK_ERR_ALIAS;
  if (kv_touches(a.c, out, ob) || abi_overlap(w, p.bytes, out, ob) || kv_touches(a.c, w, p.bytes))
    return GGUF_QK_ERR_ALIAS;
  st = abi_device();
  if (st) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.table = page_table;
  a.lengths = lengths;
  a.q = static_cast<const float*>(q);
  a.out = static_cast<float*>(out);
  a.part_ml = reinterpret_cast<float*>(ws);
  a.part_o = reinterpret_cast<float*>(ws + p.ml_bytes);
  a.scores = nullptr;
  a.table_stride = table_stride;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.max_len = max_len;
  a.window = window;
  a.score_stride = 0;
  a.n_heads = (int32_t)n_heads;
  a.group = p.group;
  a.head_tiles = 0;
  a.splits = p.splits;
  a.chunk = p.chunk;
  a.chunk_pages = 64;
  a.qscale = qscale;
  a.n_seqs = (int32_t)n_seqs;
  a.share = 0.f;
  a.row_start = row_start;
  a.n_rows = n_rows;
  a.sinks = (int32_t)sinks;
  a.bf16 = type == GGUF_KV_TYPE_BF16;
  a.columns = p.columns;
  a.unit = p.unit;
  a.fill = p.fill;
  a.least = p.least;
  const dim3 grid((unsigned)a.c.hkv, (unsigned)p.tiles, (unsigned)p.splits);
  a.tiles = (int32_t)p.tiles;
  if (p.prompt) {
    if (cache->type == GGUF_KV_TYPE_F16) launch_prompt_f16(a, p.groups, grid, stream);
    else if (cache->type == GGUF_KV_TYPE_BF16) launch_prompt_bf16(a, p.groups, grid, stream);
    else launch_prompt_q8_0(a, p.groups, grid, stream);
  } else if (cache->type == GGUF_KV_TYPE_F16) launch_attn_rows_f16(a, p.columns, grid, stream);
  else if (cache->type == GGUF_KV_TYPE_BF16) launch_attn_rows_bf16(a, p.columns, grid, stream);
  else launch_attn_rows_q8_0(a, p.columns, grid, stream);
  st = abi_launched();
  if (st || p.splits == 1) return st;
  switch (a.c.dim) {
    case 64: launch_join_rows<64>(a, stream); break;
    case 96: launch_join_rows<96>(a, stream); break;
    case 128: launch_join_rows<128>(a, stream); break;
    case 192: launch_join_rows<192>(a, stream); break;
    default: launch_join_rows<256>(a, stream); break;
  }
  return abi_launched();
}

}  // extern "C"
