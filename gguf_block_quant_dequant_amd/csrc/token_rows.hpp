// Which rows of q belong to which sequence, and which slots they see
// (gguf_attn_extend in include/gguf_tokens.h). Plain C++ for host and device but
// for the searches, so that the ranges are tested on the CPU.
#pragma once

#include <stdint.h>

#include "kv_layout.hpp"

namespace gqk {

// Rows of sequence s: of row_start's entries the part within 0 .. n_rows.
struct SeqRows {
  int32_t row0, rows;
};
GQK_HD SeqRows seq_rows(const int32_t* row_start, int32_t s, int64_t n_rows) {
  if (!row_start) return {s, 1};
  int64_t a = row_start[s], b = row_start[s + 1];
  a = a < 0 ? 0 : a > n_rows ? n_rows : a;
  b = b < 0 ? 0 : b > n_rows ? n_rows : b;
  return {(int32_t)a, (int32_t)(b > a ? b - a : 0)};
}

// What the row `j` of `rows` sees of `held` slots: those below hi that are at
// least lo, or below the call's sinks.
struct SlotRange {
  int32_t lo, hi;
};
GQK_HD SlotRange slot_range(int32_t held, int32_t rows, int32_t j, int64_t window) {
  const int64_t p = (int64_t)held - rows + j;
  const int64_t lo = window > 0 && window <= p ? p - window + 1 : 0;
  return {(int32_t)lo, (int32_t)(p < 0 ? 0 : p + 1)};
}

// The lowest n bits (n of any size).
GQK_HD uint32_t low_bits(int64_t n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
// Bits of the slots at .. at + 31 that a row sees.
GQK_HD uint32_t slot_bits(const SlotRange& r, int32_t sinks, int32_t at) {
  return low_bits((int64_t)r.hi - at) & (~low_bits((int64_t)r.lo - at) | low_bits((int64_t)sinks - at));
}

// Slots that a tile of columns (row, query head) reads: [0, pad) and from
// pad + gap on to n + gap; gap and pad are multiples of `unit` (a power of two).
// Every column sees [far, full); none sees [sinks, near).
struct TileRange {
  int32_t n, pad, gap, near, far, full;
};
GQK_HD TileRange tile_range(int32_t held, int32_t rows, int32_t group, int32_t tile, int32_t columns,
                            int64_t window, int32_t sinks, int32_t unit) {
  const int64_t c0 = (int64_t)tile * columns, all = (int64_t)rows * group;
  const int64_t c1 = c0 + columns < all ? c0 + columns : all;
  const SlotRange a = slot_range(held, rows, (int32_t)(c0 / group), window);
  const SlotRange b = slot_range(held, rows, (int32_t)((c1 - 1) / group), window);
  TileRange r;
  const int64_t pad = ((int64_t)sinks + unit - 1) / unit * unit;
  const int64_t base = a.lo / unit * unit;
  r.gap = base > pad ? (int32_t)(base - pad) : 0;
  r.pad = (int32_t)(pad < base ? pad : base);
  r.n = b.hi - r.gap;
  r.near = a.lo;
  r.far = b.lo;
  r.full = a.hi;
  return r;
}

// The sequence that holds row `row` (seq -1: none), of ascending row_start.
struct SeqOf {
  int32_t seq;
  SeqRows rows;
};
GQK_HD SeqOf seq_of_row(const int32_t* row_start, int32_t n_seqs, int64_t n_rows, int64_t row) {
  if (!row_start) return {(int32_t)row, {(int32_t)row, 1}};
  int32_t lo = 0, hi = n_seqs;   // the last of 0 .. n_seqs - 1 that starts at or before the row
  while (hi - lo > 1) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (row_start[mid] <= row) lo = mid;
    else hi = mid;
  }
  const SeqRows r = seq_rows(row_start, lo, n_rows);
  return row >= r.row0 && row < (int64_t)r.row0 + r.rows ? SeqOf{lo, r} : SeqOf{-1, {0, 0}};
}

#if defined(__HIP__)
// Tile `target` of the tiles of `columns` (row, query head) pairs that all
// sequences' rows make, in order; seq -1 behind the last. All 64 lanes of a wave
// call it.
struct RowTile {
  int32_t seq, tile, row0, rows;
};
__device__ __forceinline__ RowTile find_row_tile(const int32_t* row_start, int32_t n_seqs, int64_t n_rows,
                                                 int32_t group, int32_t columns, int32_t target, int lane) {
  int64_t before = 0;   // tiles of the sequences before s0
  for (int s0 = 0; s0 < n_seqs; s0 += 64) {
    SeqRows r = {0, 0};
    if (s0 + lane < n_seqs) r = seq_rows(row_start, s0 + lane, n_rows);
    const int64_t own = ((int64_t)r.rows * group + columns - 1) / columns;
    int64_t upto = own;   // inclusive sum over the lanes
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t o = __shfl_up((long long)upto, d);
      if (lane >= d) upto += o;
    }
    const uint64_t past = __ballot(before + upto > target);
    if (past) {
      const int l = __builtin_ctzll(past);
      RowTile t;
      t.seq = s0 + l;
      t.tile = (int32_t)(target - before - __shfl((long long)(upto - own), l));
      t.row0 = __shfl(r.row0, l);
      t.rows = __shfl(r.rows, l);
      t.seq = __builtin_amdgcn_readfirstlane(t.seq);
      t.tile = __builtin_amdgcn_readfirstlane(t.tile);
      t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
      t.rows = __builtin_amdgcn_readfirstlane(t.rows);
      return t;
    }
    before += __shfl((long long)upto, 63);
  }
  return {-1, 0, 0, 0};
}

// The sequence that holds row `row` (seq -1: none). All 64 lanes of a wave call it.
__device__ __forceinline__ RowTile find_row(const int32_t* row_start, int32_t n_seqs, int64_t n_rows, int64_t row,
                                            int lane) {
  if (!row_start) return {(int32_t)row, 0, (int32_t)row, 1};
  for (int s0 = 0; s0 < n_seqs; s0 += 64) {
    SeqRows r = {0, 0};
    if (s0 + lane < n_seqs) r = seq_rows(row_start, s0 + lane, n_rows);
    const uint64_t in = __ballot(row >= r.row0 && row < (int64_t)r.row0 + r.rows);
    if (in) {
      const int l = __builtin_ctzll(in);
      return {s0 + l, 0, __builtin_amdgcn_readlane(r.row0, l), __builtin_amdgcn_readlane(r.rows, l)};
    }
  }
  return {-1, 0, 0, 0};
}
#endif

}  // namespace gqk
