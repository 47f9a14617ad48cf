// Where a slot of the paged key-value cache lies (the layout of gguf_kv_cache
// in include/gguf_kv.h): offsets, page lookups and their bounds. Plain C++ for
// host and device, so that the bounds are tested on the CPU.
#pragma once

#include <stdint.h>

#if defined(__HIP__)
#define GQK_HD __host__ __device__ __forceinline__
#else
#define GQK_HD inline
#endif

namespace gqk {

// The cache as the kernels take it (by value).
struct KvView {
  uint8_t* k;
  uint8_t* v;
  float* weight;
  int32_t* pos;
  int64_t n_pages;
  int64_t head_bytes;   // of one kv head in one page (K, and V)
  int32_t hkv, dim, ps, shift;   // ps = 1 << shift
};

// Bytes of one kv head of one page: 2 per value, or for Q8_0 a code byte per
// value and an fp16 scale per 32 of them. A multiple of 16 for every
// page size and head dim the library takes.
GQK_HD int64_t kv_head_bytes(bool q8, int64_t dim, int64_t ps) {
  return q8 ? ps * dim + ps * dim / 32 * 2 : ps * dim * 2;
}

// The page id at entry `lp` of a table row, or -1: outside the row, or an id
// outside the cache.
GQK_HD int32_t kv_page(const int32_t* row, int64_t lp, int64_t stride, int64_t n_pages) {
  if (lp < 0 || lp >= stride) return -1;
  const int32_t id = row[lp];
  return id >= 0 && (int64_t)id < n_pages ? id : -1;
}

// Byte offset of kv head h of page `page` in K or V.
GQK_HD int64_t kv_head_at(const KvView& c, int32_t page, int32_t h) {
  return ((int64_t)page * c.hkv + h) * c.head_bytes;
}
// Index of a slot in weight and pos.
GQK_HD int64_t kv_slot_at(const KvView& c, int32_t page, int32_t h, int32_t slot) {
  return (((int64_t)page * c.hkv + h) << c.shift) + slot;
}

// Slots of a sequence that a call looks at: its length cut to the call's
// bound and to the table's row.
GQK_HD int64_t kv_length(int32_t length, int64_t max_len, int64_t stride, int32_t shift) {
  int64_t n = length;
  if (n > max_len) n = max_len;
  if (stride <= (INT64_MAX >> shift) && n > (stride << shift)) n = stride << shift;
  return n < 0 ? 0 : n;
}

}  // namespace gqk
