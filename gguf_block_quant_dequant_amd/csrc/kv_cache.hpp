// Kernels that write the paged key-value cache: append and the moves of an
// eviction, and the eviction's selection.
#pragma once

#include "device_common.hpp"
#include "kv_layout.hpp"
#include "wave_ops.hpp"

namespace gqk {

enum KvKind { kKvF16 = 0, kKvBF16 = 1, kKvQ80 = 2 };

// ------------------------------------------------------------------ append

struct AppendArgs {
  KvView c;
  const void* k;
  const void* v;
  const int32_t* seq;
  const int32_t* slot;
  const int32_t* pos;
  const int32_t* table;
  int64_t row_stride, table_stride, n_tokens, n_seqs;
  int32_t tile;   // tokens per block: 8, 16, 32 or 64
};

constexpr int kAppendThreads = 256;
constexpr int kAppendTile = 64;

// Eight input values from element `i` of a row, as loaded.
template <bool BF16SRC>
struct Raw8 {
  uint4 w[BF16SRC ? 1 : 2];
  __device__ __forceinline__ void load(const void* base, int64_t i) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + i * (BF16SRC ? 2 : 4));
#pragma unroll
    for (int j = 0; j < (BF16SRC ? 1 : 2); ++j) w[j] = p[j];
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    if constexpr (BF16SRC) {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(u[j] << 16);
        x[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        x[4 * j] = __uint_as_float(w[j].x);
        x[4 * j + 1] = __uint_as_float(w[j].y);
        x[4 * j + 2] = __uint_as_float(w[j].z);
        x[4 * j + 3] = __uint_as_float(w[j].w);
      }
    }
  }
};

// Rounds eight values to their cache form: 16-bit patterns, or Q8_0 codes (in
// the low bytes) with the scale of the 32-dim block, whose other values the
// lanes differing in the two low bits of `lane` hold.
template <int KIND>
__device__ __forceinline__ void append_round8(const float (&x)[8], uint16_t (&o)[8], uint16_t* scale) {
  if constexpr (KIND == kKvF16) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = __builtin_bit_cast(uint16_t, (_Float16)x[j]);
  } else if constexpr (KIND == kKvBF16) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = to_bf16(x[j]);
  } else {
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
    amax = fmaxf(amax, __shfl_xor(amax, 1));
    amax = fmaxf(amax, __shfl_xor(amax, 2));
    const _Float16 d16 = (_Float16)(amax / 127.0f);
    const float d = (float)d16;
    *scale = __builtin_bit_cast(uint16_t, d16);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float q = d == 0.f ? 0.f : rintf(x[j] / d);
      o[j] = (uint8_t)(int8_t)(int)fminf(fmaxf(q, -127.f), 127.f);
    }
  }
}

__device__ __forceinline__ uint4 pack8x16(const uint16_t (&o)[8]) {
  return make_uint4(o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16, o[4] | (uint32_t)o[5] << 16,
                    o[6] | (uint32_t)o[7] << 16);
}
__device__ __forceinline__ uint2 pack8x8(const uint16_t (&o)[8]) {
  return make_uint2((o[0] & 255u) | (o[1] & 255u) << 8 | (o[2] & 255u) << 16 | (uint32_t)o[3] << 24,
                    (o[4] & 255u) | (o[5] & 255u) << 8 | (o[6] & 255u) << 16 | (uint32_t)o[7] << 24);
}

// One block: `tile` consecutive tokens of one kv head. K rows go out as they
// are; V goes through LDS to be written along the positions, eight consecutive
// slots per 16-byte store where the tile holds a whole aligned group of them
// (the groups of a dim side by side: 128 bytes of 64 positions), single slots
// elsewhere. Bound by the bytes read and written (8 prompts of 4096 tokens, bf16
// to F16, 4 heads of 128: 38 us for 134 MB, 3.5 TB/s, where HBM writes 83 MB for
// the 67 stored) or by its dependent loads: the token's slot, its page, its row
// (16 tokens: 4.5 us).
template <int KIND, bool BF16SRC, int DIM>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(const AppendArgs a) {
  constexpr int kOct = DIM / 8;             // 8-value groups of a row
  constexpr int kLdsRow = DIM + 2;          // uint16; odd words: a column's reads spread over the banks
  __shared__ __align__(16) uint16_t vt[kAppendTile * kLdsRow];
  __shared__ uint16_t vs[KIND == kKvQ80 ? kAppendTile * (DIM / 32) : 1];
  __shared__ int64_t head_at[kAppendTile];  // byte offset of the token's page and head; -1: dropped
  __shared__ int32_t slot_of[kAppendTile];  // slot within the page
  __shared__ uint8_t leads_at[kAppendTile], single_at[kAppendTile];   // tokens that lead a whole group, single ones
  __shared__ int n_lead, n_single;
  const int h = blockIdx.y, tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * a.tile;
  if (tid < kAppendTile) {   // one wave
    const int64_t t = t0 + tid;
    int64_t at = -1;
    int32_t in_page = 0;
    if (tid < a.tile && t < a.n_tokens) {
      const int64_t s = a.seq ? a.seq[t] : t;
      const int32_t slot = a.slot[t];
      if (s >= 0 && s < a.n_seqs && slot >= 0) {
        const int32_t page = kv_page(a.table + s * a.table_stride, slot >> a.c.shift, a.table_stride, a.c.n_pages);
        in_page = slot & (a.c.ps - 1);
        if (page >= 0) {
          at = kv_head_at(a.c, page, h);
          const int64_t i = kv_slot_at(a.c, page, h, in_page);
          if (a.c.weight) a.c.weight[i] = 0.f;
          if (a.c.pos) a.c.pos[i] = a.pos ? a.pos[t] : slot;
        }
      }
    }
    head_at[tid] = at;
    slot_of[tid] = in_page;
    // whole groups: token tid on a slot that is a multiple of 8, the seven
    // tokens behind it on the seven slots behind it
    bool lead = at >= 0 && (in_page & 7) == 0 && tid + 8 <= kAppendTile;
#pragma unroll
    for (int j = 1; j < 8; ++j) {
      const int64_t at_j = __shfl(at, (tid + j) & 63);
      const int32_t slot_j = __shfl(in_page, (tid + j) & 63);
      lead = lead && at_j == at && slot_j == in_page + j;
    }
    // the same pages named again by an overlapping run of tokens would be two
    // tokens on one slot, which the contract excludes
    bool covered = false;
    const uint64_t leads = __ballot(lead);
#pragma unroll
    for (int j = 1; j < 8; ++j) covered = covered || (tid >= j && (leads >> (tid - j) & 1));
    const bool single = at >= 0 && !lead && !covered;
    const uint64_t singles = __ballot(single), below = (uint64_t(1) << tid) - 1;
    if (lead) leads_at[__popcll((unsigned long long)(leads & below))] = (uint8_t)tid;
    if (single) single_at[__popcll((unsigned long long)(singles & below))] = (uint8_t)tid;
    if (tid == 0) {
      n_lead = __popcll((unsigned long long)leads);
      n_single = __popcll((unsigned long long)singles);
    }
  }
  __syncthreads();
  const int rows = a.tile;
  constexpr int kRowStep = kAppendThreads / kOct;   // rows per pass (threads past the last whole row idle)
  constexpr int kPasses = (kAppendTile + kRowStep - 1) / kRowStep;
  const int oct = tid % kOct, r0 = tid / kOct;
  Raw8<BF16SRC> rk[kPasses], rv[kPasses];
  int64_t at[kPasses];   // all loads in flight before the first is used
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = r0 + i * kRowStep;
    at[i] = r0 < kRowStep && r < rows ? head_at[r] : -1;
    if (at[i] >= 0) {
      const int64_t e = (t0 + r) * a.row_stride + (int64_t)h * DIM + oct * 8;
      rk[i].load(a.k, e);
      rv[i].load(a.v, e);
    }
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    if (at[i] < 0) continue;   // whole rows drop: the lanes of a 32-dim block agree
    const int r = r0 + i * kRowStep;
    float x[8];
    uint16_t o[8], sc = 0;
    rk[i].values(x);
    append_round8<KIND>(x, o, &sc);
    uint8_t* kp = a.c.k + at[i];
    if constexpr (KIND == kKvQ80) {
      *reinterpret_cast<uint2*>(kp + slot_of[r] * DIM + oct * 8) = pack8x8(o);
      if ((oct & 3) == 0)
        reinterpret_cast<uint16_t*>(kp + a.c.ps * DIM)[slot_of[r] * (DIM / 32) + (oct >> 2)] = sc;
    } else {
      *reinterpret_cast<uint4*>(kp + (slot_of[r] * DIM + oct * 8) * 2) = pack8x16(o);
    }
    rv[i].values(x);
    append_round8<KIND>(x, o, &sc);
    uint32_t* dst = reinterpret_cast<uint32_t*>(vt + r * kLdsRow + oct * 8);
    const uint4 w = pack8x16(o);
    dst[0] = w.x; dst[1] = w.y; dst[2] = w.z; dst[3] = w.w;
    if constexpr (KIND == kKvQ80)
      if ((oct & 3) == 0) vs[r * (DIM / 32) + (oct >> 2)] = sc;
  }
  __syncthreads();
  // V, a dim's groups side by side
  const int nl = n_lead, ns = n_single;
  for (int i = tid; i < nl * DIM; i += kAppendThreads) {
    const int d = nl == 8 ? i >> 3 : i / nl, r = leads_at[i - d * nl];
    uint8_t* vp = a.c.v + head_at[r];
    const int to = d * a.c.ps + slot_of[r];
    uint16_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = vt[(r + j) * kLdsRow + d];
    if constexpr (KIND == kKvQ80) *reinterpret_cast<uint2*>(vp + to) = pack8x8(o);
    else *reinterpret_cast<uint4*>(vp + to * 2) = pack8x16(o);
  }
  for (int i = tid; i < ns * DIM; i += kAppendThreads) {
    const int d = i / ns, r = single_at[i - d * ns];
    uint8_t* vp = a.c.v + head_at[r];
    const int to = d * a.c.ps + slot_of[r];
    if constexpr (KIND == kKvQ80) vp[to] = (uint8_t)vt[r * kLdsRow + d];
    else reinterpret_cast<uint16_t*>(vp)[to] = vt[r * kLdsRow + d];
  }
  if constexpr (KIND == kKvQ80) {
    for (int i = tid; i < rows * (DIM / 32); i += kAppendThreads) {
      const int r = i / (DIM / 32), b = i % (DIM / 32);
      if (head_at[r] < 0) continue;
      reinterpret_cast<uint16_t*>(a.c.v + head_at[r] + a.c.ps * DIM)[b * a.c.ps + slot_of[r]] =
          vs[r * (DIM / 32) + b];
    }
  }
}

// ------------------------------------------------------------------ eviction

struct EvictArgs {
  KvView c;
  const int32_t* table;
  int32_t* lengths;
  int32_t* count;     // [n_seqs][hkv] moves
  int32_t* src;       // [n_seqs][hkv][max_moves] slots of the sequence, ascending
  int32_t* dst;       // the same: the vacated slots
  int64_t table_stride, max_len, budget, recent, max_moves;
};

constexpr int kEvictThreads = 1024;
constexpr int kEvictWaves = kEvictThreads / 64;
constexpr int kEvictFew = 2;      // slots past the budget up to which they are picked one by one
constexpr int kHistCopies = 16;   // copies of a digit's histogram, lane & 15: a few shared leading
                                  // digits (weights have few exponents) would queue on one LDS word

// A weight as an unsigned key of the same order; zeros of either sign equal,
// every NaN above the infinities, below the protected slots' key.
constexpr uint32_t kKeyProtected = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t b = __float_as_uint(w + 0.0f);
  const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return w != w ? 0xFFFFFFFEu : k;
}

// Exclusive prefix sum over the block's threads; *total: the sum. Two barriers.
__device__ __forceinline__ int block_scan(int v, int* lds /* kEvictWaves + 1 */, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kEvictWaves; ++w) {
    const int s = lds[w];
    before += w < wave ? s : 0;
    all += s;
  }
  __syncthreads();
  *total = all;
  return before + x - v;
}

// One block per (kv head, sequence): the budget-th greatest key by radix
// select, eight bits at a time from the top (keys in registers for R > 0, up
// to R per thread; read again per pass for R == 0), then the lists of the
// vacated slots before the budget and of the kept ones behind it, both in
// slot order. Thread t holds slots [t S, (t + 1) S): prefix sums over threads
// are prefix sums over slots.
// Bound by the passes of its one CU over the keys, not by the 8 bytes per slot:
// 25 us for 32768 slots (7 the loads, 3.5 the keys, 8 the digits, 7 the lists)
// with keys in registers, 108 read again per pass, 31 in LDS with a lane per
// slot and the lists from wave masks (a CU's 16 waves share one scalar unit).
// Each count of keys per thread is a kernel of its own (4097 slots by radix
// select: 12.2 us with 8 per thread, 14.0 with 32).
template <int R>
__global__ __launch_bounds__(kEvictThreads) void kv_evict_select_kernel(const EvictArgs a) {
  __shared__ __align__(16) int hist[256 * kHistCopies + 1024];
  __shared__ int digit_sum[256];
  __shared__ int scan[kEvictWaves + 1];
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
  const int64_t pair = (int64_t)s * a.c.hkv + h;
  const int n = (int)kv_length(a.lengths[s], a.max_len, a.table_stride, a.c.shift);
  const int budget = (int)a.budget;
  if (a.budget >= n) {   // nothing to evict
    if (tid == 0) a.count[pair] = 0;
    return;
  }
  const int32_t* row = a.table + (int64_t)s * a.table_stride;
  const int S = R > 0 ? R : ((n + kEvictThreads - 1) / kEvictThreads + 3) & ~3;   // slots per thread
  const int first = tid * S;   // 1024 * S < 2^31: n is
  // Four consecutive slots share a page. Every load goes out, from page 0 where
  // there is none (the value is then not used), so that none waits for another.
  auto entry4 = [&](int slot) { return row[slot < n ? slot >> a.c.shift : 0]; };   // n lies within the row
  auto page_of = [&](int32_t id, int slot) {
    return (int)(slot < n) & (int)(id >= 0) & (int)((int64_t)id < a.c.n_pages) ? id : -1;
  };
  auto page4 = [&](int slot) { return page_of(entry4(slot), slot); };
  const int32_t* const pos = a.recent > 0 ? a.c.pos : reinterpret_cast<const int32_t*>(a.c.weight);   // not used for 0
  auto at4 = [&](int32_t page, int slot) { return kv_slot_at(a.c, page < 0 ? 0 : page, h, slot & (a.c.ps - 1)); };
  constexpr int kRegs = R > 0 ? R : 4;
  uint32_t key[kRegs];
  // the keys of four slots, a slot without a page below all others
  int newest = 0;   // position; protected: within `recent` of it (the difference fits 32 bits unsigned)
  const uint32_t recent = (uint32_t)a.recent;
  auto keys4 = [&](int32_t page, const float4& w, const int4& p, uint32_t* k) {
    const float f[4] = {w.x, w.y, w.z, w.w};
    const int q[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t of = weight_key(f[j]), kept = (uint32_t)newest - (uint32_t)q[j] < recent ? kKeyProtected : of;
      k[j] = page < 0 ? 0u : kept;
    }
  };
  auto newest4 = [&](int32_t page, int slot, const int4& p, int m) {
    const int q[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = (int)(page >= 0) & (int)(slot + j < n) ? q[j] : INT32_MIN;
      m = v > m ? v : m;
    }
    return m;
  };
  auto block_max = [&](int m) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
      const int o = __shfl_xor(m, d);
      m = o > m ? o : m;
    }
    if (lane == 0) scan[tid >> 6] = m;
    __syncthreads();
    m = INT32_MIN;
#pragma unroll
    for (int w = 0; w < kEvictWaves; ++w) m = scan[w] > m ? scan[w] : m;
    __syncthreads();
    return m;
  };
  if constexpr (R > 0) {
    // A wave's 64 R slots as they lie in memory, 256 per load (a thread's own R
    // would cost a cache line per lane and load); through LDS they then go to
    // their threads.
    const int base = (tid >> 6) * 64 * R + lane * 4;
    int32_t page[R / 4];
    float4 w[R / 4];
    int4 p[R / 4];
#pragma unroll
    for (int r = 0; r < R / 4; ++r) page[r] = entry4(base + 256 * r);
#pragma unroll
    for (int r = 0; r < R / 4; ++r) {
      page[r] = page_of(page[r], base + 256 * r);
      const int64_t at = at4(page[r], base + 256 * r);
      w[r] = *reinterpret_cast<const float4*>(a.c.weight + at);
      p[r] = *reinterpret_cast<const int4*>(pos + at);
    }
    if (a.recent > 0) {
      int m = INT32_MIN;
#pragma unroll
      for (int r = 0; r < R / 4; ++r) m = newest4(page[r], base + 256 * r, p[r], m);
      newest = block_max(m);
    }
    // 256 slots in rows of R, one row per thread; padded against bank conflicts
    constexpr int kRow = R >= 16 ? R + 4 : R, kRows = 256 / R;
    uint32_t* const tile = reinterpret_cast<uint32_t*>(hist) + (tid >> 6) * (kRows * kRow);
    static_assert(kEvictWaves * kRows * kRow <= 256 * kHistCopies + 1024, "the tiles fit the histogram's memory");
#pragma unroll
    for (int r = 0; r < R / 4; ++r) {
      uint32_t k4[4];
      keys4(page[r], w[r], p[r], k4);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (base + 256 * r + j >= n) k4[j] = 0u;   // behind the end: after every slot in every order
      *reinterpret_cast<uint4*>(tile + 4 * lane / R * kRow + 4 * lane % R) = make_uint4(k4[0], k4[1], k4[2], k4[3]);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (lane / kRows == r) {
#pragma unroll
        for (int j = 0; j < R; j += 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(tile + lane % kRows * kRow + j);
          key[j] = v.x; key[j + 1] = v.y; key[j + 2] = v.z; key[j + 3] = v.w;
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    __syncthreads();   // the memory becomes the histogram
  } else if (a.recent > 0) {
    int m = INT32_MIN;
    for (int r = 0; r < S; r += 4) {
      const int32_t page = page4(first + r);
      m = newest4(page, first + r, *reinterpret_cast<const int4*>(pos + at4(page, first + r)), m);
    }
    newest = block_max(m);
  }
  // Calls fn(index, key) for the thread's slots first + index in order. With
  // keys in registers also for those behind the end: key 0 and the highest
  // slots, they are never among the kept, nor before the budget.
  auto each = [&](auto&& fn) {
    if constexpr (R > 0) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        fn(r, key[r]);
    } else {
      for (int r = 0; r < S && first + r < n; r += 4) {
        const int32_t page = page4(first + r);
        const int64_t at = at4(page, first + r);
        keys4(page, *reinterpret_cast<const float4*>(a.c.weight + at), *reinterpret_cast<const int4*>(pos + at), key);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (first + r + j < n) fn(r + j, key[j]);
      }
    }
  };
  const int over = n - budget;
  if (over <= kEvictFew) {
    // A sequence that grew past its budget by a few slots (one, step by step):
    // the least key, of equal ones the highest slot, goes, `over` times. A call
    // for 16 sequences, 4 heads: past 4096 by one 8.3 us (by radix select 10.5),
    // by two 9.7 (10.7), by three 11.6 (11.1); past 16384 by one 13.4 (20.5).
    __shared__ uint64_t least[kEvictWaves];
    uint64_t gone = 0;   // keys up to this one are out
    int out[kEvictFew];
    for (int i = 0; i < over; ++i) {
      uint64_t best = ~0ull;
      each([&](int r, uint32_t k) {
        const uint64_t c = (uint64_t)k << 32 | (uint32_t)(INT32_MAX - first - r);   // above 0, and distinct
        if (first + r < n && c > gone && c < best) best = c;
      });
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)best, d);
        best = o < best ? o : best;
      }
      if (lane == 0) least[tid >> 6] = best;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kEvictWaves; ++w) best = least[w] < best ? least[w] : best;
      __syncthreads();
      gone = best;
#pragma unroll
      for (int j = 0; j < kEvictFew; ++j)
        if (j == i) out[j] = INT32_MAX - (int)(uint32_t)best;
    }
    if (tid == 0) {
      int32_t* dst = a.dst + pair * a.max_moves;
      int32_t* src = a.src + pair * a.max_moves;
      int moves = 0, tails = 0;
      // kept slots behind the budget, and the vacated ones before it, ascending
      for (int slot = budget; slot < n; ++slot) {
        bool keep = true;
#pragma unroll
        for (int j = 0; j < kEvictFew; ++j) keep = keep && !(j < over && out[j] == slot);
        if (keep) src[tails++] = slot;
      }
      for (int last = -1; moves < tails; ++moves) {
        int next = INT32_MAX;
#pragma unroll
        for (int j = 0; j < kEvictFew; ++j)
          if (j < over && out[j] > last && out[j] < next) next = out[j];
        dst[moves] = last = next;
      }
      a.count[pair] = moves;
    }
    return;
  }
  uint32_t prefix = 0;   // digits chosen so far
  int want = budget;     // rank (from the top) still to place among keys with the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    reinterpret_cast<int4*>(hist)[tid] = make_int4(0, 0, 0, 0);
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    each([&](int, uint32_t k) {
      if ((k & mask) == prefix) atomicAdd(&hist[((k >> shift) & 255u) * kHistCopies + (lane & (kHistCopies - 1))], 1);
    });
    __syncthreads();
    {
      const int4 c = reinterpret_cast<const int4*>(hist)[tid];   // a quarter of a digit's copies
      uint32_t sum = (uint32_t)(c.x + c.y + c.z + c.w);
      sum += dpp_word<0xB1>(sum);
      sum += dpp_word<0x4E>(sum);
      if ((tid & 3) == 0) digit_sum[tid >> 2] = (int)sum;
    }
    __syncthreads();
    // every wave finds the digit: lane l holds digits 255 - 4 l down to 252 - 4 l
    int part[4], sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      part[j] = digit_sum[255 - 4 * lane - j];
      sum += part[j];
    }
    int x = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(x, d);
      if (lane >= d) x += y;
    }
    int above = x - sum;   // keys of greater digits
    int digit = -1, rest = 0, held = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (above < want && want <= above + part[j]) {
        digit = 255 - 4 * lane - j;
        rest = want - above;
        held = part[j];
      }
      above += part[j];
    }
    const int at = __ffsll((unsigned long long)__ballot(digit >= 0)) - 1;   // one lane: 0 < want <= the keys' number
    prefix |= lane_word((uint32_t)digit, at) << shift;
    want = (int)lane_word((uint32_t)rest, at);
    if (want == (int)lane_word((uint32_t)held, at)) {   // all that share the digits so far are kept
      --prefix;   // not 0: there are more keys than the budget
      want = 0;
      break;
    }
  }
  // Kept are the keys above prefix and `want` of those equal to it, lowest slots
  // first.
  int all, eq_rank = 0;
  if (want > 0) {   // the same in all threads
    int equal = 0;
    each([&](int, uint32_t k) { equal += k == prefix; });
    eq_rank = block_scan(equal, scan, &all);
  }
  const int cut = budget - first;   // the thread's slots from this index on are behind the budget
  int holes = 0, tails = 0, e = eq_rank;
  if constexpr (R > 0) {
    uint32_t keep = 0;   // bit per slot
    each([&](int r, uint32_t k) {
      const bool same = k == prefix;
      keep |= (uint32_t)(k > prefix || (same && e < want)) << r;
      e += same;
    });
    const uint32_t before = cut <= 0 ? 0u : cut >= R ? (uint32_t)((uint64_t(1) << R) - 1) : (1u << cut) - 1u;
    uint32_t hole = ~keep & before, tail = keep & ~before;
    holes = __popc(hole);
    tails = __popc(tail);
    // both counts in one sum: they are equal at the end, half of 1024 R slots at most
    const uint32_t both = (uint32_t)block_scan(holes | tails << 16, scan, &all);
    all &= 0xFFFF;
    int32_t* dst = a.dst + pair * a.max_moves + (both & 0xFFFFu);
    int32_t* src = a.src + pair * a.max_moves + (both >> 16);
    while (hole) {
      const int r = __ffs(hole) - 1;
      hole &= hole - 1;
      *dst++ = first + r;
    }
    while (tail) {
      const int r = __ffs(tail) - 1;
      tail &= tail - 1;
      *src++ = first + r;
    }
  } else {
    each([&](int r, uint32_t k) {
      bool keep = k > prefix;
      if (k == prefix) keep = e++ < want;
      holes += r < cut && !keep;
      tails += r >= cut && keep;
    });
    int hole_at = block_scan(holes, scan, &all);
    int tail_at = block_scan(tails, scan, &all);
    e = eq_rank;
    int32_t* dst = a.dst + pair * a.max_moves;
    int32_t* src = a.src + pair * a.max_moves;
    each([&](int r, uint32_t k) {
      bool keep = k > prefix;
      if (k == prefix) keep = e++ < want;
      if (r < cut && !keep) dst[hole_at++] = first + r;
      if (r >= cut && keep) src[tail_at++] = first + r;
    });
  }
  if (tid == 0) a.count[pair] = all;
}

constexpr int kMoveTile = 64;
constexpr int kMoveThreads = 256;

// Blocks of one kv head of one sequence, 64 moves at a time. Sources lie at or
// behind the budget and destinations before it, so no block reads what another
// writes. K rows move as 16-byte (Q8_0: 8-byte) pieces; V moves lane per
// move, row of a dim by row, so that the ascending slots of a wave share lines.
// Block (0, 0, s) also cuts the length (the selection has read it). Bound by HBM:
// a kept slot's V is one element of each of head_dim lines, so 4 sequences of
// 32768 cut to 8192 read 131 MB and write 62 for the 52 MB each way that move,
// in 49 us (3.9 TB/s).
template <int KIND, int DIM>
__global__ __launch_bounds__(kMoveThreads) void kv_evict_move_kernel(const EvictArgs a) {
  __shared__ int64_t sp[kMoveTile], dp[kMoveTile];   // byte offset of page and head
  __shared__ int32_t ss[kMoveTile], ds[kMoveTile];   // slot within the page; ss -1: no move
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
  if (blockIdx.z == 0 && h == 0 && tid == 0 && (int64_t)a.lengths[s] > a.budget) a.lengths[s] = (int32_t)a.budget;
  if (a.max_moves == 0) return;
  const int64_t pair = (int64_t)s * a.c.hkv + h;
  const int count = a.count[pair];
  const int32_t* row = a.table + (int64_t)s * a.table_stride;
  for (int64_t j0 = (int64_t)blockIdx.z * kMoveTile; j0 < count; j0 += (int64_t)gridDim.z * kMoveTile) {
  __syncthreads();   // the last tile's moves are read
  if (tid < kMoveTile) {
    ss[tid] = -1;
    if (j0 + tid < count) {
      const int from = a.src[pair * a.max_moves + j0 + tid], to = a.dst[pair * a.max_moves + j0 + tid];
      const int32_t fp = kv_page(row, from >> a.c.shift, a.table_stride, a.c.n_pages);
      const int32_t tp = kv_page(row, to >> a.c.shift, a.table_stride, a.c.n_pages);
      if (fp >= 0 && tp >= 0) {
        const int m = a.c.ps - 1;
        sp[tid] = kv_head_at(a.c, fp, h);
        dp[tid] = kv_head_at(a.c, tp, h);
        ss[tid] = from & m;
        ds[tid] = to & m;
        const int64_t i = kv_slot_at(a.c, fp, h, from & m), o = kv_slot_at(a.c, tp, h, to & m);
        a.c.weight[o] = a.c.weight[i];
        if (a.c.pos) a.c.pos[o] = a.c.pos[i];
      }
    }
  }
  __syncthreads();
  const int rows = count - j0 < kMoveTile ? (int)(count - j0) : kMoveTile;
  constexpr int kOct = DIM / 8;
  for (int i = tid; i < rows * kOct; i += kMoveThreads) {
    const int r = i / kOct, o = i % kOct;
    if (ss[r] < 0) continue;
    if constexpr (KIND == kKvQ80)
      *reinterpret_cast<uint2*>(a.c.k + dp[r] + ds[r] * DIM + o * 8) =
          *reinterpret_cast<const uint2*>(a.c.k + sp[r] + ss[r] * DIM + o * 8);
    else
      *reinterpret_cast<uint4*>(a.c.k + dp[r] + (ds[r] * DIM + o * 8) * 2) =
          *reinterpret_cast<const uint4*>(a.c.k + sp[r] + (ss[r] * DIM + o * 8) * 2);
  }
  // Moves of a prompt's eviction: 50 us a lane per move (4 sequences of 32768 to
  // 8192, 4 heads), 156 a thread per dim; one move per head (16 sequences): 4.8
  // us against 4.0.
  if (rows >= 16) {
    // lane per move, kBatch dims of a wave in flight
    constexpr int kBatch = 16;
    if (lane < rows && ss[lane] >= 0) {
      const uint8_t* from = a.c.v + sp[lane];
      uint8_t* to = a.c.v + dp[lane];
      const int f = ss[lane], t = ds[lane];
      for (int d0 = (tid >> 6) * kBatch; d0 < DIM; d0 += (kMoveThreads / 64) * kBatch) {
        if constexpr (KIND == kKvQ80) {
          uint8_t x[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) x[j] = from[(d0 + j) * a.c.ps + f];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) to[(d0 + j) * a.c.ps + t] = x[j];
        } else {
          uint16_t x[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) x[j] = reinterpret_cast<const uint16_t*>(from)[(d0 + j) * a.c.ps + f];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) reinterpret_cast<uint16_t*>(to)[(d0 + j) * a.c.ps + t] = x[j];
        }
      }
    }
  } else {
    // few moves: thread per dim
    for (int i = tid; i < rows * DIM; i += kMoveThreads) {
      const int r = i / DIM, d = i % DIM;
      if (ss[r] < 0) continue;
      if constexpr (KIND == kKvQ80)
        a.c.v[dp[r] + d * a.c.ps + ds[r]] = a.c.v[sp[r] + d * a.c.ps + ss[r]];
      else
        reinterpret_cast<uint16_t*>(a.c.v + dp[r])[d * a.c.ps + ds[r]] =
            reinterpret_cast<const uint16_t*>(a.c.v + sp[r])[d * a.c.ps + ss[r]];
    }
  }
  if constexpr (KIND == kKvQ80) {   // the scales behind the codes
    constexpr int NB = DIM / 32;
    for (int i = tid; i < rows * NB; i += kMoveThreads) {
      const int r = i / NB, b = i % NB;
      if (ss[r] < 0) continue;
      reinterpret_cast<uint16_t*>(a.c.k + dp[r] + a.c.ps * DIM)[ds[r] * NB + b] =
          reinterpret_cast<const uint16_t*>(a.c.k + sp[r] + a.c.ps * DIM)[ss[r] * NB + b];
      reinterpret_cast<uint16_t*>(a.c.v + dp[r] + a.c.ps * DIM)[b * a.c.ps + ds[r]] =
          reinterpret_cast<const uint16_t*>(a.c.v + sp[r] + a.c.ps * DIM)[b * a.c.ps + ss[r]];
    }
  }
  }
}

}  // namespace gqk
