// Attention of many new tokens per sequence over the paged key-value cache (BF16
// queries; gguf_attn_extend in include/gguf_tokens.h).
//
// A block takes 128 columns, (row, query head) pairs of one kv head, 32 per wave, and
// walks over the slots they see in tiles of 64, which its waves share in LDS:
//   S^T = K Q^T    32 x 32 tiles, A = K (rows: slots), B = Q (columns), in registers
//   O^T += V^T P^T A = V^T (rows: dims), B = P^T
// Transposed products leave a lane with one column throughout, so that the running
// maximum and sum are per-lane values (the two halves of the wave hold a column each
// half). K's rows lie in LDS with bits 2 and 3 of the slot swapped: the sixteen
// scores of a lane then are two runs of eight consecutive slots, which is the B operand
// of the second product as it stands, and V, stored transposed in the cache, is its A
// operand. Columns are pairs so that the query heads of a kv head share its K and V, and
// the causal mask costs a tile or two per block, not one per head.
//
// Bound: the matrix units' power. 16384 tokens, causal, 16 heads of 128 over 4, BF16:
// 1.06 ms, 1.04 PFLOP/s, where a library product of 8192 x 8192 x 8192 reaches 1.19 (with
// inputs of zeros the two reach 1.33 and 1.79: the clock follows the power that the data
// draws). What the order of instructions gave (prompt of 4096): the vector work of a
// half tile's softmax between the matrix instructions of the other half's product, operands
// read from LDS four instructions ahead, 229 -> 167 us at head dim 256, 147 -> 130 at 192.
// At smaller sizes a block's start and end, about 10 us (its place, the page ids, q, the
// first tiles of K and V in turn; the join of the two groups and the store), beside 2.2 us
// per pair of tiles: one prompt of 4096 90 - 104 us (0.66 - 0.76 PFLOP/s), of 512 18.
//
// Weights enter the second product as bf16 (BF16 caches) or fp16, as the values do: a
// wider weight would double the product. Maxima, sums and outputs are fp32.
#pragma once

#include "attn.hpp"

namespace gqk {

// Most groups of four waves of a block: registers hold two up to head dim 128 (Q8_0,
// whose codes are converted on the way, 64).
constexpr int prompt_groups(bool q8, int dim) { return dim <= (q8 ? 64 : 128) ? 2 : 1; }

struct AttnPromptArgs : AttnRowsArgs {
  int32_t tiles;   // tiles of columns of the grid
};

constexpr int kPromptWaves = 4;     // that share a tile of slots
constexpr int kPromptThreads = kPromptWaves * 64;
// The maximum that weights are relative to is raised only where one exceeds it by a
// factor of 2^8: rescaling the output costs half as much as a tile's exponentials.
constexpr float kPromptSlack = 8.0f;
constexpr int kPromptAhead = 4;   // reads of LDS before their matrix instruction

typedef float f32x16v __attribute__((ext_vector_type(16)));

template <int KIND>
__device__ __forceinline__ f32x16v prompt_mfma(const uint4& a, const uint4& b, const f32x16v& c) {
  if constexpr (KIND == kKvBF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8v, a), __builtin_bit_cast(bf16x8v, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Slots of a tile, and where its values lie in LDS: rows of 16-byte chunks, a chunk at
// chunk ^ swizzle(row), so that sixteen consecutive rows' chunks of one number lie in
// sixteen different groups of banks.
template <int NB>
struct PromptTile {
  static constexpr int kDim = NB * 32;
  static constexpr int kSlots = kPromptSlots;
  static constexpr int kKChunks = kDim / 8;    // of a slot's row of K
  static constexpr int kVChunks = kSlots / 8;  // of a dim's row of V
  static constexpr int kBytes = kSlots * kDim * 2;
  static constexpr int kLoads = kBytes / (kPromptThreads * 16);   // 16-byte loads of a thread, K and V each
  __device__ static __forceinline__ int k_swizzle(int row) {
    return kKChunks % 16 == 0 ? row & 15 : kKChunks % 8 == 0 ? row >> 1 & 7 : row >> 2 & 3;
  }
  static_assert(kVChunks == 8, "v_swizzle");
  __device__ static __forceinline__ int v_swizzle(int row) { return row >> 1 & 7; }
};

// Slot (within 32) of row `r` of K in LDS, and back.
__device__ __forceinline__ int prompt_slot(int r) { return (r & ~12) | (r & 4) << 1 | (r & 8) >> 1; }

// Sixteen bytes per lane from global memory to 1 KiB of LDS at `lds` (uniform), lane by
// lane. Assembly, so that the compiler, which cannot tell which bytes of LDS are in
// flight, does not wait for all loads before each read of LDS; the caller waits. M0 is
// never live in compiled code here: only such loads of the compiler's own would set it.
// The compiler may hold uniform values in vector registers; what the assembly takes as
// scalars is read from the first lane.
__device__ __forceinline__ void prompt_load_lds(const uint8_t* base, uint32_t offset, uint32_t lds) {
  lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds);
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  base = reinterpret_cast<const uint8_t*>((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(b >> 32)) << 32 |
                                          (uint32_t)__builtin_amdgcn_readfirstlane((int)b));
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(base), "s"(lds)
               : "memory");
}
__device__ __forceinline__ void prompt_load_lds(const uint8_t* p, uint32_t lds) {
  lds = (uint32_t)__builtin_amdgcn_readfirstlane((int)lds);
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(lds) : "memory");
}

// 16 bytes of LDS.
__device__ __forceinline__ uint4 prompt_lds16(uint32_t at) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(16)));
  const u32x4 v = *reinterpret_cast<const __attribute__((address_space(3))) u32x4*>(at);
  return make_uint4(v.x, v.y, v.z, v.w);
}

// N matrix instructions, their operands read from LDS `kPromptAhead` of them before, with
// the chunks 0 .. CHUNKS - 1 of vector work spread between them, in this order: left to
// itself the compiler puts each read right before its use and the vector work behind.
template <int N, int CHUNKS, class Load, class Mma, class Work>
__device__ __forceinline__ void prompt_phase(Load&& load, Mma&& mma, Work&& work) {
  uint4 f[N];
#pragma unroll
  for (int i = 0; i < N && i < kPromptAhead; ++i) f[i] = load(i);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int c = i * CHUNKS / N; c < (i + 1) * CHUNKS / N; ++c) work(c);
    __builtin_amdgcn_sched_barrier(0);
    mma(i, f[i]);
    if (i + kPromptAhead < N) f[i + kPromptAhead] = load(i + kPromptAhead);
    __builtin_amdgcn_sched_barrier(0);
  }
}

__device__ __forceinline__ void prompt_store16(uint32_t at, const uint4& x) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(16)));
  *reinterpret_cast<__attribute__((address_space(3))) u32x4*>(at) = u32x4{x.x, x.y, x.z, x.w};
}

// A value the compiler takes for new each time: what is formed from it is not kept in
// registers over the loop.
__device__ __forceinline__ int prompt_anew(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// The greater of a value and the other half wave's.
__device__ __forceinline__ float prompt_half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// GROUPS of four waves take the tiles of slots in turn and join in LDS.
template <int KIND, int NB, int GROUPS>
__global__ __launch_bounds__(kPromptThreads * GROUPS, NB <= 4 ? 2 : 1) void attn_prompt_kernel(const AttnPromptArgs a) {
  using Tile = PromptTile<NB>;
  constexpr int DIM = Tile::kDim, T = Tile::kSlots, KC = Tile::kKChunks, VC = Tile::kVChunks, LOADS = Tile::kLoads;
  constexpr int KS = DIM / 16, NT = DIM / 32;   // steps of S, tiles of O
  constexpr int MM = KIND == kKvBF16 ? kKvBF16 : kKvF16;     // type of the products
  constexpr bool Q8 = KIND == kKvQ80;
  constexpr int RUNS = (NB + 1) / 2;               // Q8_0: runs of sixteen codes of a lane, K and V each
  constexpr int SC = T * NB * 2 / 16;              // Q8_0: 16-byte chunks of a tile's scales, K and V each (at most 64)
  const int tid = threadIdx.x, lane = tid & 63;
  const int group = GROUPS == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid / kPromptThreads);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) % kPromptWaves;   // of the group
  const int col = lane & 31, hf = lane >> 5;
  const int h = blockIdx.x, split = blockIdx.z;
  // the last tiles of a sequence see most: they go first
  const RowsPlan plan = attn_rows_plan<kPromptColumns>(a, a.tiles - 1 - (int)blockIdx.y, lane);
  const RowTile rt = plan.t;
  if (rt.seq < 0) return;
  const int s = rt.seq, held = plan.held, chunk = plan.chunk;
  const int width = rt.rows * a.group;
  const int unit = a.c.ps > T ? a.c.ps : T;
  const TileRange r = tile_range(held, rt.rows, a.group, rt.tile, kPromptColumns, a.window, a.sinks, unit);
  const int begin = split * chunk, end = r.n - begin < chunk ? r.n : begin + chunk;   // numbered without the gap
  const int c = rt.tile * kPromptColumns + wave * 32 + col;   // this lane's column
  const bool live = c < width;
  const int cc = live ? c : width - 1;
  const int64_t row = rt.row0 + cc / a.group;
  const int head = h * a.group + cc % a.group;
  uint16_t* const out = reinterpret_cast<uint16_t*>(a.out) + row * a.out_stride + (int64_t)head * DIM;
  if (begin >= r.n) {
    if (a.splits == 1 && live && group == 0) {   // nothing seen
#pragma unroll
      for (int i = 0; i < DIM / 8; ++i)
        if ((i & 1) == hf) *reinterpret_cast<uint4*>(out + 8 * i) = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const SlotRange range = slot_range(held, rt.rows, cc / a.group, a.window);
  const bool idle = rt.tile * kPromptColumns + wave * 32 >= width;   // no column of this wave
  const TileRange wr = tile_range(held, rt.rows, a.group, idle ? rt.tile * kPromptWaves : rt.tile * kPromptWaves + wave, 32,
                                  a.window, a.sinks, unit);
  const int w_hi = wr.n + wr.gap;   // slots from here on no column of this wave sees

  // K and V of two tiles of each group: K, K, V, V
  __shared__ __align__(1024) uint8_t lds[GROUPS][4][Tile::kBytes];
  // Q8_0, per wave: the scales of a tile of K and of V, the codes of K that it converts
  constexpr int kRaw = 2 * SC * 16, kWave = Q8 ? kRaw + 32 * NB * 16 : 16;
  __shared__ __align__(1024) uint8_t lds_wave[Q8 ? GROUPS * kPromptWaves : 1][kWave];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&lds[group][0][0];
  const uint32_t scales0 =
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&lds_wave[Q8 ? group * kPromptWaves + wave : 0][0];

  const uint8_t* const kh = a.c.k + (int64_t)h * a.c.head_bytes;
  const uint8_t* const vh = a.c.v + (int64_t)h * a.c.head_bytes;
  const int64_t page_bytes = (int64_t)a.c.hkv * a.c.head_bytes;
  const int shift = a.c.shift, smask = a.c.ps - 1;
  const int32_t* const table = a.table + (int64_t)s * a.table_stride;

  // Page ids of 64 pages from page0 on, one per lane (numbered without the gap; -1:
  // bad). Behind the block's last slot whatever the entry is not followed.
  int page0 = 0, pid = 0;
  const int pages = (end + smask) >> shift;
  auto fetch_pages = [&](int first) {
    page0 = first;
    pid = 0;
    const int p = first + lane;
    if (p < pages) pid = kv_page(table, p + (p >= r.pad >> shift ? r.gap >> shift : 0), a.table_stride, a.c.n_pages);
  };
  auto real_of = [&](int v0) { return v0 + (v0 >= r.pad ? r.gap : 0); };
  // the next tile from v on that any column sees
  auto seen_from = [&](int v) {
    while (v < end && real_of(v) >= a.sinks && real_of(v) + T <= r.near) v += T;
    return v;
  };
  // This lane's chunk of load i. Of K a wave loads sixteen slots, which lie in one
  // page; of V whole rows of dims, whose chunks of eight slots lie in up to four pages,
  // of two patterns over the lanes that loads take in turn (v_swizzle).
  uint32_t k_at[Q8 ? 1 : LOADS], v_at[Q8 ? 1 : LOADS];   // offset in the page's head, of V without the slot where pages are small
  const bool whole = a.c.ps >= T;
#pragma unroll
  for (int i = 0; i < (Q8 ? 0 : LOADS); ++i) {
    const int L = (wave * LOADS + i) * 64 + lane;
    const int kr = L / KC, vr = L / VC;
    const int slot = (kr & ~31) | prompt_slot(kr & 31);
    k_at[i] = (slot - 16 * wave) * (DIM * 2) + ((L % KC) ^ Tile::k_swizzle(kr)) * 16;
    v_at[i] = (vr * a.c.ps + (whole ? ((L % VC) ^ Tile::v_swizzle(vr)) * 8 : 0)) * 2;
  }
  auto page_at = [&](int v) {   // of uniform slot v
    const int id = __builtin_amdgcn_readlane(pid, (v >> shift) - page0);
    return (id < 0 ? 0 : id) * page_bytes;
  };
  // Slots of a tile whose values are looked at.
  auto present = [&](int v0) -> uint64_t {
    const int n = end - v0;
    uint64_t m = n >= T ? ~0ull : (1ull << n) - 1;
    for (int p = v0; p < v0 + T && p < end; p += a.c.ps) {
      const int id = __builtin_amdgcn_readlane(pid, (p >> shift) - page0);
      if (id < 0) m &= whole ? 0 : ~(((1ull << a.c.ps) - 1) << (p - v0));
    }
    return m;
  };

  auto issue = [&](int v, int buf) {
    const uint32_t to = lds0 + buf * Tile::kBytes + wave * LOADS * 1024;
    const int vk = v + 16 * wave;
    const uint8_t* from = kh + page_at(vk) + (vk & smask) * (DIM * 2);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) prompt_load_lds(from, k_at[i], to + i * 1024);
    if (whole) {
      from = vh + page_at(v) + (v & smask) * 2;
#pragma unroll
      for (int i = 0; i < LOADS; ++i) prompt_load_lds(from, v_at[i], to + 2 * Tile::kBytes + i * 1024);
    } else {
      const uint8_t* of[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int p = v + ((lane % VC) ^ Tile::v_swizzle(j * 8 + lane / VC)) * 8, id = __shfl(pid, (p >> shift) - page0);
        of[j] = vh + (id < 0 ? 0 : id) * page_bytes + (p & smask) * 2;
      }
#pragma unroll
      for (int i = 0; i < LOADS; ++i)
        prompt_load_lds(of[(wave * LOADS + i) & 1] + v_at[i], to + 2 * Tile::kBytes + i * 1024);
    }
  };
  // Q8_0. A wave converts sixteen slots of K and DIM / 4 dims of V, by runs of sixteen
  // codes: run u is codes 16 (u % (2 NB)) .. of slot u / (2 NB), or slots 16 (u % 4) .. of
  // dim u / 4; lane l takes u = l, l + 64, ... Of a tile's V codes go through registers,
  // K's (registers are short) and the scales through LDS as they are.
  constexpr bool POW2 = (NB & (NB - 1)) == 0;   // a lane's runs of K then lie 64 / (2 NB) slots apart
  uint4 v_raw[Q8 ? RUNS : 1];
  uint32_t v_run = 0;           // offset of run l of V in a page's head, from the tile's slot on
  uint32_t k_lo = 0, v_lo = 0;  // where run l goes in LDS: its first chunk (the second is at ^ 16)
  auto k_target = [&](int u) {
    const int slot = 16 * wave + u / (2 * NB), r = (slot & ~31) | prompt_slot(slot & 31);
    return lds0 + r * (DIM * 2) + ((u % (2 * NB) * 2 ^ Tile::k_swizzle(r)) << 4);
  };
  auto v_target = [&](int u) {
    const int r = wave * 8 * NB + u / 4;
    return lds0 + 2 * Tile::kBytes + r * (T * 2) + ((u % 4 * 2 ^ Tile::v_swizzle(r)) << 4);
  };
  if constexpr (Q8) {
    v_run = (wave * 8 * NB + lane / 4) * a.c.ps + (whole ? lane % 4 * 16 : 0);
    k_lo = k_target(lane);
    v_lo = v_target(lane);
  }
  // (Inlined by force: of a call the compiler keeps what the lambdas capture, all of the
  // kernel's state, in scratch memory; 8 sequences of 8 rows behind 500 slots took 127 us so
  // at head dim 256, 32 inlined.)
  auto fetch = [&](auto is_k, int v) __attribute__((always_inline)) {
    if constexpr (Q8) {
      constexpr bool K = decltype(is_k)::value;
      if constexpr (K) {
        // sixteen slots of one page
        const int vk = v + 16 * wave;
        const uint8_t* from = kh + page_at(vk) + (vk & smask) * DIM;
#pragma unroll
        for (int i = 0; i < RUNS; ++i) {
          if (NB % 2 && i * 64 + lane >= 32 * NB) continue;
          prompt_load_lds(from + i * 1024, lane * 16, scales0 + kRaw + i * 1024);   // their codes lie in a row
        }
        // chunk l of [slot][block], behind the page's codes
        if (whole) {
          from = kh + page_at(v) + a.c.ps * DIM + (v & smask) * (NB * 2);
          if (lane < SC) prompt_load_lds(from, lane * 16, scales0);
        } else {
          const int ln = prompt_anew(lane), p = v + ln * 8 / NB, id = __shfl(pid, ((p >> shift) - page0) & 63);
          const uint8_t* mine = kh + (id < 0 ? 0 : id) * page_bytes + a.c.ps * DIM + ((p & smask) * NB + ln * 8 % NB) * 2;
          if (lane < SC) prompt_load_lds(mine, scales0);
        }
      } else if (whole) {
        const uint8_t* from = vh + page_at(v) + (v & smask);
#pragma unroll
        for (int i = 0; i < RUNS; ++i)
          if (!(NB % 2) || i * 64 + lane < 32 * NB) v_raw[i] = load16(from + i * 16 * a.c.ps + v_run);
        const int l = prompt_anew(lane);
        const uint32_t at = l / (T / 8) * a.c.ps * 2 + l % (T / 8) * 16;   // chunk l of [block][slot]
        if (lane < SC) prompt_load_lds(from + a.c.ps * DIM + (v & smask), at, scales0 + SC * 16);
      } else {
        const int ln = prompt_anew(lane), p = v + ln % 4 * 16, id = __shfl(pid, (p >> shift) - page0);
        const uint8_t* from = vh + (id < 0 ? 0 : id) * page_bytes + (p & smask) + v_run;
#pragma unroll
        for (int i = 0; i < RUNS; ++i)
          if (!(NB % 2) || i * 64 + lane < 32 * NB) v_raw[i] = load16(from + i * 16 * a.c.ps);
        const int ps = v + ln % (T / 8) * 8, ids = __shfl(pid, (ps >> shift) - page0);
        const uint8_t* mine = vh + (ids < 0 ? 0 : ids) * page_bytes + a.c.ps * DIM + (ln / (T / 8) * a.c.ps + (ps & smask)) * 2;
        if (lane < SC) prompt_load_lds(mine, scales0 + SC * 16);
      }
    }
  };
  // A value enters fp16 as code * (d 2^e), e 0 for a greatest scale of the tile from 2^-7 to
  // 2^8 and else such that it comes to [2^7, 2^8) (or e to 15): the nearest fp16 of the
  // value, or within 2^-18 of the greatest scale. (fp16 holds a code exactly, not its product
  // with a scale: two parts would double both products.) K's scores take 2^-e back tile by
  // tile; V's sums are kept in units of 2^-ve, which follow the greatest scale met so far.
  // The conversions double the vector work: 1024 rows behind 30000 slots 400 us, F16 285.
  int ke = 0, ve = 0;
  bool first_v = true;
  auto settle = [&](auto is_k, uint64_t here) __attribute__((always_inline)) {
    if constexpr (Q8) {
      constexpr bool K = decltype(is_k)::value;
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      auto max_pair = [](uint32_t a, uint32_t b) {   // of unsigned halves
        typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
      };
      uint32_t pair = 0;
      const int ln = prompt_anew(lane), c = ln < SC ? ln : 0;
      const uint4 d = prompt_lds16(scales0 + ((K ? 0 : SC) + c) * 16);
      const uint32_t w[4] = {d.x, d.y, d.z, d.w};
      if (here == ~0ull) {
#pragma unroll
        for (int j = 0; j < 4; ++j) pair = max_pair(pair, w[j] & 0x7FFF7FFFu);
      } else {   // behind the end: anything
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int slot = K ? (c * 8 + j) / NB : c % (T / 8) * 8 + j;
          if (here >> slot & 1) pair = max_pair(pair, w[j / 2] >> (j % 2 * 16) & 0x7FFFu);
        }
      }
      pair = max_word(pair >> 16, pair & 0xFFFFu);
      // the usual case: a greatest scale of 2^-7 to 2^8 before and now
      if (__any(pair >= 8u << 10) && !__any(pair >= 23u << 10) && (K || ve == 0)) {
        if (K) ke = 0;
        first_v &= K;
        return;
      }
      pair = max_word(pair, dpp_word<0xB1>(pair));
      pair = max_word(pair, dpp_word<0x4E>(pair));
      pair = max_word(pair, dpp_word<0x141>(pair));
      pair = max_word(pair, dpp_word<0x140>(pair));
      pair = max_word(max_word(lane_word(pair, 0), lane_word(pair, 16)), max_word(lane_word(pair, 32), lane_word(pair, 48)));
      // an exponent field E: below 2^(E - 14). Scales of 2^-7 to 2^8 enter as they are.
      const int E = (int)(pair >> 10);
      int e = E >= 8 && E <= 22 ? 0 : 22 - E;
      e = e > 15 ? 15 : e < -8 ? -8 : e;
      if (K) ke = e;
      else ve = first_v || e < ve ? e : ve;
      if (!K) first_v = false;
    }
  };
  auto times = [](uint32_t x, uint32_t y) {
    return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, x) * __builtin_bit_cast(f16x2, y));
  };
  // The runs of codes to buffer buf, each in three chunks of work: where it goes and its
  // scales, the first eight codes, the others.
  uint32_t to_lo = 0, bits = 0;
  uint4 d0, d1;
  auto convert = [&](auto is_k, int chunk, int buf, uint64_t here) __attribute__((always_inline)) {
    if constexpr (Q8) {
      constexpr bool K = decltype(is_k)::value;
      const int i = chunk / 3, part = chunk % 3;
      if (part == 0) {
        const uint32_t mul = 0x00010001u * (uint32_t)((15 + (K ? ke : ve)) << 10);   // 2^e twice
        uint32_t at;
        if constexpr (K) {
          if constexpr (POW2) {
            // slots 8 further (NB 4) lie 4 rows further, whose swizzle is that of the first ^ 4
            constexpr int kStep = 64 / (2 * NB);
            const int r = kStep == 8 ? 4 * i : kStep == 4 ? (i & 1) * 8 + (i >> 1) * 4 : 0;
            to_lo = (k_lo ^ (Tile::k_swizzle(r) << 4)) + r * (DIM * 2);
          } else {
            to_lo = k_target(i * 64 + prompt_anew(lane));
          }
          int u = i * 64 + prompt_anew(lane);
          if (NB % 2 && u >= 32 * NB) u = 0;
          at = scales0 + ((16 * wave + u / (2 * NB)) * NB + u % (2 * NB) / 2) * 2;
          uint32_t d = *reinterpret_cast<const __attribute__((address_space(3))) uint16_t*>(at);
          d |= d << 16;
          if (ke != 0) d = times(d, mul);
          d0 = d1 = make_uint4(d, d, d, d);
        } else {
          if constexpr (NB % 2 == 0) {
            // sixteen dims further: the same swizzle
            to_lo = v_lo + i * 16 * (T * 2);
            at = scales0 + (SC + (wave * 8 * NB + i * 16) / 32 * (T / 8)) * 16 + prompt_anew(lane) % 4 * 32;
          } else {
            const int u = i * 64 + prompt_anew(lane);
            to_lo = v_target(u);
            at = scales0 + (SC + (u < 32 * NB ? (wave * 8 * NB + u / 4) / 32 * (T / 8) : 0) + u % 4 * 2) * 16;
          }
          d0 = prompt_lds16(at);
          d1 = prompt_lds16(at + 16);
          if (ve != 0) {
            d0 = make_uint4(times(d0.x, mul), times(d0.y, mul), times(d0.z, mul), times(d0.w, mul));
            d1 = make_uint4(times(d1.x, mul), times(d1.y, mul), times(d1.z, mul), times(d1.w, mul));
          }
          bits = (uint32_t)(here >> (prompt_anew(lane) % 4 * 16)) & 0xFFFFu;
        }
        to_lo += buf * Tile::kBytes;
        return;
      }
      uint4 raw = v_raw[i];
      if (K) raw = prompt_lds16(scales0 + kRaw + (NB % 2 && i * 64 + lane >= 32 * NB ? 0 : i * 1024 + lane * 16));
      const uint4 d = part == 1 ? d0 : d1;
      uint4 x = codes_f16(part == 1 ? make_uint2(raw.x, raw.y) : make_uint2(raw.z, raw.w));
      x = make_uint4(times(x.x, d.x), times(x.y, d.y), times(x.z, d.z), times(x.w, d.w));
      if (!K && here != ~0ull) {   // behind the end: zero
        auto keep = [&](int j) {
          return ((bits >> (8 * part - 8 + 2 * j) & 1) ? 0xFFFFu : 0u) | ((bits >> (8 * part - 8 + 2 * j) & 2) ? 0xFFFF0000u : 0u);
        };
        x = make_uint4(x.x & keep(0), x.y & keep(1), x.z & keep(2), x.w & keep(3));
      }
      if (NB % 2 && i * 64 + lane >= 32 * NB) return;
      prompt_store16(part == 1 ? to_lo : to_lo ^ 16, x);
    }
  };
  using K_ = std::true_type;
  using V_ = std::false_type;
  auto convert_all = [&](auto is_k, int buf, uint64_t here) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 3 * RUNS; ++i) convert(is_k, i, buf, here);
  };

  // the group's tile and the one behind its next; all groups count alike
  int first = seen_from(begin);
  auto mine = [&](int v) {
    for (int g = 0; g < group; ++g) v = seen_from(v + T);
    return v;
  };
  fetch_pages(first >> shift);
  uint64_t here0 = 0, here1 = 0;   // Q8_0: of the tile in hand and the next
  if (mine(first) < end) {
    if constexpr (Q8) {
      here0 = present(mine(first));
      fetch(K_{}, mine(first));
      fetch(V_{}, mine(first));
    } else {
      issue(mine(first), 0);
    }
  }

  // q of this lane's column: the B operand, dims 16 k + 8 hf .. + 7
  uint4 q[KS];
  float factor;   // of the products, to the log2 domain
  {
    const uint16_t* qp = reinterpret_cast<const uint16_t*>(a.q) + row * a.q_stride + (int64_t)head * DIM + 8 * hf;
    const uint32_t sign = a.qscale < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      q[k] = *reinterpret_cast<const uint4*>(qp + 16 * k);
      q[k] = make_uint4(q[k].x ^ sign, q[k].y ^ sign, q[k].z ^ sign, q[k].w ^ sign);
      if (!live || a.qscale == 0.f) q[k] = make_uint4(0, 0, 0, 0);
    }
    factor = a.qscale == 0.f ? 1.f : fabsf(a.qscale);
    if constexpr (MM == kKvF16) {
      // to fp16: the row's greatest magnitude goes to [512, 1024). Exact down to 2^-26 of it
      // (2^-17, whose eight bits end at fp16's last, 2^-24); what lies lower is within 2^-34 of
      // it (half of that last place)
      float x[KS][8], amax = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint32_t u[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[k][2 * j] = __uint_as_float(u[j] << 16);
          x[k][2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
          amax = fmaxf(amax, fmaxf(fabsf(x[k][2 * j]), fabsf(x[k][2 * j + 1])));
        }
      }
      amax = fmaxf(amax, __shfl_xor(amax, 32));
      int e = 0;
      if (amax > 0.f && amax < __builtin_inff()) {
        (void)__builtin_frexpf(amax, &e);
        e = 10 - e < 100 ? 10 - e : 100;
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          u[j] = __builtin_bit_cast(uint32_t, to_f16x2(__builtin_ldexpf(x[k][2 * j], e), __builtin_ldexpf(x[k][2 * j + 1], e)));
        q[k] = make_uint4(u[0], u[1], u[2], u[3]);
      }
      factor = __builtin_ldexpf(factor, -e);
    }
  }

  // Offsets of this lane's operands in LDS: K's row of 32, V's row of 32.
  uint32_t k_off[KS], v_off[T / 16];
#pragma unroll
  for (int k = 0; k < KS; ++k) k_off[k] = lds0 + col * (DIM * 2) + (((2 * k + hf) ^ Tile::k_swizzle(col)) * 16);
#pragma unroll
  for (int k = 0; k < T / 16; ++k) v_off[k] = lds0 + 2 * Tile::kBytes + col * (T * 2) + (((2 * k + hf) ^ Tile::v_swizzle(col)) * 16);

  f32x16v o[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) o[t] = f32x16v{};
  float m = -__builtin_inff(), l = 0.f;
  int unit_o = 0;   // Q8_0: O's sums are in units of 2^-unit_o

  // What a column does not see of the 32 slots from `real` on.
  auto mask = [&](f32x16v& sc, int real, uint32_t here) {
    const uint32_t bits = slot_bits(range, a.sinks, real) & here;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(bits >> ((i & 8) * 2 + 8 * hf + (i & 7)) & 1)) sc[i] = -__builtin_inff();
  };
  // The softmax of 32 slots in ten chunks: the maximum; whether it is raised, and the
  // factor alpha that the sums so far then take; eight pairs of weights.
  float mx, base, alpha, by = factor;   // by: factor of the tile's scores
  bool raise;
  uint32_t w[8];
  auto soften = [&](const f32x16v& sc, int chunk) {
    if (chunk == 0) {
      mx = sc[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) mx = fmaxf(mx, sc[i]);
    } else if (chunk == 1) {
      mx = prompt_half_max(mx) * by;
      raise = __any(mx > m + kPromptSlack);
      const float old = m;
      m = raise ? fmaxf(m, mx) : m;
      base = m == -__builtin_inff() ? 0.f : m;   // nothing seen yet
      alpha = __builtin_amdgcn_exp2f(old - base);
      l *= alpha;
    } else {
      const int j = chunk - 2;
      const float x = __builtin_amdgcn_exp2f(fmaf(sc[2 * j], by, -base));
      const float y = __builtin_amdgcn_exp2f(fmaf(sc[2 * j + 1], by, -base));
      l += x + y;
      w[j] = MM == kKvBF16 ? pack_bf16x2(x, y) : __builtin_bit_cast(uint32_t, to_f16x2(x, y));
    }
  };
  auto weights = [&](uint4 (&p)[2]) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      p[t] = make_uint4(w[4 * t], w[4 * t + 1], w[4 * t + 2], w[4 * t + 3]);
      asm volatile("" : "+v"(p[t].x), "+v"(p[t].y), "+v"(p[t].z), "+v"(p[t].w));   // computed here, not where it is used
    }
  };
  // Scores of 32 slots, K's rows `at` bytes behind the first buffer's, beside chunks of work.
  auto scores = [&](uint32_t at, f32x16v& sc, auto chunks, auto&& work) {
    sc = f32x16v{};
    prompt_phase<KS, decltype(chunks)::value>([&](int i) { return prompt_lds16(k_off[i] + at); },
                                              [&](int i, const uint4& f) { sc = prompt_mfma<MM>(f, q[i], sc); }, work);
  };
  // Weights times V of 32 slots.
  auto weigh = [&](uint32_t at, int n, const uint4 (&p)[2], auto chunks, auto&& work) {
    prompt_phase<2 * NT, decltype(chunks)::value>(
        [&](int i) { return prompt_lds16(v_off[2 * n + i / NT] + at + i % NT * 32 * T * 2); },
        [&](int i, const uint4& f) { o[i % NT] = prompt_mfma<MM>(f, p[i / NT], o[i % NT]); }, work);
  };
  auto rescale = [&]() {
#pragma unroll
    for (int t = 0; t < NT; ++t) o[t] *= alpha;
  };

  // One tile, in buffer BUF.
  auto step = [&](auto buffer) __attribute__((always_inline)) {
    constexpr int BUF = decltype(buffer)::value;
    constexpr uint32_t kt = BUF * Tile::kBytes, vt = BUF * Tile::kBytes;
    const int v0 = mine(first), real0 = real_of(v0);
    const bool any = v0 < end;
    const uint64_t here = Q8 ? here0 : any ? present(v0) : 0;
    if constexpr (!Q8) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this tile's loads have arrived
      if (any && here != ~0ull) {
        // V behind the end may hold anything: zero, each wave what it has loaded
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
          const int L = (wave * LOADS + i) * 64 + lane;
          const uint32_t bits = (uint32_t)(here >> (8 * ((L % VC) ^ Tile::v_swizzle(L / VC)))) & 0xFFu;
          uint16_t* p = reinterpret_cast<uint16_t*>(lds[group][2 + BUF] + L * 16);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (!(bits >> j & 1)) p[j] = 0;
        }
      }
    }
    __syncthreads();   // everyone's have, and the other buffer is free
    int next = first;
    for (int g = 0; g < GROUPS; ++g) next = seen_from(next + T);
    first = next;
    const int v1 = mine(next);
    if (!Q8 && v1 < end) {
      if (((v1 + T - 1) >> shift) - page0 >= 64) fetch_pages(v1 >> shift);
      issue(v1, BUF ^ 1);
    }
    // Q8_0: K of the next tile is converted beside this one's first scores, then K of the
    // one behind is asked for; V of the next is asked for before and converted beside the
    // last products.
    const bool more = Q8 && v1 < end;
    auto ask_k = [&]() {
      here0 = here1;
      for (int g = 0; g < GROUPS; ++g) next = seen_from(next + T);
      const int v2 = mine(next);
      if (v2 < end) {
        if (((v2 + T - 1) >> shift) - page0 >= 64) fetch_pages(v2 >> shift);
        here1 = present(v2);
        fetch(K_{}, v2);
      }
    };
    if constexpr (Q8) by = __builtin_ldexpf(factor, -ke);   // of this tile's scores
    if (!any || idle || real0 >= w_hi || (real0 >= a.sinks && real0 + T <= wr.near)) {
      if (more) {
        settle(K_{}, here1);
        convert_all(K_{}, BUF ^ 1, here1);
        fetch(V_{}, v1);
        settle(V_{}, here1);
        convert_all(V_{}, BUF ^ 1, here1);
        ask_k();
      }
      return;
    }
    if constexpr (Q8) {
      if (ve != unit_o) {
        alpha = __builtin_ldexpf(1.0f, ve - unit_o);
        rescale();
        unit_o = ve;
      }
    }
    using Softmax = std::integral_constant<int, 10>;
    uint4 p[2];
    f32x16v sa, sb;
    const bool edge = here != ~0ull || real0 < wr.far || real0 + T > wr.full;
    // matrix and vector units side by side, by halves of the tile
    // (behind the last tile old codes are converted once more, into a buffer no one reads)
    using Convert = std::integral_constant<int, Q8 ? 3 * RUNS : 0>;
    settle(K_{}, here1);
    if (more) fetch(V_{}, v1);
    scores(kt, sa, Convert{}, [&](int c) { convert(K_{}, c, BUF ^ 1, here1); });
    const uint64_t here_v = here1;
    if (more) ask_k();
    if (edge) mask(sa, real0, (uint32_t)here);
    scores(kt + 32 * DIM * 2, sb, Softmax{}, [&](int c) { soften(sa, c); });
    weights(p);
    if (raise) rescale();
    if (edge) mask(sb, real0 + 32, (uint32_t)(here >> 32));
    weigh(vt, 0, p, Softmax{}, [&](int c) { soften(sb, c); });
    weights(p);
    if (raise) rescale();
    settle(V_{}, here_v);
    weigh(vt, 1, p, Convert{}, [&](int c) { convert(V_{}, c, BUF ^ 1, here_v); });
  };
  if (Q8 && mine(first) < end) {
    settle(K_{}, here0);
    settle(V_{}, here0);
    convert_all(K_{}, 0, here0);
    convert_all(V_{}, 0, here0);
    int next = first;
    for (int g = 0; g < GROUPS; ++g) next = seen_from(next + T);
    next = mine(next);
    if (next < end) {
      if (((next + T - 1) >> shift) - page0 >= 64) fetch_pages(next >> shift);
      here1 = present(next);
      fetch(K_{}, next);
    }
  }
  unit_o = ve;
  while (first < end) {
    step(std::integral_constant<int, 0>{});
    if (first >= end) break;
    step(std::integral_constant<int, 1>{});
  }

  l += __shfl_xor(l, 32);
  if constexpr (Q8) {
    alpha = __builtin_ldexpf(1.0f, -unit_o);
    rescale();
  }
  if constexpr (GROUPS == 2) {
    // the second group's sums go to the first's waves, lane by lane
    static_assert(kPromptThreads * NT * 64 + kPromptThreads * 8 <= sizeof(lds), "sums fit");
    f32x4* const os = reinterpret_cast<f32x4*>(&lds[0][0][0]) + wave * NT * 4 * 64 + lane;
    float2* const ms = reinterpret_cast<float2*>(&lds[0][0][0] + kPromptThreads * NT * 64) + wave * 64 + lane;
    __syncthreads();
    if (group == 1) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) os[(t * 4 + i) * 64] = f32x4{o[t][4 * i], o[t][4 * i + 1], o[t][4 * i + 2], o[t][4 * i + 3]};
      *ms = make_float2(m, l);
    }
    __syncthreads();
    if (group == 1) return;
    const float2 other = *ms;
    const float top = fmaxf(m, other.x), from = top == -__builtin_inff() ? 0.f : top;
    const float f0 = __builtin_amdgcn_exp2f(m - from), f1 = __builtin_amdgcn_exp2f(other.x - from);
    m = top;
    l = fmaf(other.y, f1, l * f0);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 x = os[(t * 4 + i) * 64];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[t][4 * i + j] = fmaf(x[j], f1, o[t][4 * i + j] * f0);
      }
  }
  if (!live) return;
  // a lane holds dims 32 t + 8 i + 4 hf .. + 3
  if (a.splits > 1) {
    const int64_t at = (row * a.n_heads + head) * a.splits + split;
    if (hf == 0) {
      a.part_ml[2 * at] = m;
      a.part_ml[2 * at + 1] = l;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x4*>(a.part_o + at * DIM + 32 * t + 8 * i + 4 * hf) =
            f32x4{o[t][4 * i], o[t][4 * i + 1], o[t][4 * i + 2], o[t][4 * i + 3]};
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint2*>(out + 32 * t + 8 * i + 4 * hf) =
          make_uint2(pack_bf16x2(o[t][4 * i] * inv, o[t][4 * i + 1] * inv),
                     pack_bf16x2(o[t][4 * i + 2] * inv, o[t][4 * i + 3] * inv));
}

}  // namespace gqk
