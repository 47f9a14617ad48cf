// Attention of many new tokens per sequence over the paged key-value cache (BF16
// queries; gguf_attn_extend in include/gguf_tokens.h).
//
// A block takes 128 columns, (row, query head) pairs of one kv head, 32 per wave, and
// walks over the slots they see in tiles of 64 (32 past head dim 128), which its waves
// share in LDS:
//   S^T = K Q^T    32 x 32 tiles, A = K (rows: slots), B = Q (columns), in registers
//   O^T += V^T P^T A = V^T (rows: dims), B = P^T
// Transposed products leave a lane with one column throughout, so that the running
// maximum and sum are per-lane values (the two halves of the wave hold a column each
// half). K's rows lie in LDS with bits 2 and 3 of the slot swapped: the sixteen
// scores of a lane then are two runs of eight consecutive slots, which is the B operand
// of the second product as it stands, and V, stored transposed in the cache, is its A
// operand.
#pragma once

#include "attn.hpp"

namespace gqk {

struct AttnPromptArgs : AttnRowsArgs {
  int32_t tiles;   // tiles of columns of the grid
};

constexpr int kPromptColumns = 128;
constexpr int kPromptThreads = 256;
constexpr int kPromptWaves = 4;
// The maximum that weights are relative to is raised only where one exceeds it by a
// factor of 2^8: rescaling the output costs half as much as a tile's exponentials.
constexpr float kPromptSlack = 8.0f;

typedef float f32x16v __attribute__((ext_vector_type(16)));

template <int KIND>
__device__ __forceinline__ f32x16v prompt_mfma(const uint4& a, const uint4& b, const f32x16v& c) {
  if constexpr (KIND == kKvBF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8v, a), __builtin_bit_cast(bf16x8v, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

constexpr int prompt_slots(int dim) { return dim <= 128 ? 64 : 32; }   // of a tile

// Slots of a tile, and where its values lie in LDS: rows of 16-byte chunks, a chunk at
// chunk ^ swizzle(row), so that sixteen consecutive rows' chunks of one number lie in
// sixteen different groups of banks.
template <int NB>
struct PromptTile {
  static constexpr int kDim = NB * 32;
  static constexpr int kSlots = prompt_slots(kDim);
  static constexpr int kKChunks = kDim / 8;    // of a slot's row of K
  static constexpr int kVChunks = kSlots / 8;  // of a dim's row of V
  static constexpr int kBytes = kSlots * kDim * 2;
  static constexpr int kLoads = kBytes / (kPromptThreads * 16);   // 16-byte loads of a thread, K and V each
  __device__ static __forceinline__ int k_swizzle(int row) {
    return kKChunks % 16 == 0 ? row & 15 : kKChunks % 8 == 0 ? row >> 1 & 7 : row >> 2 & 3;
  }
  __device__ static __forceinline__ int v_swizzle(int row) { return kVChunks == 8 ? row >> 1 & 7 : row >> 2 & 3; }
};

// Slot (within 32) of row `r` of K in LDS, and back.
__device__ __forceinline__ int prompt_slot(int r) { return (r & ~12) | (r & 4) << 1 | (r & 8) >> 1; }

// Sixteen bytes per lane from global memory to 1 KiB of LDS at `lds` (uniform), lane by
// lane. Assembly, so that the compiler, which cannot tell which bytes of LDS are in
// flight, does not wait for all loads before each read of LDS; the caller waits. M0 is
// never live in compiled code here: only such loads of the compiler's own would set it.
__device__ __forceinline__ void prompt_load_lds(const uint8_t* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(base), "s"(lds)
               : "memory");
}
__device__ __forceinline__ void prompt_load_lds(const uint8_t* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(lds) : "memory");
}

template <int KIND, int NB>
__global__ __launch_bounds__(kPromptThreads, NB <= 6 ? 2 : 1) void attn_prompt_kernel(const AttnPromptArgs a) {
  using Tile = PromptTile<NB>;
  constexpr int DIM = Tile::kDim, T = Tile::kSlots, KC = Tile::kKChunks, VC = Tile::kVChunks, LOADS = Tile::kLoads;
  constexpr int KS = DIM / 16, NS = T / 32, NT = DIM / 32;   // steps of S, tiles of S, tiles of O
  constexpr int MM = KIND == kKvBF16 ? kKvBF16 : kKvF16;     // type of the products
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, hf = lane >> 5;
  const int h = blockIdx.x, split = blockIdx.z;
  // the last tiles of a sequence see most: they go first
  const RowTile rt = find_row_tile(a.row_start, a.n_seqs, a.n_rows, a.group, kPromptColumns, a.tiles - 1 - (int)blockIdx.y, lane);
  if (rt.seq < 0) return;
  const int s = rt.seq;
  const int held = (int)kv_length(a.lengths[s], a.max_len, a.table_stride, a.c.shift);
  const int width = rt.rows * a.group;
  const int unit = a.c.ps > T ? a.c.ps : T;
  const TileRange r = tile_range(held, rt.rows, a.group, rt.tile, kPromptColumns, a.window, a.sinks, unit);
  const int begin = split * a.chunk, end = r.n - begin < a.chunk ? r.n : begin + a.chunk;   // numbered without the gap
  const int c = rt.tile * kPromptColumns + wave * 32 + col;   // this lane's column
  const bool live = c < width;
  const int cc = live ? c : width - 1;
  const int64_t row = rt.row0 + cc / a.group;
  const int head = h * a.group + cc % a.group;
  uint16_t* const out = reinterpret_cast<uint16_t*>(a.out) + row * a.out_stride + (int64_t)head * DIM;
  if (begin >= r.n) {
    if (a.splits == 1 && live) {   // nothing seen
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

  // K and V of two tiles
  __shared__ __align__(1024) uint8_t lds[2][2][Tile::kBytes];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)&lds[0][0][0];

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
  // Whole tile in one page: offsets within a page are the same for every tile.
  const bool whole = a.c.ps >= T;
  uint32_t k_at[LOADS], v_at[LOADS];   // this lane's chunks: offset in the page's head, from the tile's slot on
  int k_slot[LOADS], v_slot[LOADS];    // and the slot in the tile
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int L = (wave * LOADS + i) * 64 + lane;
    const int kr = L / KC, kc = (L % KC) ^ Tile::k_swizzle(kr);
    k_slot[i] = (kr & ~31) | prompt_slot(kr & 31);
    k_at[i] = kc * 16;
    const int vr = L / VC, vc = (L % VC) ^ Tile::v_swizzle(vr);
    v_slot[i] = vc * 8;
    v_at[i] = vr * a.c.ps * 2;
  }
  auto issue = [&](int v0, int buf) {
    if (((v0 + T - 1) >> shift) - page0 >= 64) fetch_pages(v0 >> shift);
    const uint32_t to = lds0 + buf * 2 * Tile::kBytes + wave * LOADS * 1024;
    if (whole) {
      const int id = __builtin_amdgcn_readlane(pid, (v0 >> shift) - page0);
      const int64_t page = (id < 0 ? 0 : id) * page_bytes;
      const uint8_t* kb = kh + page + (v0 & smask) * (DIM * 2);
      const uint8_t* vb = vh + page + (v0 & smask) * 2;
#pragma unroll
      for (int i = 0; i < LOADS; ++i) prompt_load_lds(kb, k_at[i] + k_slot[i] * (DIM * 2), to + i * 1024);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) prompt_load_lds(vb, v_at[i] + v_slot[i] * 2, to + Tile::kBytes + i * 1024);
    } else {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int p = v0 + k_slot[i], id = __shfl(pid, (p >> shift) - page0);
        prompt_load_lds(kh + (id < 0 ? 0 : id) * page_bytes + (p & smask) * (DIM * 2) + k_at[i], to + i * 1024);
      }
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int p = v0 + v_slot[i], id = __shfl(pid, (p >> shift) - page0);
        prompt_load_lds(vh + (id < 0 ? 0 : id) * page_bytes + (p & smask) * 2 + v_at[i], to + Tile::kBytes + i * 1024);
      }
    }
  };
  // Slots of a tile whose values are looked at.
  auto present = [&](int v0) -> uint64_t {
    const int n = end - v0;
    uint64_t m = n >= 64 ? ~0ull : (1ull << n) - 1;
    if (T < 64) m &= (1ull << (T & 63)) - 1;
    for (int p = v0; p < v0 + T && p < end; p += a.c.ps) {
      const int id = __builtin_amdgcn_readlane(pid, (p >> shift) - page0);
      if (id < 0) m &= whole ? 0 : ~(((1ull << a.c.ps) - 1) << (p - v0));
    }
    return m;
  };

  fetch_pages(begin >> shift);
  int v0 = seen_from(begin);
  if (v0 < end) issue(v0, 0);

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
      // to fp16 (exact): the row's greatest magnitude goes to [512, 1024), what lies
      // 2^-34 of it and lower loses bits
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
  for (int k = 0; k < KS; ++k) k_off[k] = col * (DIM * 2) + (((2 * k + hf) ^ Tile::k_swizzle(col)) * 16);
#pragma unroll
  for (int k = 0; k < T / 16; ++k) v_off[k] = col * (T * 2) + (((2 * k + hf) ^ Tile::v_swizzle(col)) * 16);

  f32x16v o[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) o[t] = f32x16v{};
  float m = -__builtin_inff(), l = 0.f;

  for (int buf = 0; v0 < end; buf ^= 1) {
    // this tile's loads have arrived, everyone's; the other buffer is free
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    const int real0 = real_of(v0);
    const uint64_t here = present(v0);
    const int next = seen_from(v0 + T);
    if (next < end) issue(next, buf ^ 1);
    const bool whole_tile = here == (T < 64 ? (1ull << (T & 63)) - 1 : ~0ull);
    uint8_t* const kt = lds[buf][0];
    uint8_t* const vt = lds[buf][1];
    if (!whole_tile) {
      // V behind the end may hold anything: zero
      for (int i = tid; i < DIM * VC; i += kPromptThreads) {
        const int vr = i / VC, vc = (i % VC) ^ Tile::v_swizzle(vr);
        const uint32_t bits = (uint32_t)(here >> (8 * vc)) & 0xFFu;
        if (bits == 0xFFu) continue;
        uint16_t* p = reinterpret_cast<uint16_t*>(vt + i * 16);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!(bits >> j & 1)) p[j] = 0;
      }
      __syncthreads();
    }
    const bool none = idle || real0 >= w_hi || (real0 >= a.sinks && real0 + T <= wr.near);
    if (!none) {
      f32x16v sc[NS];
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        sc[n] = f32x16v{};
#pragma unroll
        for (int k = 0; k < KS; ++k) sc[n] = prompt_mfma<MM>(load16(kt + n * 32 * DIM * 2 + k_off[k]), q[k], sc[n]);
      }
      if (!(whole_tile && real0 >= wr.far && real0 + T <= wr.full)) {
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          const uint32_t bits = slot_bits(range, a.sinks, real0 + 32 * n) & (uint32_t)(here >> (32 * n));
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (!(bits >> ((i & 8) * 2 + 8 * hf + (i & 7)) & 1)) sc[n][i] = -__builtin_inff();
        }
      }
      float mx = sc[0][0];
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, sc[n][i]);
      mx = fmaxf(mx, __shfl_xor(mx, 32)) * factor;
      if (__any(mx > m + kPromptSlack)) {
        const float mn = fmaxf(m, mx);
        const float alpha = mn == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= alpha;
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t] *= alpha;
      }
      const float base = m == -__builtin_inff() ? 0.f : m;   // nothing seen yet
      uint4 p[T / 16];
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = __builtin_amdgcn_exp2f(fmaf(sc[n][8 * t + 2 * j], factor, -base));
            const float y = __builtin_amdgcn_exp2f(fmaf(sc[n][8 * t + 2 * j + 1], factor, -base));
            l += x + y;
            w[j] = MM == kKvBF16 ? pack_bf16x2(x, y) : __builtin_bit_cast(uint32_t, to_f16x2(x, y));
          }
          p[2 * n + t] = make_uint4(w[0], w[1], w[2], w[3]);
        }
#pragma unroll
      for (int k = 0; k < T / 16; ++k)
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t] = prompt_mfma<MM>(load16(vt + t * 32 * T * 2 + v_off[k]), p[k], o[t]);
    }
    v0 = next;
  }

  l += __shfl_xor(l, 32);
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
