// Attention of one new token per sequence over the paged key-value cache
// ("GGUF Inferencer in R", section 5.2.1, attend: softmax(q k^T / sqrt(d)) v),
// the cache's positions split over blocks and joined.
//
// A wave takes 32 positions at a time and up to 16 query heads of one kv head:
//   S^T = K Q^T   16 x 16 tiles, A = K (rows: positions), B = Q (columns: heads)
//   O^T += V^T P^T   A = V^T (rows: dims), B = P^T (columns: heads)
// Transposed products leave a lane with one head (its column) throughout: the
// running maximum, sum and rescale are per-lane values, and the lane's eight
// weights are already the B operand of the second product when the row of K
// that feeds row r of tile t is position 8 (r / 4) + 4 t + r % 4 (a lane of
// group g = lane / 16 then holds positions 8 g .. 8 g + 7). V is stored
// transposed, so those eight positions of a dim are one aligned load. Nothing
// goes through LDS but the join of a block's waves. The waves of a block take
// tiles in turn: two (Q8_0: four) of them then ask for a cache line of V at the
// same time (with ranges of their own instead they fetched it twice: 345 against
// 298 us for 1.1 GB; 64 positions per step of a Q8_0 cache took 256 registers
// and 85 against 70 us).
//
// The kernel reads each cache byte once: the bound is HBM (F16, 1.07 GB of 32
// ragged sequences in 200 us: 5.3 TB/s; tracked BF16, 0.27 GB in 67 us: 4.0;
// Q8_0, 0.23 GB in 60 us: 3.8, beside its conversions). The matrix cores
// run at a fraction of their rate (16 columns for n_heads / n_kv_heads heads,
// times two or three parts of the fp32 operand), which costs nothing here and
// keeps fp32 accuracy.
#pragma once

#include <type_traits>

#include "kv_cache.hpp"
#include "wave_ops.hpp"

namespace gqk {

struct AttnArgs {
  KvView c;
  const int32_t* table;
  const int32_t* lengths;
  const float* q;
  float* out;
  float* part_o;    // [n_seqs][n_heads][splits][dim], unnormalized (splits > 1)
  float* part_ml;   // [n_seqs][n_heads][splits][2]: maximum (log2 domain) and sum
  float* scores;    // [n_seqs][n_heads][score_stride] (track): log2-domain scores
  int64_t table_stride, q_stride, out_stride, max_len, window, score_stride;
  int32_t n_heads, group, head_tiles, splits, chunk, chunk_pages;
  float qscale;     // scale * log2(e)
  int32_t n_seqs;   // chunks by the lengths (share > 0): at most 64 sequences
  float share;      // chunk per position of all sequences together; 0: `chunk` for every call
};

constexpr int kAttnJ = 8;                 // positions of a lane
constexpr int kAttnTile = 4 * kAttnJ;     // and of a wave's step
constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = kAttnWaves * 64;
constexpr int kAttnLeast = 2 * kAttnTile * kAttnWaves;   // positions of the shortest chunk
constexpr float kPScaleF16 = 16384.0f;   // softmax weights enter fp16 times 2^14: 22 bits down to 2^-17 of the largest, then to 2^-39

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// First slot that a sequence's attention covers: a window counts slots, not cache positions.
__device__ __forceinline__ int attn_first(int n, int64_t window) {
  return window > 0 && (int64_t)n > window ? (int)(n - window) : 0;
}

// Positions per split. Host code knows a bound on the lengths only; where it
// leaves room (share > 0) the chunk is cut to the lengths there are, the same in
// every block: long enough for the launched splits to cover the longest
// sequence, and for all sequences to take about the blocks that run at once.
// All 64 lanes of a wave call it.
__device__ __forceinline__ int attn_chunk(const AttnArgs& a, int lane) {
  if (a.share == 0.f) return a.chunk;
  uint32_t span = 0;
  if (lane < a.n_seqs) {
    const int n = (int)kv_length(a.lengths[lane], a.max_len, a.table_stride, a.c.shift);
    span = (uint32_t)(n - (attn_first(n, a.window) & ~(kAttnTile - 1)));
  }
  uint32_t total = span, most = span;   // < 2^32: 64 spans of at most 2^25
  auto step = [&](uint32_t t, uint32_t m) {
    total += t;
    most = max_word(most, m);
  };
  step(dpp_word<0xB1>(total), dpp_word<0xB1>(most));
  step(dpp_word<0x4E>(total), dpp_word<0x4E>(most));
  step(dpp_word<0x141>(total), dpp_word<0x141>(most));
  step(dpp_word<0x140>(total), dpp_word<0x140>(most));
  total = lane_word(total, 0) + lane_word(total, 16) + lane_word(total, 32) + lane_word(total, 48);
  most = max_word(max_word(lane_word(most, 0), lane_word(most, 16)), max_word(lane_word(most, 32), lane_word(most, 48)));
  constexpr int kRound = kAttnTile * kAttnWaves;
  const float fair = (float)total * a.share;
  int c = fair < (float)a.chunk ? (int)fair + 1 : a.chunk;
  const int cover = ((int)most + a.splits - 1) / a.splits;
  c = c > cover ? c : cover;
  c = (c + kRound - 1) / kRound * kRound;
  c = c < kAttnLeast ? kAttnLeast : c;
  return c < a.chunk ? c : a.chunk;   // splits * a.chunk covers any length
}

// Two values rounded to fp16 (nearest-even), in one instruction.
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ f16x2 to_f16x2(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_convertvector((f32x2){a, b}, f16x2);
}

// Eight fp32 values as parts whose sum they are: three bf16 by truncation (8
// significant bits each: exact), or two fp16, which is two matrix products for
// three: 22 bits of magnitudes from 2^-3 on, smaller ones to 2^-25. Callers bring
// their greatest value near fp16's top first.
template <int KIND>
struct Parts {
  static constexpr int kN = KIND == kKvF16 ? 2 : 3;
  uint4 p[kN];
  __device__ __forceinline__ void set(const float (&x)[8]) {
    uint32_t w[kN][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = x[2 * j], b = x[2 * j + 1];
      if constexpr (KIND == kKvF16) {
        const f16x2 h = to_f16x2(a, b);
        w[0][j] = __builtin_bit_cast(uint32_t, h);
        w[1][j] = __builtin_bit_cast(uint32_t, to_f16x2(a - (float)h.x, b - (float)h.y));
      } else {
        const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
        const float ra = a - __uint_as_float(ua & 0xFFFF0000u), rb = b - __uint_as_float(ub & 0xFFFF0000u);
        const uint32_t va = __float_as_uint(ra), vb = __float_as_uint(rb);
        const float sa = ra - __uint_as_float(va & 0xFFFF0000u), sb = rb - __uint_as_float(vb & 0xFFFF0000u);
        // bytes 2, 3 of each word
        w[0][j] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
        w[1][j] = __builtin_amdgcn_perm(vb, va, 0x07060302u);
        w[2][j] = __builtin_amdgcn_perm(__float_as_uint(sb), __float_as_uint(sa), 0x07060302u);
      }
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) p[i] = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
  }
};

template <int KIND>
__device__ __forceinline__ f32x4 attn_mfma(const uint4& a, const uint4& b, const f32x4& c) {
  if constexpr (KIND == kKvF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8v, a), __builtin_bit_cast(bf16x8v, b), c,
                                                   0, 0, 0);
}

// Eight int8 codes as fp16 (exact): with the sign bit flipped a code is 0 .. 255,
// as the low byte of an fp16 between 1024 and 1279 (one unit per code).
__device__ __forceinline__ uint4 codes_f16(const uint2& q) {
  const f16x2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
  const uint32_t a = q.x ^ 0x80808080u, b = q.y ^ 0x80808080u;
  const uint32_t w[4] = {__builtin_amdgcn_perm(0x64646464u, a, 0x04010400u), __builtin_amdgcn_perm(0x64646464u, a, 0x04030402u),
                         __builtin_amdgcn_perm(0x64646464u, b, 0x04010400u), __builtin_amdgcn_perm(0x64646464u, b, 0x04030402u)};
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, w[j]) - off);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A wave's tile of K or V as loaded. Q8_0: the scales of a lane's eight positions
// (4 NB words, pairs of halves; K [position][block], V [block][position]) are
// the same for the 16 lanes of its group: lane c of the 16 holds words c and c +
// 16 (all of them in every lane took 30 registers more).
template <int KIND, int NB>
struct AttnK {
  uint4 x[2][KIND == kKvQ80 ? 1 : NB];
  uint2 c[2][KIND == kKvQ80 ? NB : 1];
  uint32_t d[(4 * NB + 15) / 16];
};
template <int KIND, int NB>
struct AttnV {
  uint4 x[KIND == kKvQ80 ? 1 : 2 * NB];
  uint2 c[KIND == kKvQ80 ? 2 * NB : 1];
  uint32_t d[(4 * NB + 15) / 16];
};

__device__ __forceinline__ uint4 load16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ uint2 load8(const uint8_t* p) { return *reinterpret_cast<const uint2*>(p); }

__device__ __forceinline__ uint32_t load4(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }

// The lanes' word I as an array of both halves, from the lane of the 16 that
// holds it (a broadcast within rows of 16 lanes).
template <int I, int N>
__device__ __forceinline__ uint32_t scale_word(const uint32_t (&d)[N]) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)d[I / 16], 0x150 + I % 16, 0xF, 0xF, true);
}
// fn(I, word I) for words I .. END - 1.
template <int I, int END, class Fn, int N>
__device__ __forceinline__ void each_scale(const uint32_t (&d)[N], Fn&& fn) {
  if constexpr (I < END) {
    fn(I, scale_word<I>(d));
    each_scale<I + 1, END>(d, fn);
  }
}

// fn(integral constant b) for blocks I .. END - 1.
template <int I, int END, class Fn>
__device__ __forceinline__ void each_block(Fn&& fn) {
  if constexpr (I < END) {
    fn(std::integral_constant<int, I>{});
    each_block<I + 1, END>(fn);
  }
}

// One block: a chunk of one sequence's positions, up to 16 query heads of one
// kv head; its waves take the chunk's tiles in turn and join in LDS.
template <int KIND, int NB, bool TRACK>
__global__ __launch_bounds__(kAttnThreads) void attn_decode_kernel(const AttnArgs a) {
  constexpr int DIM = NB * 32;
  constexpr int NT = 2 * NB;   // 16-dim tiles of the output
  constexpr int J = kAttnJ, TILE = kAttnTile, WORDS = 4 * NB, NW = (WORDS + 15) / 16;
  // operand parts: bf16 triples beside a BF16 cache, fp16 pairs otherwise
  constexpr int PART = KIND == kKvBF16 ? kKvBF16 : kKvF16;
  using Q = Parts<PART>;
  using P = Parts<PART>;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, g = lane >> 4;
  // Heads run fastest, splits slowest: consecutive blocks go to the eight XCDs
  // in turn, and with the splits fastest the empty ones behind the sequences'
  // ends would leave the same XCDs idle (8 splits, half of them empty: 315
  // instead of 190 us for 1 GB). The sequences move on by one from split to
  // split: with 4 heads a sequence would else keep to four XCDs, and the longer
  // ones wait for a second round (32 sequences of 1 .. 16384, 8 heads: 221 us,
  // with the turn 203; 64 of 0 .. 4096, 4 heads: 68.5, 66.5).
  const int split = blockIdx.z, s = (int)((blockIdx.y + blockIdx.z) % (uint32_t)a.n_seqs);
  const int h = blockIdx.x / a.head_tiles, ht = blockIdx.x % a.head_tiles;
  // The chunk's page ids, one per lane (a chunk spans at most 64 pages). Without
  // a window and with a chunk known beforehand they are asked for beside the
  // length, not behind it.
  const int32_t length = a.lengths[s];
  int32_t pid = 0;
  if (a.window == 0 && a.share == 0.f && lane < a.chunk_pages)
    pid = kv_page(a.table + (int64_t)s * a.table_stride, ((int64_t)split * a.chunk >> a.c.shift) + lane, a.table_stride,
                  a.c.n_pages);
  const int n = (int)kv_length(length, a.max_len, a.table_stride, a.c.shift);
  const int first = attn_first(n, a.window);
  const int base = first & ~(kAttnTile - 1);
  const int heads = a.group - ht * 16 < 16 ? a.group - ht * 16 : 16;   // valid columns
  const int head0 = h * a.group + ht * 16;
  // splits cover little more than 2^25 positions: no overflow
  if (base + split * (a.share == 0.f ? a.chunk : kAttnLeast) >= n) {
    // nothing here, whatever the chunk; a sequence without positions is zero
    // (with more splits than one the join writes it)
    if (a.splits == 1) {
      for (int i = tid; i < heads * DIM; i += kAttnThreads)
        a.out[(int64_t)s * a.out_stride + (int64_t)(head0 + i / DIM) * DIM + i % DIM] = 0.f;
    }
    return;
  }
  const int chunk = __builtin_amdgcn_readfirstlane(attn_chunk(a, lane));
  const int begin = base + split * chunk;
  if (begin >= n) return;   // not with one split
  const int end = n - begin < chunk ? n : begin + chunk;

  const int page0 = begin >> a.c.shift;
  const bool paged = page0 + lane <= (end - 1) >> a.c.shift;
  if ((a.window > 0 || a.share > 0.f) && paged)
    pid = kv_page(a.table + (int64_t)s * a.table_stride, page0 + lane, a.table_stride, a.c.n_pages);
  if (!paged) pid = 0;   // behind the sequence's last page: whatever the entry, not followed
  const bool any_bad = __any(pid < 0);

  const int k_row = J * (col >> 2) + (col & 3);   // + 4 t: the position in the tile of this lane's K row
  const uint8_t* const kh = a.c.k + (int64_t)h * a.c.head_bytes;
  const uint8_t* const vh = a.c.v + (int64_t)h * a.c.head_bytes;
  const int64_t page_bytes = (int64_t)a.c.hkv * a.c.head_bytes;
  const int smask = a.c.ps - 1;

  // Byte offset of the page of position `at` of tile t0 (page 0 for a bad one
  // and behind the sequence, whose values are then masked): the tile's one page,
  // or one per lane where pages are smaller than the tile.
  auto page_base = [&](int t0, int at) -> int64_t {
    const int local = (t0 >> a.c.shift) - page0;
    int id = __builtin_amdgcn_readlane(pid, local);
    if (a.c.ps < TILE) id = __shfl(pid, (((t0 + at) >> a.c.shift) - page0) & 63);
    return (id < 0 ? 0 : id) * page_bytes;
  };
  auto load_k = [&](AttnK<KIND, NB>& K, int t0) {
    const uint8_t* p = kh + page_base(t0, k_row);
#pragma unroll
    for (int t = 0; t < J / 4; ++t) {
      const int slot = (t0 + k_row + 4 * t) & smask;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if constexpr (KIND == kKvQ80) K.c[t][b] = load8(p + slot * DIM + b * 32 + 8 * g);
        else K.x[t][b] = load16(p + (slot * DIM + b * 32 + 8 * g) * 2);
      }
    }
    if constexpr (KIND == kKvQ80) {
      const uint8_t* dp = kh + page_base(t0, J * g) + a.c.ps * DIM + ((t0 + J * g) & smask) * (NB * 2);
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        const int w = col + 16 * j;
        K.d[j] = load4(dp + 4 * (w < WORDS ? w : 0));
      }
    }
  };
  auto load_v = [&](AttnV<KIND, NB>& V, int t0) {
    const uint8_t* p = vh + page_base(t0, J * g);
    const int slot = (t0 + J * g) & smask;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      if constexpr (KIND == kKvQ80) V.c[t] = load8(p + (t * 16 + col) * a.c.ps + slot);
      else V.x[t] = load16(p + ((t * 16 + col) * a.c.ps + slot) * 2);
    if constexpr (KIND == kKvQ80) {
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        const int w = col + 16 * j < WORDS ? col + 16 * j : 0;
        V.d[j] = load4(p + a.c.ps * DIM + ((w >> 2) * a.c.ps + slot) * 2 + (w & 3) * 4);
      }
    }
  };

  // Tiles of positions that all count, [t_lo, t_hi), run through a loop that
  // holds the next tile's loads in flight; the others (the window's first, the
  // last, and every one of a chunk with a bad page) behind it, masked.
  constexpr int step = TILE * kAttnWaves;
  const int mine = begin + wave * TILE;
  int t_lo = mine, t_hi = end & ~(TILE - 1);
  if (t_lo < first) t_lo += step;
  if (any_bad) t_hi = t_lo;
  AttnK<KIND, NB> K;
  AttnV<KIND, NB> V;
  if (t_lo < t_hi) {
    load_k(K, t_lo);
    load_v(V, t_lo);
  }

  // q of this lane's head: the B operand, dims 32 b + 8 g .. + 7
  Q q[NB];
  float sfac = 1.0f;   // undoes the row's power-of-two scale (fp16 parts)
  {
    float x[NB][8];
    const bool live = col < heads;
    const float* qp = a.q + (int64_t)s * a.q_stride + (int64_t)(head0 + (live ? col : 0)) * DIM + 8 * g;
    float amax = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float4 u = *reinterpret_cast<const float4*>(qp + 32 * b);
      const float4 v = *reinterpret_cast<const float4*>(qp + 32 * b + 4);
      const float y[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[b][j] = live ? y[j] * a.qscale : 0.f;
        amax = fmaxf(amax, fabsf(x[b][j]));
      }
    }
    if constexpr (PART == kKvF16) {
      // the row's largest magnitude to [512, 1024): 22 bits down to 2^-12 of it,
      // smaller elements to 2^-34 of it
      amax = fmaxf(amax, __shfl_xor(amax, 16));
      amax = fmaxf(amax, __shfl_xor(amax, 32));
      int e = 0;
      if (amax > 0.f && amax < __builtin_inff()) {
        (void)__builtin_frexpf(amax, &e);
        e = 10 - e < 100 ? 10 - e : 100;   // -118 at least: 2^-e is finite
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[b][j] = __builtin_ldexpf(x[b][j], e);
      sfac = __builtin_ldexpf(1.0f, -e);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) q[b].set(x[b]);
  }

  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  f32x4 o[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) o[t] = zero;
  float m = -__builtin_inff(), l = 0.f;   // of this lane's head; l over this lane's positions

  // Scores of positions t0 + J g + j of this lane's head, from the K loaded.
  auto scores = [&](const AttnK<KIND, NB>& K, float (&sc)[J]) {
    if constexpr (KIND == kKvQ80) {
      auto tile = [&](auto tt) {
        constexpr int t = decltype(tt)::value;
        f32x4 r[NB];   // per 32-dim block, before its scale
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint4 kc = codes_f16(K.c[t][b]);
          r[b] = zero;
#pragma unroll
          for (int i = Q::kN - 1; i >= 0; --i) r[b] = attn_mfma<PART>(kc, q[b].p[i], r[b]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[4 * t + i] = 0.f;
        each_scale<2 * NB * t, 2 * NB * (t + 1)>(K.d, [&](int w, uint32_t d) {
          const int j0 = 2 * w / NB, b0 = 2 * w % NB, j1 = (2 * w + 1) / NB, b1 = (2 * w + 1) % NB;
          sc[j0] = fmaf(r[b0][j0 & 3], half_lo(d), sc[j0]);
          sc[j1] = fmaf(r[b1][j1 & 3], half_hi(d), sc[j1]);
        });
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[4 * t + i] *= sfac;
      };
      tile(std::integral_constant<int, 0>{});
      tile(std::integral_constant<int, 1>{});
    } else {
#pragma unroll
      for (int t = 0; t < J / 4; ++t) {
        f32x4 acc = zero;
#pragma unroll
        for (int i = Q::kN - 1; i >= 0; --i)
#pragma unroll
          for (int b = 0; b < NB; ++b) acc = attn_mfma<PART>(K.x[t][b], q[b].p[i], acc);
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[4 * t + i] = acc[i] * sfac;
      }
    }
  };
  auto keep_scores = [&](int t0, const float (&sc)[J]) {
    if constexpr (TRACK) {
      if (col < heads) {
        float* sp = a.scores + ((int64_t)s * a.n_heads + head0 + col) * a.score_stride + t0 + J * g;
#pragma unroll
        for (int j = 0; j < J; j += 4)
          *reinterpret_cast<float4*>(sp + j) = make_float4(sc[j], sc[j + 1], sc[j + 2], sc[j + 3]);
      }
    }
  };
  // Running maximum and sum; p becomes the weights relative to the maximum.
  auto softmax = [&](const float (&sc)[J], float (&p)[J]) {
    float mx = sc[0];
#pragma unroll
    for (int j = 1; j < J; ++j) mx = fmaxf(mx, sc[j]);
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    if (__any(mx > m)) {
      const float mn = fmaxf(m, mx);
      const float alpha = __builtin_amdgcn_exp2f(m - mn);   // mn is finite where a position counts
      const float al = mn == -__builtin_inff() ? 1.0f : alpha;
      m = mn;
      l *= al;
#pragma unroll
      for (int t = 0; t < NT; ++t) o[t] *= al;
    }
    const float base = m == -__builtin_inff() ? 0.f : m;   // nothing seen yet
#pragma unroll
    for (int j = 0; j < J; ++j) {
      p[j] = __builtin_amdgcn_exp2f(sc[j] - base);
      l += p[j];
    }
  };
  // Weights enter fp16 times a power of two. F16: 2^14. Q8_0: a weight times its
  // position's scale d has any magnitude, so o of each 32-dim block b is kept in
  // units of 2^-(ks + e_b), with d 2^e_b (exact) and the product with the weight
  // 2^ks within fp16's range for every scale met so far. The greatest scale then
  // comes to [2^14, 2^15): products down to 2^-17 of it keep 22 bits, smaller ones
  // are off by at most 2^-39 of it. ks is one for all blocks and e_b at most 15, so
  // in a block far below the head's greatest scale that is 2^-54 of the latter (and
  // 2^-54 where no scale reaches 2). Three bf16 parts without units took 63 us for
  // 60 (8 sequences of 20001 .. 32768). A lane keeps e for the blocks of its scale
  // words, as the bits of the greatest scale e allows.
  int ks = 14, e[NW];
  uint32_t top[NW], most[NW], mul[NW];   // greatest scale met and allowed (bits), 2^e twice
#pragma unroll
  for (int j = 0; j < NW; ++j) {
    e[j] = 15;
    top[j] = most[j] = 0;
    mul[j] = 0x78007800u;
  }
  auto fit_scales = [&](const uint32_t (&d)[NW]) {
    bool over = false;
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      const uint32_t lo = d[j] & 0x7FFFu, hi = d[j] >> 16 & 0x7FFFu, mx = lo > hi ? lo : hi;
      over |= mx > most[j];
      top[j] = mx > top[j] ? mx : top[j];
    }
    if (!__any(over)) return;
    uint32_t all = 0;
#pragma unroll
    for (int j = 0; j < NW; ++j) {   // over the 16 lanes that share a block, then over all
      uint32_t t = top[j];
      t = max_word(t, dpp_word<0xB1>(t));
      t = max_word(t, dpp_word<0x4E>(t));
      t = max_word(t, (uint32_t)__shfl_xor((int)t, 16));
      top[j] = t = max_word(t, (uint32_t)__shfl_xor((int)t, 32));
      all = max_word(all, t);
    }
    all = max_word(all, (uint32_t)__shfl_xor((int)all, 4));
    all = max_word(all, (uint32_t)__shfl_xor((int)all, 8));
    // a scale with exponent field E lies below 2^(E - 14): E + e + ks <= 30, one
    // power of two to spare
    const int E = (int)(all >> 10), k = E >= 29 ? 0 : E <= 15 ? 14 : 29 - E;
    int grow[NW];
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      const int room = 29 - k - (int)(top[j] >> 10), n = room < 0 ? 0 : room > 15 ? 15 : room;
      grow[j] = k - ks + n - e[j];
      e[j] = n;
      const int last = 30 - k - n;   // greatest exponent field
      most[j] = last >= 30 ? 0x7FFFu : (uint32_t)last << 10 | 0x3FFu;
      mul[j] = 0x00010001u * (uint32_t)((15 + n) << 10);
    }
    ks = k;
    auto block = [&](auto bb) {
      constexpr int b = decltype(bb)::value;
      uint32_t by[NW];
#pragma unroll
      for (int j = 0; j < NW; ++j) by[j] = (uint32_t)grow[j];
      const float f = __builtin_ldexpf(1.0f, (int)scale_word<4 * b>(by));
      o[2 * b] *= f;
      o[2 * b + 1] *= f;
    };
    each_block<0, NB>(block);
  };
  // O^T += V^T P^T, from the V given.
  auto accumulate = [&](const AttnV<KIND, NB>& v, float (&p)[J]) {
    if constexpr (KIND == kKvQ80) {
      fit_scales(v.d);
      const float up = __builtin_ldexpf(1.0f, ks);
#pragma unroll
      for (int j = 0; j < J; ++j) p[j] *= up;
      uint32_t sd[NW];
#pragma unroll
      for (int j = 0; j < NW; ++j)
        sd[j] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, v.d[j]) * __builtin_bit_cast(f16x2, mul[j]));
      float pd[8];   // weights times scales: eight positions of a 32-dim block
      each_scale<0, WORDS>(sd, [&](int w, uint32_t d) {
        const int b = w / 4, j = 2 * (w % 4);
        pd[j] = fmaf(p[j], half_lo(d), 0.f);
        pd[j + 1] = fmaf(p[j + 1], half_hi(d), 0.f);
        if (w % 4 == 3) {
          P pp;
          pp.set(pd);
#pragma unroll
          for (int t = 2 * b; t < 2 * b + 2; ++t) {
            const uint4 vc = codes_f16(v.c[t]);
#pragma unroll
            for (int i = P::kN - 1; i >= 0; --i) o[t] = attn_mfma<PART>(vc, pp.p[i], o[t]);
          }
        }
      });
    } else {
      if constexpr (KIND == kKvF16) {
#pragma unroll
        for (int j = 0; j < J; ++j) p[j] *= kPScaleF16;
      }
      P pp;
      pp.set(p);
#pragma unroll
      for (int i = P::kN - 1; i >= 0; --i)
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t] = attn_mfma<PART>(v.x[t], pp.p[i], o[t]);
    }
  };

  for (int t0 = t_lo; t0 < t_hi; t0 += step) {
    float sc[J], p[J];
    scores(K, sc);
    const bool more = t0 + step < t_hi;   // uniform over the wave
    if (more) load_k(K, t0 + step);
    keep_scores(t0, sc);
    softmax(sc, p);
    accumulate(V, p);
    if (more) load_v(V, t0 + step);
  }
  for (int t0 = mine; t0 < end; t0 += step) {
    if (t0 >= t_lo && t0 < t_hi) continue;
    AttnK<KIND, NB> ek;
    AttnV<KIND, NB> ev;
    load_k(ek, t0);
    load_v(ev, t0);
    const int p0 = t0 + J * g;
    int hi = end - p0, lo = first - p0;
    hi = hi < 0 ? 0 : hi > J ? J : hi;
    lo = lo < 0 ? 0 : lo > J ? J : lo;
    uint32_t live = ((1u << hi) - 1u) & ~((1u << lo) - 1u);   // of the lane's positions
    if (any_bad && __shfl(pid, ((p0 >> a.c.shift) - page0) & 63) < 0) live = 0u;
    float sc[J], p[J];
    scores(ek, sc);
#pragma unroll
    for (int j = 0; j < J; ++j) sc[j] = (live >> j & 1) ? sc[j] : -__builtin_inff();
    keep_scores(t0, sc);
    softmax(sc, p);
    // V behind the length may hold anything: masked positions become 0 (Q8_0:
    // their scales; any code is finite)
    auto pair = [&](int i) { return ((live >> 2 * i & 1) ? 0xFFFFu : 0u) | ((live >> 2 * i & 2) ? 0xFFFF0000u : 0u); };
    AttnV<KIND, NB> mv = ev;
    if constexpr (KIND == kKvQ80) {
      const uint32_t mask = pair(col & 3);
#pragma unroll
      for (int j = 0; j < NW; ++j) mv.d[j] = ev.d[j] & mask;
    } else {
      const uint32_t w0 = pair(0), w1 = pair(1), w2 = pair(2), w3 = pair(3);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        mv.x[t] = make_uint4(ev.x[t].x & w0, ev.x[t].y & w1, ev.x[t].z & w2, ev.x[t].w & w3);
    }
    accumulate(mv, p);
  }
  if constexpr (KIND == kKvF16) {
#pragma unroll
    for (int t = 0; t < NT; ++t) o[t] *= 1.0f / kPScaleF16;
  }
  if constexpr (KIND == kKvQ80) {
    auto block = [&](auto bb) {
      constexpr int b = decltype(bb)::value;
      uint32_t by[NW];
#pragma unroll
      for (int j = 0; j < NW; ++j) by[j] = (uint32_t)-(ks + e[j]);
      const float f = __builtin_ldexpf(1.0f, (int)scale_word<4 * b>(by));
      o[2 * b] *= f;
      o[2 * b + 1] *= f;
    };
    each_block<0, NB>(block);
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);

  // Join of the waves, 32 dims at a time: [wave][head][32 + 4 floats].
  constexpr int kRow = 36;
  __shared__ __align__(16) float ml[kAttnWaves][16][2];
  __shared__ __align__(16) float part[kAttnWaves][16][kRow];
  if (lane < 16) {
    ml[wave][lane][0] = m;
    ml[wave][lane][1] = l;
  }
  __syncthreads();
  auto joined = [&](int c, float* wf) {   // weight of each wave, returns {M, L}
    float M = ml[0][c][0];
#pragma unroll
    for (int w = 1; w < kAttnWaves; ++w) M = fmaxf(M, ml[w][c][0]);
    const float base = M == -__builtin_inff() ? 0.f : M;
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      wf[w] = __builtin_amdgcn_exp2f(ml[w][c][0] - base);
      L = fmaf(ml[w][c][1], wf[w], L);
    }
    return make_float2(M, L);
  };
  const bool partial = a.splits > 1;
  if ((partial || TRACK) && tid < heads) {
    float wf[kAttnWaves];
    const float2 r = joined(tid, wf);
    float* d = a.part_ml + (((int64_t)s * a.n_heads + head0 + tid) * a.splits + split) * 2;
    d[0] = r.x;
    d[1] = r.y;
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
      *reinterpret_cast<f32x4*>(&part[wave][col][16 * t + 4 * g]) = o[2 * b + t];
    __syncthreads();
    for (int i = tid; i < heads * 8; i += kAttnThreads) {   // four dims each
      const int c = i >> 3, d4 = (i & 7) * 4;
      float wf[kAttnWaves];
      const float2 r = joined(c, wf);
      f32x4 sum = zero;
#pragma unroll
      for (int w = 0; w < kAttnWaves; ++w) sum += *reinterpret_cast<const f32x4*>(&part[w][c][d4]) * wf[w];
      if (partial) {
        *reinterpret_cast<f32x4*>(a.part_o + (((int64_t)s * a.n_heads + head0 + c) * a.splits + split) * DIM + 32 * b +
                                  d4) = sum;
      } else {
        const float inv = r.y == 0.f ? 0.f : 1.0f / r.y;   // no position left: zeros
        *reinterpret_cast<f32x4*>(a.out + (int64_t)s * a.out_stride + (int64_t)(head0 + c) * DIM + 32 * b + d4) =
            sum * inv;
      }
    }
    if (b + 1 < NB) __syncthreads();
  }
}

// Maximum and sum of one head over the splits that hold positions, by one wave;
// every lane returns them.
__device__ __forceinline__ float2 attn_join_ml(const float* ml, int splits, int lane) {
  const float2* p = reinterpret_cast<const float2*>(ml);
  const float2 own = lane < splits ? p[lane] : make_float2(-__builtin_inff(), 0.f);   // the usual whole of it
  float m = own.x;
  for (int i = lane + 64; i < splits; i += 64) m = fmaxf(m, p[i].x);
  m = wave_max(m);
  const float base = m == -__builtin_inff() ? 0.f : m;
  float l = own.y * __builtin_amdgcn_exp2f(own.x - base);
  for (int i = lane + 64; i < splits; i += 64) l = fmaf(p[i].y, __builtin_amdgcn_exp2f(p[i].x - base), l);
  return make_float2(base, wave_sum(l));
}

constexpr int kJoinThreads = 256;
constexpr int kWeightTile = 1024;   // positions per block of the weight update

// Blocks x < join_blocks: the joined output of query head x. The others: the
// weights of 1024 positions of one kv head, summed over its query heads in
// order (p = exp2(score - max) / sum) and added to the slots' weight.
template <int DIM>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(const AttnArgs a, int join_blocks, int weight_tiles) {
  constexpr int kLanes = DIM / 4;                    // float4 lanes of a row
  constexpr int kGroups = kJoinThreads / kLanes;     // splits in flight side by side
  const int s = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
  const int n = (int)kv_length(a.lengths[s], a.max_len, a.table_stride, a.c.shift);
  const int first = attn_first(n, a.window);
  const int base = first & ~(kAttnTile - 1);
  const int chunk = attn_chunk(a, lane);
  const int splits = n > base ? (n - base + chunk - 1) / chunk : 0;   // that wrote partials
  if ((int)blockIdx.x < join_blocks) {
    const int head = blockIdx.x;
    const int64_t row = (int64_t)s * a.n_heads + head;
    const float* ml = a.part_ml + row * a.splits * 2;
    __shared__ __align__(16) f32x4 part[kGroups][kLanes];
    const int c = tid % kLanes, grp = tid / kLanes;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    // the first partials are asked for before the maximum is known
    constexpr int kAhead = 4;
    const float* po = a.part_o + row * a.splits * DIM + c * 4;
    f32x4 v[kAhead];
    float vm[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = grp + u * kGroups, at = i < splits ? i : 0;   // loads without a branch between them
      v[u] = *reinterpret_cast<const f32x4*>(po + (int64_t)at * DIM);
      vm[u] = ml[2 * at];
    }
    const float2 r = attn_join_ml(ml, splits, lane);
    if (grp < kGroups) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (grp + u * kGroups < splits) sum += v[u] * __builtin_amdgcn_exp2f(vm[u] - r.x);
#pragma unroll 4
      for (int i = grp + kAhead * kGroups; i < splits; i += kGroups)
        sum += *reinterpret_cast<const f32x4*>(po + (int64_t)i * DIM) * __builtin_amdgcn_exp2f(ml[2 * i] - r.x);
      part[grp][c] = sum;
    }
    __syncthreads();
    if (tid < kLanes) {
      sum = part[0][tid];
#pragma unroll
      for (int i = 1; i < kGroups; ++i) sum += part[i][tid];
      const float inv = r.y == 0.f ? 0.f : 1.0f / r.y;
      *reinterpret_cast<f32x4*>(a.out + (int64_t)s * a.out_stride + (int64_t)head * DIM + tid * 4) = sum * inv;
    }
    return;
  }
  const int wb = blockIdx.x - join_blocks;
  const int h = wb / weight_tiles;
  const int p0 = base + (wb % weight_tiles) * kWeightTile;
  if (p0 >= n) return;
  __shared__ float2 hml[16];
  const int pos = p0 + tid * 4;
  const bool live = pos < n;
  // the slots and the first heads' scores are asked for before the maxima are known
  int32_t page = -1;
  float* w = nullptr;
  float4 old = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
    page = kv_page(a.table + (int64_t)s * a.table_stride, pos >> a.c.shift, a.table_stride, a.c.n_pages);
    w = a.c.weight + kv_slot_at(a.c, page < 0 ? 0 : page, h, pos & (a.c.ps - 1));
    old = *reinterpret_cast<const float4*>(w);
  }
  const float* sp = a.scores + ((int64_t)s * a.n_heads + h * a.group) * a.score_stride + pos;
  constexpr int kAhead = 4;
  float4 ahead[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (live && i < a.group) ahead[i] = *reinterpret_cast<const float4*>(sp + i * a.score_stride);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  auto add = [&](const float4& sc, const float2& r) {
    acc[0] = fmaf(__builtin_amdgcn_exp2f(sc.x - r.x), r.y, acc[0]);
    acc[1] = fmaf(__builtin_amdgcn_exp2f(sc.y - r.x), r.y, acc[1]);
    acc[2] = fmaf(__builtin_amdgcn_exp2f(sc.z - r.x), r.y, acc[2]);
    acc[3] = fmaf(__builtin_amdgcn_exp2f(sc.w - r.x), r.y, acc[3]);
  };
  for (int h0 = 0; h0 < a.group; h0 += 16) {
    const int hn = a.group - h0 < 16 ? a.group - h0 : 16;
    __syncthreads();
    for (int i = tid >> 6; i < hn; i += kJoinThreads / 64) {
      const float2 r = attn_join_ml(a.part_ml + ((int64_t)s * a.n_heads + h * a.group + h0 + i) * a.splits * 2, splits, lane);
      if (lane == 0) hml[i] = make_float2(r.x, r.y == 0.f ? 0.f : 1.0f / r.y);
    }
    __syncthreads();
    if (!live) continue;
    if (h0 == 0) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (i < hn) add(ahead[i], hml[i]);
    }
#pragma unroll 4
    for (int i = h0 == 0 ? kAhead : 0; i < hn; ++i)
      add(*reinterpret_cast<const float4*>(sp + (h0 + i) * a.score_stride), hml[i]);
  }
  if (page < 0) return;
  const float o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (pos + j >= first && pos + j < n) w[j] = o[j] + acc[j];
}

}  // namespace gqk
