// Log probabilities, entropy and top alternatives of rows of logits: one read
// of the logits, rows cut into splits of 8192 values (32 per thread, held in
// registers), the splits joined by a second launch.
//
// Per split: maximum m, l = sum e^(x - m), t = sum e^(x - m) (x - m), and the
// top k. With M, L, T the joined ones (T = sum of f (t + l (m - M)), f = e^(m -
// M)): log p_i = x_i - M - log L and the entropy is log L - T / L.
//
// The top k of a split: the k-th greatest of its lanes' maxima (of four lanes'
// for few alternatives) bounds its k-th value from below, and little more than k
// values reach that bound. They are put in order by counting, per value, the
// greater ones. Where ties make them too many to hold, or NaN is among the
// values, k block-wide maxima take their place; a split where fewer than k
// lanes (or fours of them) hold a value above -inf is such a case of ties (64 rows of 128256, top 20: 15 us with
// 99 % of the logits -inf, 234 with 99.9 %).
//
// Measured at a vocabulary of 128256: 1024 bf16 rows with the top 8 66 us for
// 263 MB (4.0 TB/s; 49 us without a top, 5.4 TB/s) and 6 us for the joins; 64
// fp32 rows 12 + 5 us, one row 5.3 + 4.1 (its dependent steps).
#pragma once

#include "wave_ops.hpp"

namespace gqk {

struct LogprobArgs {
  const uint8_t* x;
  const int32_t* tokens;
  float* token_lp;
  float* entropy;
  int32_t* top_id;
  float* top_lp;
  float* part;        // [n_rows][splits][4]: m, l, t
  uint64_t* cand;     // [n_rows][splits][top_k]: (key, ~index), greatest first
  int64_t n_rows, row_stride;
  int32_t vocab, n_tokens, top_k, splits;
};

constexpr int kLpThreads = 256;
constexpr int kLpWaves = kLpThreads / 64;
constexpr int kLpPer = 32;                          // values per thread
constexpr int kLpSplit = kLpThreads * kLpPer;
constexpr int kLpMaxTop = 64;
constexpr int kLpQuadTop = 16;                      // of four lanes' maxima up to here: 66 us, lanes' own 77 (1024 rows, top 8)
constexpr int kLpCand = 512;                        // values held for the ordering
constexpr int kLpWaveCand = kLpCand / kLpWaves;     // of one wave

// An unsigned key of a float's order: zeros of either sign equal, NaN greatest
// (and below all ones, so that no candidate is the greatest 64-bit value).
constexpr uint32_t kNanKey = 0xFFFFFFFEu;
__device__ __forceinline__ uint32_t logit_key(float x) {
  if (x != x) return kNanKey;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  if (k == kNanKey) return __builtin_nanf("");
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
// Greater value first, then lower index.
__device__ __forceinline__ uint64_t logit_order(uint32_t key, uint32_t index) {
  return (uint64_t)key << 32 | (uint32_t)~index;
}

__device__ __forceinline__ float lp_exp(float d) { return __builtin_amdgcn_exp2f(d * 1.44269504088896340736f); }

__device__ __forceinline__ uint64_t lp_wave_max_order(uint64_t v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const uint64_t o = __shfl_xor((unsigned long long)v, d);
    v = o > v ? o : v;
  }
  return v;
}

// Value `i` of a row's logits.
template <bool BF16>
__device__ __forceinline__ float lp_at(const uint8_t* row, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
  else return reinterpret_cast<const float*>(row)[i];
}

// The outputs of one row that follow from M, log L and T / L.
template <bool BF16>
__device__ __forceinline__ void lp_finish(const LogprobArgs& a, int64_t r, const uint8_t* row, float M, float L,
                                          float T, int tid) {
  const float logl = logf(L);
  if (tid == 0 && a.entropy) a.entropy[r] = logl - T / L;
  for (int j = tid; j < a.n_tokens; j += kLpThreads) {
    const int32_t t = a.tokens[r * a.n_tokens + j];
    a.token_lp[r * a.n_tokens + j] = t >= 0 && t < a.vocab ? (lp_at<BF16>(row, t) - M) - logl : -__builtin_inff();
  }
}

// Writes the greatest top_k of `count` candidates in LDS, in order: fn(rank, candidate).
template <class Fn>
__device__ __forceinline__ void lp_order(const uint64_t* cand, int count, int top_k, int tid, Fn&& fn) {
  for (int i = tid; i < count; i += kLpThreads) {
    const uint64_t c = cand[i];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += cand[j] > c;
    if (rank < top_k) fn(rank, c);
  }
}

template <bool BF16>
__global__ __launch_bounds__(kLpThreads) void logprobs_split_kernel(const LogprobArgs a) {
  constexpr int ES = BF16 ? 2 : 4, VE = 16 / ES, NV = kLpPer / VE;   // values per load, loads per thread
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int split = blockIdx.x;
  const int64_t r = (int64_t)blockIdx.y + (int64_t)blockIdx.z * gridDim.y;
  if (r >= a.n_rows) return;
  const uint8_t* row = a.x + r * a.row_stride * ES;
  // 16-byte words from the aligned address at or below the row's start; a word
  // that reaches outside the row is read value by value
  const int shift = (int)(reinterpret_cast<uintptr_t>(row) & 15) / ES;
  __shared__ float red[kLpWaves][3];
  __shared__ uint32_t maxima[kLpThreads];   // keys
  __shared__ int counts[kLpWaves];
  __shared__ uint64_t cand[kLpCand];
  float x[kLpPer];
  int idx0[NV];   // index of a word's first value
  uint4 words_in[NV];
  auto take = [&](int v) {
    const uint4& w = words_in[v];
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BF16) {
        x[v * VE + 2 * j] = __uint_as_float(u[j] << 16);
        x[v * VE + 2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
      } else {
        x[v * VE + j] = __uint_as_float(u[j]);
      }
    }
  };
  const int64_t start = (int64_t)split * kLpSplit - shift;   // of the split's first value
  const bool within = start >= 0 && start + kLpSplit <= a.vocab;
  if (within) {
    // all loads in flight before the first is used
    const uint4* p = reinterpret_cast<const uint4*>(row + start * ES) + tid;
#pragma unroll
    for (int v = 0; v < NV; ++v) words_in[v] = p[v * kLpThreads];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      idx0[v] = (int)start + (v * kLpThreads + tid) * VE;
      take(v);
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t first = start + (v * kLpThreads + tid) * VE;
      idx0[v] = first >= a.vocab ? a.vocab : (int)first;
      if (first >= 0 && first + VE <= a.vocab) words_in[v] = *reinterpret_cast<const uint4*>(row + first * ES);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int first = idx0[v];
      if (first >= 0 && first <= a.vocab - VE) {
        take(v);
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j)
          x[v * VE + j] = first + j >= 0 && first + j < a.vocab ? lp_at<BF16>(row, first + j) : -__builtin_inff();
      }
    }
  }
  float quad_max[kLpPer / 4], m = -__builtin_inff();   // maxima pass NaN over; the sums do not
#pragma unroll
  for (int i = 0; i < kLpPer / 4; ++i) {
    quad_max[i] = fmaxf(fmaxf(x[4 * i], x[4 * i + 1]), fmaxf(x[4 * i + 2], x[4 * i + 3]));
    m = fmaxf(m, quad_max[i]);
  }
  const float lane_max = m;
  m = wave_max(m);
  // Sums relative to the wave's own maximum: no barrier before the last value.
  float l = 0.f, t = 0.f;
  const float own = m == -__builtin_inff() ? 0.f : m;   // nothing but -inf: sums of 0
#pragma unroll
  for (int i = 0; i < kLpPer; ++i) {
    const float d = x[i] - own, e = lp_exp(d);
    l += e;
    t = fmaf(e, fmaxf(d, -1000.f), t);   // e is 0 there: 0 for -inf, too
  }
  l = wave_sum(l);
  t = wave_sum(t);
  if (lane == 0) {
    red[wave][0] = m;
    red[wave][1] = l;
    red[wave][2] = t;
  }
  // few alternatives of many values: the maxima of four lanes serve as well as
  // the lanes' own
  const bool quads = a.top_k <= kLpQuadTop && a.vocab - start >= kLpThreads / 2 * VE;
  if (a.top_k > 0) {
    if (quads) {
      float v = fmaxf(lane_max, dpp_float<0xB1>(lane_max));
      v = fmaxf(v, dpp_float<0x4E>(v));
      if ((lane & 3) == 0) maxima[tid >> 2] = logit_key(v);
    } else {
      maxima[tid] = logit_key(lane_max);
    }
  }
  __syncthreads();
  if (a.top_k > 0) {
    // the top 16 bits of the k-th greatest maximum, by bisection
    uint32_t bits = 0;
    if (quads) {
      const uint32_t v = maxima[lane];
#pragma unroll
      for (int bit = 31; bit >= 16; --bit) {
        const uint32_t trial = bits | 1u << bit;
        if (__popcll((unsigned long long)__ballot(v >= trial)) >= a.top_k) bits = trial;
      }
    } else {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = maxima[lane + 64 * i];
#pragma unroll
      for (int bit = 31; bit >= 16; --bit) {
        const uint32_t trial = bits | 1u << bit;
        int n = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) n += __popcll((unsigned long long)__ballot(v[i] >= trial));
        if (n >= a.top_k) bits = trial;
      }
    }
    // keys below the one of -inf (no maximum there) are NaN patterns
    const float low = bits < 0x00800000u ? -__builtin_inff() : key_logit(bits);
    // each wave's values at or above the bound, in a list of its own
    int n = 0;
    uint64_t* list = cand + wave * kLpWaveCand;   // (bits, index), not yet in order
#pragma unroll
    for (int q = 0; q < kLpPer / 4; ++q) {
      if (!__ballot(quad_max[q] >= low)) continue;
#pragma unroll
      for (int i = 4 * q; i < 4 * q + 4; ++i) {
        uint64_t at = __ballot(x[i] >= low);
        if (!at) continue;
        const int index = idx0[i / VE] + i % VE;
        if (!within) at &= __ballot(index >= 0 && index < a.vocab);   // not what fills up an edge split
        const int rank = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(at >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)at, 0));
        if ((at >> lane & 1) && rank < kLpWaveCand) list[rank] = (uint64_t)__float_as_uint(x[i]) << 32 | (uint32_t)index;
        n += __popcll((unsigned long long)at);
      }
    }
    if (lane == 0) counts[wave] = n;
    __syncthreads();
  }
  const bool whole = a.splits == 1;
  // the split's sums; the first wave needs them, and every wave where the row
  // ends here
  float nan_sum = 0.f;
#pragma unroll
  for (int w = 0; w < kLpWaves; ++w) nan_sum += red[w][1];
  float base = 0.f;
  if (wave == 0 || whole) {
    m = fmaxf(fmaxf(red[0][0], red[1][0]), fmaxf(red[2][0], red[3][0]));
    base = m == -__builtin_inff() ? 0.f : m;
    l = t = 0.f;
#pragma unroll
    for (int w = 0; w < kLpWaves; ++w) {
      const float wm = red[w][0], d = wm == -__builtin_inff() ? 0.f : wm - base, f = lp_exp(d);
      l = fmaf(f, red[w][1], l);
      t = fmaf(f, fmaf(red[w][1], fmaxf(d, -1000.f), red[w][2]), t);
    }
  }
  if (tid == 0 && !whole) *reinterpret_cast<float4*>(a.part + (r * a.splits + split) * 4) = make_float4(base, l, t, m);
  if (a.top_k > 0) {
    const float logl = whole ? logf(l) : 0.f;
    auto put = [&](int rank, uint64_t c) {
      if (whole) {
        a.top_id[r * a.top_k + rank] = (int32_t)~(uint32_t)c;
        a.top_lp[r * a.top_k + rank] = (key_logit((uint32_t)(c >> 32)) - m) - logl;
      } else {
        a.cand[(r * a.splits + split) * a.top_k + rank] = c;
      }
    };
    int have = 0;
    bool fits = nan_sum == nan_sum;   // NaN passed the maxima over
#pragma unroll
    for (int w = 0; w < kLpWaves; ++w) {
      have += counts[w];
      fits = fits && counts[w] <= kLpWaveCand;
    }
    if (fits) {
      if (have <= 64) {
        // one wave, a value per lane, read out lane by lane (66 us for 1024
        // rows; by the whole block out of LDS 81)
        if (wave == 0) {
          int w = 0, before = 0;
#pragma unroll
          for (int v = 0; v < kLpWaves - 1; ++v) {
            if (lane >= before + counts[v] && w == v) {
              before += counts[v];
              w = v + 1;
            }
          }
          uint64_t c = 0;
          if (lane < have) {
            const uint64_t v = cand[w * kLpWaveCand + lane - before];
            c = logit_order(logit_key(__uint_as_float((uint32_t)(v >> 32))), (uint32_t)v);
          }
          int rank = 0;
          for (int j = 0; j < have; ++j)
            rank += ((uint64_t)lane_word((uint32_t)(c >> 32), j) << 32 | lane_word((uint32_t)c, j)) > c;
          if (lane < have && rank < a.top_k) put(rank, c);
        }
      } else {
        for (int i = tid; i < kLpCand; i += kLpThreads) {
          const uint64_t v = cand[i];
          if (i % kLpWaveCand < counts[i / kLpWaveCand])
            cand[i] = logit_order(logit_key(__uint_as_float((uint32_t)(v >> 32))), (uint32_t)v);
        }
        __syncthreads();
        for (int i = tid; i < kLpCand; i += kLpThreads) {
          const int w = i / kLpWaveCand;
          if (i % kLpWaveCand >= counts[w]) continue;
          const uint64_t c = cand[i];
          int rank = 0;
          for (int v = 0; v < kLpWaves; ++v)
            for (int j = 0; j < counts[v]; ++j) rank += cand[v * kLpWaveCand + j] > c;
          if (rank < a.top_k) put(rank, c);
        }
      }
      // a split of fewer values than k
      if (!whole && tid >= have && tid < a.top_k) put(tid, 0);
    } else {
      // more ties than fit, or NaN: k times the greatest value below the last
      // one, the split read again for each
      const int64_t first = start < 0 ? 0 : start;
      const int64_t past = start + kLpSplit < a.vocab ? start + kLpSplit : a.vocab;
      uint64_t last = ~0ull;
      for (int k = 0; k < a.top_k; ++k) {
        uint64_t best = 0;
        for (int64_t i = first + tid; i < past; i += kLpThreads) {
          const uint64_t c = logit_order(logit_key(lp_at<BF16>(row, i)), (uint32_t)i);
          if (c < last && c > best) best = c;
        }
        best = lp_wave_max_order(best);
        __syncthreads();
        if (lane == 0) cand[wave] = best;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kLpWaves; ++w) best = cand[w] > best ? cand[w] : best;
        if (tid == 0) put(k, best);
        last = best;
      }
    }
  }
  if (whole) lp_finish<BF16>(a, r, row, m, l, t, tid);
}

// One block per row: joins the splits.
template <bool BF16>
__global__ __launch_bounds__(kLpThreads) void logprobs_join_kernel(const LogprobArgs a) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t r = (int64_t)blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
  if (r >= a.n_rows) return;
  // every wave joins the sums (splits are few), lanes over splits
  const float4* part = reinterpret_cast<const float4*>(a.part) + r * a.splits;
  float M = -__builtin_inff();
  for (int i = lane; i < a.splits; i += 64) M = fmaxf(M, part[i].w);
  M = wave_max(M);
  const float base = M == -__builtin_inff() ? 0.f : M;
  float L = 0.f, T = 0.f;
  for (int i = lane; i < a.splits; i += 64) {
    const float4 p = part[i];
    if (p.w == -__builtin_inff()) {   // no finite value, or NaN alone (l NaN)
      L += p.y;
      continue;
    }
    const float d = p.x - base, f = lp_exp(d);
    L += p.y * f;
    T += f > 0.f ? f * (p.z + p.y * d) : 0.f;
  }
  L = wave_sum(L);
  T = wave_sum(T);
  const uint8_t* row = a.x + r * a.row_stride * (BF16 ? 2 : 4);
  lp_finish<BF16>(a, r, row, M, L, T, tid);
  if (a.top_k == 0) return;
  const float logl = logf(L);
  // Candidates: the splits' lists, each in order. The q-th greatest of the
  // lists' r-th values, q r >= k, bounds the row's k-th value from below; r is
  // chosen to make q about half of the lists. What reaches the bound (a few
  // more than k) is put in order by counting.
  __shared__ uint64_t cand[kLpCand];
  __shared__ uint64_t best[kLpMaxTop];
  __shared__ uint64_t low;
  __shared__ int count;
  const uint64_t* lists = a.cand + r * a.splits * a.top_k;
  const int64_t total = (int64_t)a.splits * a.top_k;
  auto put = [&](int rank, uint64_t c) {
    a.top_id[r * a.top_k + rank] = (int32_t)~(uint32_t)c;
    a.top_lp[r * a.top_k + rank] = (key_logit((uint32_t)(c >> 32)) - M) - logl;
  };
  // (one read of every list: 5 us for 64 rows of 16 lists of 20, 36 in rounds)
  if (total <= 16 * kLpThreads) {
    uint64_t mine[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) mine[i] = tid + i * kLpThreads < total ? lists[tid + i * kLpThreads] : 0;
    const int heads = a.splits < 64 ? a.splits : 64;
    int at = (2 * a.top_k + heads - 1) / heads;   // r
    if (at > a.top_k) at = a.top_k;
    const int q = (a.top_k + at - 1) / at;        // <= heads: at >= 2 k / heads, or at = k
    if (tid == 0) {
      low = 0;
      count = 0;
    }
    if (tid < heads) cand[tid] = lists[(int64_t)tid * a.top_k + at - 1];
    __syncthreads();
    if (tid < heads) {
      const uint64_t c = cand[tid];
      int rank = 0;
      for (int j = 0; j < heads; ++j) rank += cand[j] > c;
      if (rank == q - 1 && c) low = c;   // values differ; 0 stands for a list too short
    }
    __syncthreads();
    const uint64_t bound = low;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (mine[i] && mine[i] >= bound) {
        const int w = atomicAdd(&count, 1);
        if (w < kLpCand) cand[w] = mine[i];
      }
    }
    __syncthreads();
    const int have = count;
    if (have <= kLpCand) {
      lp_order(cand, have, a.top_k, tid, put);
      return;
    }
    __syncthreads();
  }
  // too many to hold: in rounds that fit, the best so far ahead
  int held = 0;   // best so far, in cand[0 .. held)
  for (int64_t at = 0; at < total;) {
    const int64_t room = kLpCand - held;
    const int n = (int)(total - at < room ? total - at : room);
    for (int i = tid; i < n; i += kLpThreads) cand[held + i] = lists[at + i];
    __syncthreads();
    at += n;
    const int count = held + n;
    const bool done = at >= total;
    lp_order(cand, count, a.top_k, tid, [&](int rank, uint64_t c) {
      if (!done) best[rank] = c;
      else if (c) put(rank, c);
    });
    if (done) break;
    __syncthreads();
    // top_k candidates at least have been seen (a list holds top_k)
    if (tid < a.top_k) cand[tid] = best[tid];
    held = a.top_k;
    __syncthreads();
  }
}

}  // namespace gqk
