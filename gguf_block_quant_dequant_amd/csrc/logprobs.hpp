// Log probabilities, entropy and top alternatives of rows of logits: one read
// of the logits, rows cut into splits of 8192 values (32 per thread, held in
// registers), the splits joined by a second launch.
//
// Per split: maximum m, l = sum e^(x - m), t = sum e^(x - m) (x - m), and the
// top k. With M, L, T the joined ones (T = sum of f (t + l (m - M)), f = e^(m -
// M)): log p_i = x_i - M - log L and the entropy is log L - T / L.
//
// The top k of a split: the least of the four waves' ceil(k / 4)-th greatest
// lane maxima bounds the split's k-th value from below; the values
// at or above that bound (about twice k of them on ordinary logits) are put in
// order by counting, per value, the greater ones. Where ties make them too
// many to hold, k block-wide maxima take their place.
#pragma once

#include "device_common.hpp"

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
constexpr int kLpCand = 512;                        // values held for the ordering

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

__device__ __forceinline__ float lp_wave_max(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
__device__ __forceinline__ float lp_wave_sum(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ uint32_t lp_wave_max_key(uint32_t v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const uint32_t o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}
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
  float x[kLpPer];
  int idx0[NV];   // index of a word's first value
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int64_t first = ((int64_t)split * (kLpSplit / VE) + v * kLpThreads + tid) * VE - shift;
    idx0[v] = first >= a.vocab ? a.vocab : (int)first;
    if (first >= 0 && first + VE <= a.vocab) {
      const uint4 w = *reinterpret_cast<const uint4*>(row + first * ES);
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
    } else {
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const int64_t i = first + j;
        x[v * VE + j] = i >= 0 && i < a.vocab ? lp_at<BF16>(row, i) : -__builtin_inff();
      }
    }
  }
  // waves whose every lane holds a value of the row; with none the split has
  // fewer than 64 words, all of which can be held
  const int64_t words = (a.vocab + shift + VE - 1) / VE - (int64_t)split * (kLpSplit / VE);
  const int full = words >= kLpThreads ? kLpWaves : words < 0 ? 0 : (int)(words / 64);
  __shared__ float red[kLpWaves][2];
  __shared__ uint32_t bound[kLpWaves];
  __shared__ int count;
  __shared__ uint64_t cand[kLpCand];
  float m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kLpPer; ++i) m = fmaxf(m, x[i]);
  uint32_t lane_key = 0;   // of this lane's maximum, NaN above all
  if (a.top_k > 0) {
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kLpPer; ++i) nan = nan || x[i] != x[i];
    lane_key = nan ? kNanKey : logit_key(m);
  }
  m = lp_wave_max(m);
  if (lane == 0) red[wave][0] = m;
  if (a.top_k > 0) {
    // the ceil(k / full)-th greatest lane maximum of this wave
    uint32_t k = lane_key, b = 0;
    const int need = full > 0 ? (a.top_k + full - 1) / full : 0;
    for (int i = 0; i < need; ++i) {
      b = lp_wave_max_key(k);
      const uint64_t at = __ballot(k == b);
      if (lane == __ffsll((unsigned long long)at) - 1) k = 0;
    }
    if (lane == 0) bound[wave] = b;
    if (tid == 0) count = 0;
  }
  __syncthreads();
  m = fmaxf(fmaxf(red[0][0], red[1][0]), fmaxf(red[2][0], red[3][0]));
  __syncthreads();
  const float base = m == -__builtin_inff() ? 0.f : m;   // nothing but -inf: sums of 0
  float l = 0.f, t = 0.f;
#pragma unroll
  for (int i = 0; i < kLpPer; ++i) {
    const float d = x[i] - base, e = lp_exp(d);
    l += e;
    t += e > 0.f ? e * d : 0.f;
  }
  l = lp_wave_sum(l);
  t = lp_wave_sum(t);
  if (lane == 0) {
    red[wave][0] = l;
    red[wave][1] = t;
  }
  uint32_t low = 0;
  if (a.top_k > 0) {
    low = full > 0 ? bound[0] : 0;
    for (int w = 1; w < full; ++w) low = bound[w] < low ? bound[w] : low;
    if (lane_key >= low) {
#pragma unroll
      for (int i = 0; i < kLpPer; ++i) {
        const int index = idx0[i / VE] + i % VE;
        const uint32_t key = logit_key(x[i]);
        if (key >= low && index >= 0 && index < a.vocab) {
          const int at = atomicAdd(&count, 1);
          if (at < kLpCand) cand[at] = logit_order(key, (uint32_t)index);
        }
      }
    }
  }
  __syncthreads();
  l = (red[0][0] + red[1][0]) + (red[2][0] + red[3][0]);
  t = (red[0][1] + red[1][1]) + (red[2][1] + red[3][1]);
  const bool whole = a.splits == 1;
  if (tid == 0 && !whole) *reinterpret_cast<float4*>(a.part + (r * a.splits + split) * 4) = make_float4(base, l, t, m);
  if (a.top_k > 0) {
    const float logl = logf(l);
    auto put = [&](int rank, uint64_t c) {
      if (whole) {
        a.top_id[r * a.top_k + rank] = (int32_t)~(uint32_t)c;
        a.top_lp[r * a.top_k + rank] = (key_logit((uint32_t)(c >> 32)) - m) - logl;
      } else {
        a.cand[(r * a.splits + split) * a.top_k + rank] = c;
      }
    };
    const int have = count;
    if (have <= kLpCand) {
      lp_order(cand, have, a.top_k, tid, put);
      // a split of fewer values than k
      if (!whole && tid >= have && tid < a.top_k) put(tid, 0);
    } else {
      // more ties than fit: k times the greatest value below the last one
      uint64_t last = ~0ull;
      for (int k = 0; k < a.top_k; ++k) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < kLpPer; ++i) {
          const int index = idx0[i / VE] + i % VE;
          const uint64_t c = index >= 0 && index < a.vocab ? logit_order(logit_key(x[i]), (uint32_t)index) : 0;
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
  M = lp_wave_max(M);
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
  L = lp_wave_sum(L);
  T = lp_wave_sum(T);
  const uint8_t* row = a.x + r * a.row_stride * (BF16 ? 2 : 4);
  lp_finish<BF16>(a, r, row, M, L, T, tid);
  if (a.top_k == 0) return;
  const float logl = logf(L);
  // Candidates: the splits' lists, in rounds that fit (the best so far ahead).
  __shared__ uint64_t cand[kLpCand];
  __shared__ uint64_t best[kLpMaxTop];
  const uint64_t* lists = a.cand + r * a.splits * a.top_k;
  const int64_t total = (int64_t)a.splits * a.top_k;
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
      else if (c) {
        a.top_id[r * a.top_k + rank] = (int32_t)~(uint32_t)c;
        a.top_lp[r * a.top_k + rank] = (key_logit((uint32_t)(c >> 32)) - M) - logl;
      }
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
