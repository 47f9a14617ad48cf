// Verification of drafted tokens (gguf_verify_draft in include/gguf_tokens.h).
// Three launches over rows cut into splits of 8192 values:
//   sums    per split the maximum m and s = sum 2^((x - m) log2(e) / T) of target
//           and draft (T = 0: m and its lowest index);
//   choose  every block joins its sequence's splits (a few hundred values), finds the
//           first row that is not accepted and sums its split of what the next token
//           is drawn from, p or max(p - q, 0);
//   draw    one block per sequence finds the split, then the value, where the running
//           sum passes uniform * total.
// A draw is a whole number that must not depend on how sums are formed: with
// exponentials in fp32 (2^-22) a running sum over a vocabulary would cross a boundary
// that the exact one does not about once in 10^4 draws. Exponentials and sums are fp64
// instead, whose products run at fp32's rate here: a polynomial of degree 10.
#pragma once

#include "token_rows.hpp"
#include "wave_ops.hpp"

namespace gqk {

// The row that a sequence's next token is drawn from.
struct VerifyChoice {
  double mp, mq;   // maxima
  double ip, iq;   // 1 / sum (draws from p alone: 1)
  int64_t row;     // -1: nothing to draw (next is set already)
  int32_t mode;
  int32_t pad;
};
enum VerifyMode { kDrawP = 0, kDrawRest = 1, kDrawOneHot = 2 };   // p; p - q; p without the drafted token

struct VerifyArgs {
  const uint8_t* x[2];   // target, draft
  int64_t stride[2];     // elements
  const int32_t* tokens;
  const float* uniform;
  const float* uniform_next;
  const int32_t* row_start;
  const float* temperature;
  int32_t* accepted;
  int32_t* next;
  float* prob;
  double2* part;          // [2][n_rows][splits]: m, s (T = 0: m, index)
  VerifyChoice* choice;   // [n_seqs]
  double* rest;           // [n_seqs][splits]
  int64_t n_rows;
  int32_t n_seqs, vocab, splits;
};

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWaves = kVerifyThreads / 64;
constexpr int kVerifyPer = 32;
constexpr int kVerifySplit = kVerifyThreads * kVerifyPer;
constexpr int kVerifyAhead = 4;

// 2^z for z <= 0: 2^k 2^f with |f| <= 1/2 and the series of e^(f ln 2) to its tenth
// power (the next term is below 2^-42). -inf gives 0.
__device__ __forceinline__ double exp2_f64(double z) {
  z = z > -1100.0 ? z : -1100.0;
  const double k = __builtin_rint(z), f = z - k;
  double p = 7.0549116208011233e-9;   // ln(2)^n / n!, n = 10 .. 0
  p = fma(p, f, 1.0178086009239699e-7);
  p = fma(p, f, 1.3215486790144309e-6);
  p = fma(p, f, 1.5252733804059840e-5);
  p = fma(p, f, 1.5403530393381609e-4);
  p = fma(p, f, 1.3333558146428443e-3);
  p = fma(p, f, 9.6181291076284772e-3);
  p = fma(p, f, 5.5504108664821580e-2);
  p = fma(p, f, 2.4022650695910071e-1);
  p = fma(p, f, 6.9314718055994531e-1);
  p = fma(p, f, 1.0);
  return __builtin_ldexp(p, (int)k);
}

__device__ __forceinline__ double verify_temperature(const VerifyArgs& a, int seq) {
  const float t = a.temperature ? a.temperature[seq] : 1.0f;
  return t > 0.f ? (double)t : 0.0;
}
// log2(e) / T
__device__ __forceinline__ double verify_scale(double t) { return 1.4426950408889634074 / t; }

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ double wave_max_f64(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const double o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}

// max(p - q, 0) of two weights times their factors, each product rounded by itself:
// equal rows leave exactly nothing (as an fma the difference would be a rounding).
__device__ __forceinline__ double verify_rest(double p, double ip, double q, double iq) {
#pragma clang fp contract(off)
  const double r = p * ip - q * iq;
  return r > 0.0 ? r : 0.0;
}

template <bool BF16>
__device__ __forceinline__ float verify_at(const VerifyArgs& a, int which, int64_t row, int64_t i) {
  const int64_t at = row * a.stride[which] + i;
  if constexpr (BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.x[which])[at] << 16);
  else return reinterpret_cast<const float*>(a.x[which])[at];
}

// A thread's 32 values of a split. WIDE: in 16-byte words (rows aligned), else one by
// one; neighbouring threads hold neighbouring words. -inf behind the vocabulary.
template <bool BF16, bool WIDE>
struct VerifyValues {
  static constexpr int VE = !WIDE ? 1 : BF16 ? 8 : 4;
  float x[kVerifyPer];
  // index in the split of value j
  __device__ static __forceinline__ int index(int j, int tid) {
    return (j / VE * kVerifyThreads + tid) * VE + j % VE;
  }
  __device__ __forceinline__ void load(const VerifyArgs& a, int which, int64_t row, int split, int tid) {
    const int64_t first = (int64_t)split * kVerifySplit;
    const int left = a.vocab - first < kVerifySplit ? (int)(a.vocab - first) : kVerifySplit;
    const uint8_t* base = a.x[which] + (row * a.stride[which] + first) * (BF16 ? 2 : 4);
    if (WIDE && left == kVerifySplit) {
      uint4 w[kVerifyPer / VE];
#pragma unroll
      for (int v = 0; v < kVerifyPer / VE; ++v) w[v] = reinterpret_cast<const uint4*>(base)[v * kVerifyThreads + tid];
#pragma unroll
      for (int v = 0; v < kVerifyPer / VE; ++v) {
        const uint32_t u[4] = {w[v].x, w[v].y, w[v].z, w[v].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (BF16) {
            if constexpr (VE == 8) {
              x[8 * v + 2 * j] = __uint_as_float(u[j] << 16);
              x[8 * v + 2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
            }
          } else if constexpr (VE == 4) {
            x[4 * v + j] = __uint_as_float(u[j]);
          }
        }
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < kVerifyPer; ++j) {
      const int i = index(j, tid);
      x[j] = i < left ? verify_at<BF16>(a, which, row, first + i) : -__builtin_inff();
    }
  }
};

template <bool BF16, bool WIDE>
__global__ __launch_bounds__(kVerifyThreads) void verify_sums_kernel(const VerifyArgs a) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, which = blockIdx.y;
  const int64_t row = blockIdx.x / (uint32_t)a.splits;
  const int split = blockIdx.x % (uint32_t)a.splits;
  VerifyValues<BF16, WIDE> v;
  if (which == 0) v.load(a, 0, row, split, tid);   // in flight while the sequence is found
  const RowTile seq = find_row(a.row_start, a.n_seqs, a.n_rows, row, lane);
  if (seq.seq < 0) return;
  const double t = verify_temperature(a, seq.seq);
  if (which == 1) {
    if (t == 0.0 || row == seq.row0 + seq.rows - 1) return;   // not looked at
    v.load(a, 1, row, split, tid);
  }
  float m = -__builtin_inff();
  bool nan = false;
#pragma unroll
  for (int j = 0; j < kVerifyPer; ++j) {
    m = fmaxf(m, v.x[j]);
    nan |= v.x[j] != v.x[j];
  }
  __shared__ float wave_m[kVerifyWaves];
  __shared__ double wave_s[kVerifyWaves];
  m = wave_max(m);
  if (__any(nan)) m = __builtin_inff();   // no finite maximum either way
  if (lane == 0) wave_m[wave] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kVerifyWaves; ++w) m = fmaxf(m, wave_m[w]);
  double s = 0.0;
  if (t == 0.0) {
    int best = kVerifySplit;
#pragma unroll
    for (int j = kVerifyPer - 1; j >= 0; --j) {
      const int i = VerifyValues<BF16, WIDE>::index(j, tid);
      if (v.x[j] == m) best = i;   // a thread's indices ascend
    }
    s = -wave_max_f64(-(double)best);
  } else if (m > -__builtin_inff() && m < __builtin_inff()) {
    const double c = verify_scale(t), dm = (double)m;
#pragma unroll
    for (int j = 0; j < kVerifyPer; ++j) s += exp2_f64(((double)v.x[j] - dm) * c);
    s = wave_sum_f64(s);
  }
  if (lane == 0) wave_s[wave] = s;
  __syncthreads();
  if (tid != 0) return;
  if (t == 0.0) {
    for (int w = 1; w < kVerifyWaves; ++w) s = wave_s[w] < s ? wave_s[w] : s;
    s += (double)split * kVerifySplit;
  } else {
    for (int w = 1; w < kVerifyWaves; ++w) s += wave_s[w];
  }
  a.part[((int64_t)which * a.n_rows + row) * a.splits + split] = make_double2((double)m, s);
}

// Maximum and sum of a row over its splits (T > 0), by one wave; every lane returns
// them. The maximum is not finite for a row without a finite greatest logit.
__device__ __forceinline__ double2 verify_join(const VerifyArgs& a, int which, int64_t row, double c, int lane) {
  const double2* p = a.part + ((int64_t)which * a.n_rows + row) * a.splits;
  double m = -__builtin_inf();
  for (int i = lane; i < a.splits; i += 64) m = p[i].x > m ? p[i].x : m;
  m = wave_max_f64(m);
  double s = 0.0;
  for (int i = lane; i < a.splits; i += 64) s = fma(p[i].y, exp2_f64((p[i].x - m) * c), s);
  return make_double2(m, wave_sum_f64(s));
}
// The greatest value and its lowest index (T = 0).
__device__ __forceinline__ double2 verify_best(const VerifyArgs& a, int64_t row, int lane) {
  const double2* p = a.part + row * a.splits;
  double m = -__builtin_inf(), at = (double)a.vocab;
  for (int i = lane; i < a.splits; i += 64)
    if (p[i].x > m) m = p[i].x, at = p[i].y;
  const double top = wave_max_f64(m);
  return make_double2(top, -wave_max_f64(m == top ? -at : -(double)a.vocab));
}
__device__ __forceinline__ bool finite_f64(double v) { return v - v == 0.0; }

template <bool BF16, bool WIDE>
__global__ __launch_bounds__(kVerifyThreads) void verify_choose_kernel(const VerifyArgs a) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int s = blockIdx.y, split = blockIdx.x;
  const SeqRows seq = seq_rows(a.row_start, s, a.n_rows);
  if (seq.rows == 0) {
    if (split == 0 && tid == 0) {
      a.accepted[s] = 0;
      a.next[s] = -1;
      a.choice[s].row = -1;
    }
    return;
  }
  const double t = verify_temperature(a, s), c = t > 0.0 ? verify_scale(t) : 0.0;
  __shared__ int first_of[kVerifyWaves];
  __shared__ VerifyChoice chosen_of[kVerifyWaves];
  __shared__ int best_of[kVerifyWaves];
  __shared__ double sums[kVerifyWaves];
  // every wave takes rows in turn up to its first that is not accepted; the block
  // that writes accept_prob goes through all of them
  const bool writes = split == 0 && a.prob;
  int first = seq.rows;
  for (int j = wave; j < seq.rows; j += kVerifyWaves) {
    const int64_t row = (int64_t)seq.row0 + j;
    const bool last = j == seq.rows - 1;
    const int64_t token = last ? 0 : a.tokens[row];
    const bool known = token >= 0 && token < a.vocab;
    VerifyChoice ch;
    ch.mp = ch.mq = ch.ip = ch.iq = 0.0;
    ch.row = row;
    ch.mode = kDrawP;
    ch.pad = 0;
    int best = -1;
    bool ok = false;
    float prob = 0.f;
    if (t == 0.0) {
      const double2 b = verify_best(a, row, lane);
      best = finite_f64(b.x) ? (int)b.y : -1;
      ok = !last && best >= 0 && (int64_t)best == token;
      prob = (last && best >= 0) || ok ? 1.f : 0.f;
      ch.row = -1;
    } else {
      const double2 p = verify_join(a, 0, row, c, lane);
      bool valid = finite_f64(p.x);
      ch.mp = p.x;
      ch.ip = 1.0;
      if (last) {
        prob = valid ? 1.f : 0.f;
      } else {
        const double pt = valid && known ? exp2_f64(((double)verify_at<BF16>(a, 0, row, token) - p.x) * c) / p.y : 0.0;
        double qt = known ? 1.0 : 0.0;
        ch.mode = kDrawOneHot;
        if (a.x[1]) {
          const double2 q = verify_join(a, 1, row, c, lane);
          valid = valid && finite_f64(q.x);
          ch.mode = kDrawRest;
          ch.ip = 1.0 / p.y;
          ch.mq = q.x;
          ch.iq = 1.0 / q.y;
          qt = valid && known ? exp2_f64(((double)verify_at<BF16>(a, 1, row, token) - q.x) * c) / q.y : 0.0;
        }
        ok = valid && known && (double)a.uniform[row] * qt < pt;
        prob = !(valid && known) ? 0.f : pt >= qt ? (pt > 0.0 ? 1.f : 0.f) : (float)(pt / qt);
        if (ch.mode == kDrawOneHot && !known) ch.mode = kDrawP;
      }
      if (!valid) ch.row = -1;
    }
    if (writes && lane == 0) a.prob[row] = prob;
    if (!ok && j < first) {
      first = j;
      if (lane == 0) {
        chosen_of[wave] = ch;
        best_of[wave] = best;
      }
    }
    if (first < seq.rows && !writes) break;
  }
  if (lane == 0) first_of[wave] = first;
  __syncthreads();
  int at = 0;
#pragma unroll
  for (int w = 1; w < kVerifyWaves; ++w) at = first_of[w] < first_of[at] ? w : at;
  const VerifyChoice ch = chosen_of[at];
  if (split == 0 && tid == 0) {
    a.accepted[s] = first_of[at];
    a.next[s] = best_of[at];
    a.choice[s] = ch;
  }
  if (ch.row < 0) return;
  double* rest = a.rest + (int64_t)s * a.splits + split;
  if (ch.mode == kDrawP) {   // known from the sums
    if (tid == 0) {
      const double2 p = a.part[ch.row * a.splits + split];
      *rest = p.y * exp2_f64((p.x - ch.mp) * c);
    }
    return;
  }
  VerifyValues<BF16, WIDE> p, q;
  p.load(a, 0, ch.row, split, tid);
  double sum = 0.0;
  if (ch.mode == kDrawRest) {
    q.load(a, 1, ch.row, split, tid);
#pragma unroll kVerifyAhead
    for (int j = 0; j < kVerifyPer; ++j)
      sum += verify_rest(exp2_f64(((double)p.x[j] - ch.mp) * c), ch.ip, exp2_f64(((double)q.x[j] - ch.mq) * c), ch.iq);
  } else {
    const int token = a.tokens[ch.row] - split * kVerifySplit;
#pragma unroll kVerifyAhead
    for (int j = 0; j < kVerifyPer; ++j) {
      const double r = exp2_f64(((double)p.x[j] - ch.mp) * c);
      sum += VerifyValues<BF16, WIDE>::index(j, tid) == token ? 0.0 : r;
    }
  }
  sum = wave_sum_f64(sum);
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  if (tid == 0) *rest = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// What value i of the chosen row weighs.
template <bool BF16>
__device__ __forceinline__ double verify_weight(const VerifyArgs& a, const VerifyChoice& ch, double c, int64_t i) {
  const double p = exp2_f64(((double)verify_at<BF16>(a, 0, ch.row, i) - ch.mp) * c);
  if (ch.mode == kDrawRest)
    return verify_rest(p, ch.ip, exp2_f64(((double)verify_at<BF16>(a, 1, ch.row, i) - ch.mq) * c), ch.iq);
  return ch.mode == kDrawOneHot && i == a.tokens[ch.row] ? 0.0 : p;
}

template <bool BF16>
__global__ __launch_bounds__(kVerifyThreads) void verify_draw_kernel(const VerifyArgs a) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, s = blockIdx.x;
  VerifyChoice ch = a.choice[s];
  if (ch.row < 0) return;
  const double c = verify_scale(verify_temperature(a, s)), u = (double)a.uniform_next[s];
  const double* rest = a.rest + (int64_t)s * a.splits;
  const double2* part = a.part + ch.row * a.splits;
  // every thread runs through the splits' sums
  double total = 0.0;
  for (int i = 0; i < a.splits; ++i) total += rest[i];
  const bool all = !(total > 0.0) && ch.mode != kDrawP;   // p - q is nowhere above 0
  if (all) {
    ch.mode = kDrawP;
    ch.ip = 1.0;
    total = 0.0;
  }
  auto split_sum = [&](int i) { return all ? part[i].y * exp2_f64((part[i].x - ch.mp) * c) : rest[i]; };
  if (all)
    for (int i = 0; i < a.splits; ++i) total += split_sum(i);
  const double goal = u * total;
  double before = 0.0;
  int split = -1, last = 0;
  double last_before = 0.0;
  for (int i = 0; i < a.splits; ++i) {
    const double w = split_sum(i);
    if (w > 0.0) last = i, last_before = before;
    if (before + w > goal && split < 0) {
      split = i;
      break;
    }
    before += w;
  }
  if (split < 0) split = last, before = last_before;   // rounding at the very end
  const int64_t first = (int64_t)split * kVerifySplit + tid * kVerifyPer;
  const int n = a.vocab - first < kVerifyPer ? (int)(a.vocab - first < 0 ? 0 : a.vocab - first) : kVerifyPer;
  double sum = 0.0;
  int64_t tail = -1;   // last value with any weight
  for (int j = 0; j < n; ++j) {
    const double w = verify_weight<BF16>(a, ch, c, first + j);
    if (w > 0.0) tail = first + j;
    sum += w;
  }
  // exclusive sums over the threads, in order
  double upto = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_up(upto, d);
    if (lane >= d) upto += o;
  }
  __shared__ double wave_sum[kVerifyWaves];
  __shared__ int hit[kVerifyWaves], end[kVerifyWaves];
  if (lane == 63) wave_sum[wave] = upto;
  __syncthreads();
  double run = before;
  for (int w = 0; w < wave; ++w) run += wave_sum[w];
  const double reach = run + upto;
  run += upto - sum;
  int64_t found = -1;
  if (reach > goal) {
    for (int j = 0; j < n && found < 0; ++j) {
      const double w = verify_weight<BF16>(a, ch, c, first + j);
      run += w;
      if (w > 0.0 && run > goal) found = first + j;
    }
  }
  const uint64_t any = __ballot(found >= 0), ends = __ballot(tail >= 0);
  if (lane == 0) hit[wave] = any ? __builtin_ctzll(any) : -1, end[wave] = ends ? 63 - __builtin_clzll(ends) : -1;
  __syncthreads();
  int from = -1, to = -1;
  for (int w = kVerifyWaves - 1; w >= 0; --w) {
    if (hit[w] >= 0) from = w * 64 + hit[w];
    if (end[w] >= 0 && to < 0) to = w * 64 + end[w];
  }
  if (from >= 0 ? tid == from : tid == to) a.next[s] = (int32_t)(from >= 0 ? found : tail);
}

}  // namespace gqk
