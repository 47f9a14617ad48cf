// Verification of drafted tokens (gguf_verify_draft in include/gguf_tokens.h).
// Three launches over rows cut into splits of 8192 values:
//   sums    per split the maximum m and s = sum 2^((x - m) log2(e) / T) of target
//           and draft (T = 0: m and its lowest index), from registers;
//   choose  every block joins the splits' sums of its sequence's rows, sixteen lanes to a
//           row of each side, finds the first row that is not accepted and sums its split
//           of what the next token is drawn from, p or max(p - q, 0);
//   draw    one block per sequence finds the split, then the value, where the running
//           sum passes uniform * total.
// A draw is a whole number that must not depend on how sums are formed: with
// exponentials in fp32 (2^-22) a running sum over a vocabulary would cross a boundary
// that the exact one does not about once in 10^4 draws. Exponentials and sums are fp64
// instead, whose products run at fp32's rate here.
//
// Bound: one read of the logits at large sizes, beside it the exponentials; three launches
// and their chains of loads at small ones. 32 sequences of 2 to 7 drafts over 128256 values, fp32,
// both sides: sums 43 us (180 MB, 4.2 TB/s; 33 without the exponentials, 49 with a
// polynomial of degree 10 in place of the table), choose 14 (18 with blocks of 1024 threads,
// whose registers let one of them run per CU), draw 11. One sequence of 4 drafts: 6, 5, 7.
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

constexpr int kVerifyThreads = 256;   // of the sums: 32 values each, all loads in flight
constexpr int kVerifyWaves = kVerifyThreads / 64;
constexpr int kVerifySplit = kVerifyThreads * 32;
constexpr int kChooseThreads = 512;   // 16 values each
constexpr int kDrawThreads = 1024;    // 8 values each: few blocks, whose latency counts
constexpr int kDrawWaves = kDrawThreads / 64;

// 2^(j / 32)
__device__ const double kVerifyPowers[32] = {
    1.0, 1.0218971486541166, 1.0442737824274138, 1.0671404006768237,
    1.0905077326652577, 1.1143867425958924, 1.1387886347566916, 1.1637248587775775,
    1.189207115002721, 1.215247359980469, 1.241857812073484, 1.2690509571917332,
    1.2968395546510096, 1.3252366431597413, 1.3542555469368927, 1.383909881963832,
    1.4142135623730951, 1.4451808069770467, 1.4768261459394993, 1.5091644275934228,
    1.5422108254079407, 1.5759808451078865, 1.6104903319492543, 1.645755478153965,
    1.681792830507429, 1.718619298122478, 1.7562521603732995, 1.7947090750031072,
    1.8340080864093424, 1.8741676341103, 1.9152065613971474, 1.9571441241754002};

// 2^z for z <= 0: 2^k 2^(j / 32) 2^r with |r| <= 1/64, k and j from the low bits of z + 1.5 2^47
// (whose last place is 1/32), 2^(j / 32) from `powers` (the 32 above in LDS: lanes read one
// address or different banks), 2^r from the series of e^(r ln 2) to its fifth power, that one
// economized by Chebyshev's T5 into the first and third. Off by 2^-43 at most. -inf gives 0.
__device__ __forceinline__ double exp2_f64(double z, const double* powers) {
  z = __builtin_fmax(z, -1100.0);
  const double t = z + 0x1.8p47, r = z - (t - 0x1.8p47);
  const int n = (int)(uint32_t)__builtin_bit_cast(uint64_t, t);
  double p = fma(9.618129107628477e-3, r, 5.5504515572724004e-2);
  p = fma(p, r, 2.4022650695910072e-1);
  p = fma(p, r, 6.931471805351096e-1);
  p = fma(p, r, 1.0);
  return __builtin_ldexp(p * powers[n & 31], n >> 5);
}
// `powers` of a block; the caller waits for the block.
__device__ __forceinline__ void load_powers(double* powers, int tid) {
  if (tid < 32) powers[tid] = kVerifyPowers[tid];
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

// A thread's values of a split. WIDE: in 16-byte words (rows aligned), else one by one;
// neighbouring threads hold neighbouring words. -inf behind the vocabulary.
template <bool BF16, bool WIDE, int THREADS>
struct VerifyValues {
  static constexpr int VE = !WIDE ? 1 : BF16 ? 8 : 4, PER = kVerifySplit / THREADS;
  float x[PER];
  // index in the split of value j
  __device__ static __forceinline__ int index(int j, int tid) { return (j / VE * THREADS + tid) * VE + j % VE; }
  __device__ __forceinline__ void load(const VerifyArgs& a, int which, int64_t row, int split, int tid) {
    const int64_t first = (int64_t)split * kVerifySplit;
    const int left = a.vocab - first < kVerifySplit ? (int)(a.vocab - first) : kVerifySplit;
    if constexpr (WIDE) {
      if (left == kVerifySplit) {
        const uint8_t* base = a.x[which] + (row * a.stride[which] + first) * (BF16 ? 2 : 4);
        uint4 w[PER / VE];
#pragma unroll
        for (int v = 0; v < PER / VE; ++v) w[v] = reinterpret_cast<const uint4*>(base)[v * THREADS + tid];
#pragma unroll
        for (int v = 0; v < PER / VE; ++v) {
          const uint32_t u[4] = {w[v].x, w[v].y, w[v].z, w[v].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (BF16) {
              x[8 * v + 2 * j] = __uint_as_float(u[j] << 16);
              x[8 * v + 2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
            } else {
              x[4 * v + j] = __uint_as_float(u[j]);
            }
          }
        }
        return;
      }
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
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
  using Values = VerifyValues<BF16, WIDE, kVerifyThreads>;
  Values v;
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
  for (int j = 0; j < Values::PER; ++j) {
    m = fmaxf(m, v.x[j]);
    nan |= v.x[j] != v.x[j];
  }
  __shared__ double powers[32];
  load_powers(powers, tid);
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
    for (int j = Values::PER - 1; j >= 0; --j) {
      const int i = Values::index(j, tid);
      if (v.x[j] == m) best = i;   // a thread's indices ascend
    }
    s = -wave_max_f64(-(double)best);
  } else if (m > -__builtin_inff() && m < __builtin_inff()) {
    const double c = verify_scale(t), dm = (double)m;
#pragma unroll
    for (int j = 0; j < Values::PER; ++j) s += exp2_f64(((double)v.x[j] - dm) * c, powers);
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

// Sixteen lanes' maximum and sum; every lane of them returns it.
__device__ __forceinline__ double row16_max(double v) {
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) {
    const double o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}
__device__ __forceinline__ double row16_sum(double v) {
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ bool finite_f64(double v) { return v - v == 0.0; }

// What became of one row.
struct VerifyRow {
  VerifyChoice choice;
  float prob;
  int32_t ok, best;
};

// First every block judges its sequence's rows, sixteen lanes for the target's sums of a
// row and sixteen for the draft's, 16 rows at a time; then it sums its split.
template <bool BF16, bool WIDE>
__global__ __launch_bounds__(kChooseThreads) void verify_choose_kernel(const VerifyArgs a) {
  using Values = VerifyValues<BF16, WIDE, kChooseThreads>;
  constexpr int kRows = kChooseThreads / 32;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = tid & 15;
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
  __shared__ double powers[32];
  load_powers(powers, tid);
  __shared__ VerifyRow judged[kRows];
  __shared__ double sums[kChooseThreads / 64];
  const bool writes = split == 0 && a.prob;   // goes through all rows
  int first = seq.rows;
  VerifyChoice ch;
  int best_token = -1;
  for (int j0 = 0; j0 < seq.rows && (first == seq.rows || writes); j0 += kRows) {
    __syncthreads();   // judged[] is free (powers[] is there)
    const int j = j0 + tid / 32, which = tid >> 4 & 1;
    const bool live = j < seq.rows;
    const int64_t row = (int64_t)seq.row0 + (live ? j : 0);
    const bool last = j == seq.rows - 1;
    const int64_t token = live && !last ? a.tokens[row] : -1;
    const bool known = token >= 0 && token < a.vocab;
    const bool use = live && (which == 0 || (a.x[1] && !last && t > 0.0));
    float logit = 0.f;
    if (use && known) logit = verify_at<BF16>(a, which, row, token);
    const double2* part = a.part + ((int64_t)which * a.n_rows + row) * a.splits;
    double m = -__builtin_inf(), at = (double)a.vocab;
    if (use) {
      for (int i = l16; i < a.splits; i += 16) {
        const double2 p = part[i];
        if (p.x > m) m = p.x, at = p.y;   // (T = 0: its lowest index; a lane's splits ascend)
      }
    }
    const double top = row16_max(m);
    double sum = 0.0;
    if (t == 0.0) {
      sum = -row16_max(m == top ? -at : -(double)a.vocab);
    } else {
      if (use)
        for (int i = l16; i < a.splits; i += 16) sum = fma(part[i].y, exp2_f64((part[i].x - top) * c, powers), sum);
      sum = row16_sum(sum);
    }
    const double share = use && known && t > 0.0 ? exp2_f64(((double)logit - top) * c, powers) / sum : 0.0;
    const double q_top = __shfl_xor(top, 16), q_sum = __shfl_xor(sum, 16), q_share = __shfl_xor(share, 16);
    if (live && which == 0 && l16 == 0) {
      VerifyRow r;
      r.choice.mp = top;
      r.choice.mq = r.choice.iq = 0.0;
      r.choice.ip = 1.0;
      r.choice.row = row;
      r.choice.mode = kDrawP;
      r.choice.pad = 0;
      r.best = -1;
      bool valid = finite_f64(top), ok = false;
      if (t == 0.0) {
        r.best = valid ? (int)sum : -1;
        ok = !last && valid && (int64_t)r.best == token;
        r.prob = (last && valid) || ok ? 1.f : 0.f;
        valid = false;   // nothing to draw
      } else if (last) {
        r.prob = valid ? 1.f : 0.f;
      } else {
        double qt = known ? 1.0 : 0.0;
        if (a.x[1]) {
          valid = valid && finite_f64(q_top);
          r.choice.mode = kDrawRest;
          r.choice.ip = 1.0 / sum;
          r.choice.mq = q_top;
          r.choice.iq = 1.0 / q_sum;
          qt = q_share;
        } else if (known) {
          r.choice.mode = kDrawOneHot;
        }
        ok = valid && known && (double)a.uniform[row] * qt < share;
        r.prob = !(valid && known) ? 0.f : share >= qt ? (share > 0.0 ? 1.f : 0.f) : (float)(share / qt);
      }
      if (!valid) r.choice.row = -1;
      r.ok = ok;
      judged[j - j0] = r;
      if (writes) a.prob[row] = r.prob;
    }
    __syncthreads();
    if (first == seq.rows) {
      const int n = seq.rows - j0 < kRows ? seq.rows - j0 : kRows;
      const uint64_t refused = __ballot(lane < n && !judged[lane < n ? lane : 0].ok);
      if (refused) {
        const int at0 = __builtin_ctzll(refused);
        first = j0 + at0;
        ch = judged[at0].choice;
        best_token = judged[at0].best;
      }
    }
  }
  if (split == 0 && tid == 0) {
    a.accepted[s] = first;
    a.next[s] = best_token;
    a.choice[s] = ch;
  }
  if (ch.row < 0) return;
  double* rest = a.rest + (int64_t)s * a.splits + split;
  if (ch.mode == kDrawP) {   // known from the sums
    if (tid == 0) {
      const double2 p = a.part[ch.row * a.splits + split];
      *rest = p.y * exp2_f64((p.x - ch.mp) * c, powers);
    }
    return;
  }
  Values p, q;
  p.load(a, 0, ch.row, split, tid);
  double sum = 0.0;
  if (ch.mode == kDrawRest) {
    q.load(a, 1, ch.row, split, tid);
#pragma unroll
    for (int j = 0; j < Values::PER; ++j)
      sum += verify_rest(exp2_f64(((double)p.x[j] - ch.mp) * c, powers), ch.ip, exp2_f64(((double)q.x[j] - ch.mq) * c, powers), ch.iq);
  } else {
    const int token = a.tokens[ch.row] - split * kVerifySplit;
#pragma unroll
    for (int j = 0; j < Values::PER; ++j) {
      const double r = exp2_f64(((double)p.x[j] - ch.mp) * c, powers);
      sum += Values::index(j, tid) == token ? 0.0 : r;
    }
  }
  sum = wave_sum_f64(sum);
  if (lane == 0) sums[wave] = sum;
  __syncthreads();
  if (tid == 0) {
    sum = 0.0;
    for (int w = 0; w < kChooseThreads / 64; ++w) sum += sums[w];
    *rest = sum;
  }
}

// What value i of the chosen row weighs, its logits given.
__device__ __forceinline__ double verify_weight(const VerifyArgs& a, const VerifyChoice& ch, double c, float x, float y,
                                                bool token, const double* powers) {
  const double p = exp2_f64(((double)x - ch.mp) * c, powers);
  if (ch.mode == kDrawRest) return verify_rest(p, ch.ip, exp2_f64(((double)y - ch.mq) * c, powers), ch.iq);
  return ch.mode == kDrawOneHot && token ? 0.0 : p;
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ double wave_scan_f64(double v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

template <bool BF16, bool WIDE>
__global__ __launch_bounds__(kDrawThreads) void verify_draw_kernel(const VerifyArgs a) {
  using Values = VerifyValues<BF16, WIDE, kDrawThreads>;
  constexpr int PER = Values::PER;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, s = blockIdx.x;
  // everything that is at a known place is asked for at once, before any of it is looked at
  const double* rest = a.rest + (int64_t)s * a.splits;
  const double rest0 = lane < a.splits ? rest[lane] : 0.0;
  const double t = verify_temperature(a, s), u = (double)a.uniform_next[s];
  VerifyChoice ch = a.choice[s];
  __shared__ double powers[32];
  load_powers(powers, tid);
  __syncthreads();
  if (ch.row < 0) return;
  const double c = verify_scale(t);
  const int64_t refused = ch.mode == kDrawOneHot ? a.tokens[ch.row] : -1;
  const double2* part = a.part + ch.row * a.splits;
  bool all = false;   // p - q is nowhere above 0: from p
  auto split_sum = [&](int i) -> double {
    if (i >= a.splits) return 0.0;
    if (all) return part[i].y * exp2_f64((part[i].x - ch.mp) * c, powers);
    return i < 64 ? rest0 : rest[i];   // (i % 64 is the lane)
  };
  // every wave goes through the splits' sums, 64 at a time
  auto whole = [&]() {
    double sum = 0.0;
    for (int i = 0; i < a.splits; i += 64) sum += wave_sum_f64(split_sum(i + lane));
    return sum;
  };
  double total = whole();
  if (!(total > 0.0) && ch.mode != kDrawP) {
    all = true;
    ch.mode = kDrawP;
    total = whole();
  }
  const double goal = u * total;
  double before = 0.0, run = 0.0, last_before = 0.0;
  int split = -1, last = 0;
  for (int i = 0; i < a.splits && split < 0; i += 64) {
    const double w = split_sum(i + lane), upto = wave_scan_f64(w, lane);
    const uint64_t hit = __ballot(run + upto > goal && w > 0.0), any = __ballot(w > 0.0);
    if (hit) {
      split = i + __builtin_ctzll(hit);
      before = run + __shfl(upto - w, __builtin_ctzll(hit));
    }
    if (any) {
      const int at = 63 - __builtin_clzll(any);
      last = i + at;
      last_before = run + __shfl(upto - w, at);
    }
    run += __shfl(upto, 63);
  }
  if (split < 0) split = last, before = last_before;   // rounding at the very end
  // The split's logits in LDS, in order: thread t weighs values PER t .. (a word of pad per PER).
  __shared__ float logits[2][kVerifySplit + kVerifySplit / PER];
  const bool two = ch.mode == kDrawRest;
  Values p, q;
  p.load(a, 0, ch.row, split, tid);
  if (two) q.load(a, 1, ch.row, split, tid);
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = Values::index(j, tid);
    logits[0][i + i / PER] = p.x[j];
    if (two) logits[1][i + i / PER] = q.x[j];
  }
  __syncthreads();
  const int64_t token = refused - (int64_t)split * kVerifySplit;
  double w[PER], sum = 0.0;
  int tail = -1;   // last value with any weight
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = tid * PER + j, at = i + i / PER;
    w[j] = verify_weight(a, ch, c, logits[0][at], two ? logits[1][at] : 0.f, i == token, powers);
    if (w[j] > 0.0) tail = j;
    sum += w[j];
  }
  const double upto = wave_scan_f64(sum, lane);
  __shared__ double wave_sum[kDrawWaves];
  __shared__ int hit[kDrawWaves], end[kDrawWaves];
  if (lane == 63) wave_sum[wave] = upto;
  __syncthreads();
  run = before;
  for (int v = 0; v < wave; ++v) run += wave_sum[v];
  const bool reached = run + upto > goal;
  run += upto - sum;
  int found = -1;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    run += w[j];
    if (found < 0 && reached && w[j] > 0.0 && run > goal) found = j;
  }
  const uint64_t any = __ballot(found >= 0), ends = __ballot(tail >= 0);
  if (lane == 0) hit[wave] = any ? __builtin_ctzll(any) : -1, end[wave] = ends ? 63 - __builtin_clzll(ends) : -1;
  __syncthreads();
  int from = -1, to = -1;
  for (int v = kDrawWaves - 1; v >= 0; --v) {
    if (hit[v] >= 0) from = v * 64 + hit[v];
    if (end[v] >= 0 && to < 0) to = v * 64 + end[v];
  }
  if (from >= 0 ? tid == from : tid == to) a.next[s] = split * kVerifySplit + tid * PER + (from >= 0 ? found : tail);
}

}  // namespace gqk
