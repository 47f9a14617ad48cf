// Norms of queries and keys per head and the rotation by position, one pass:
//   y = w x / sqrt(mean(x^2) + eps),  (a, b) -> m (a cos t - b sin t, a sin t + b cos t)
// A block takes a few tokens: it first computes their cosines and sines, once for
// all heads (fp64 turns, so that far positions keep their angle: fp32 would lose
// 2^-24 of 131072 radians), into LDS; then groups of lanes take a head each. A lane
// holds whole pairs: two runs of VEC elements half a rotation apart, or adjacent ones.
//
// Bound: HBM, one read and one write of q and k. 8192 tokens of 32 + 8 heads of 128, bf16:
// 27 us with the rows in the Infinity Cache, 38 without (168 MB, 4.4 TB/s, as a copy of
// that size). 16 tokens: 5 us, a launch, the position and one row in turn.
#pragma once

#include "device_common.hpp"

namespace gqk {

struct RopeArgs {
  const uint8_t* in[2];    // q, k
  uint8_t* out[2];
  int64_t in_stride[2], out_stride[2];   // bytes
  const float* norm[2];
  int32_t heads[2];
  const double* freqs;
  const int32_t* axes;
  const int32_t* pos;
  int64_t pos_stride, n_tokens;
  int32_t n_axes, n_rot, head_dim, tokens, lanes;   // tokens per block, lanes per head (a power of two)
  float eps, magnitude;
};

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 512;
constexpr int kRopeAngles = 1024;   // cosine and sine pairs of a block

// VEC consecutive elements: 16 bytes, or one element.
template <bool BF16, int VEC>
struct RopeRun {
  float x[VEC];
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (VEC == 8) {
      const uint4 w = *reinterpret_cast<const uint4*>(p);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(u[j] << 16);
        x[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
      }
    } else if constexpr (VEC == 4) {
      const float4 w = *reinterpret_cast<const float4*>(p);
      x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
    } else if constexpr (BF16) {
      x[0] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16);
    } else {
      x[0] = *reinterpret_cast<const float*>(p);
    }
  }
  __device__ __forceinline__ void store(uint8_t* p) const {
    if constexpr (VEC == 8) {
      uint32_t u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
      *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else if constexpr (VEC == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    } else if constexpr (BF16) {
      *reinterpret_cast<uint16_t*>(p) = to_bf16(x[0]);
    } else {
      *reinterpret_cast<float*>(p) = x[0];
    }
  }
};

// The angle pos * freq in turns, without its whole ones: -1/2 .. 1/2. The roundings of the
// products are carried along: fp64 alone would lose 2^-21 of a radian at 2^31 radians.
__device__ __forceinline__ float rope_turn(double pos, double freq) {
#pragma clang fp contract(off)
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;   // 1 / (2 pi)
  const double x = pos * freq, dx = __builtin_fma(pos, freq, -x);
  const double t = x * kHi, dt = __builtin_fma(x, kHi, -t) + __builtin_fma(dx, kHi, x * kLo);
  return (float)((t - __builtin_rint(t)) + dt);
}

// A unit is two runs of VEC elements: within n_rot VEC pairs, behind it plain
// elements. UNITS per lane: 1 for runs of 16 bytes (head dims to 512 then take at
// most 64 lanes), 4 for single elements.
template <bool BF16, int VEC, bool HALVES>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(const RopeArgs a) {
  constexpr int ES = BF16 ? 2 : 4, UNITS = VEC == 1 ? 4 : 1;
  __shared__ float2 turn[kRopeAngles];   // [token][pair]
  const int tid = threadIdx.x, half = a.n_rot / 2;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int tokens = a.n_tokens - t0 < a.tokens ? (int)(a.n_tokens - t0) : a.tokens;
  for (int i = tid; i < tokens * half; i += kRopeThreads) {
    const int t = i / half, p = i - t * half;
    const int axis = a.axes ? a.axes[p] : 0;
    float2 cs = make_float2(1.f, 0.f);
    if (axis >= 0 && axis < a.n_axes)
      sincospif(2.0f * rope_turn((double)a.pos[axis * a.pos_stride + t0 + t], a.freqs[p]), &cs.y, &cs.x);
    turn[i] = make_float2(cs.x * a.magnitude, cs.y * a.magnitude);
  }
  __syncthreads();
  const int lanes = a.lanes, lane = tid & (lanes - 1), groups = kRopeThreads / lanes;
  const int heads = a.heads[0] + a.heads[1], units = a.head_dim / (2 * VEC), pairs = half / VEC;
  // where a unit's runs start
  auto runs = [&](int u, int& e0, int& e1) {
    if (u < pairs && HALVES) {
      e0 = u * VEC;
      e1 = e0 + half;
    } else {
      e0 = u * 2 * VEC;
      e1 = e0 + VEC;
    }
  };
  // every group makes the same number of rounds: the reductions below need whole groups
  const int rounds = (tokens * heads + groups - 1) / groups;
  for (int round = 0; round < rounds; ++round) {
    const int item = round * groups + tid / lanes;
    const bool live = item < tokens * heads;
    const int t = live ? item / heads : 0, hh = live ? item - t * heads : 0;
    const int which = hh < a.heads[0] ? 0 : 1, h = hh - (which ? a.heads[0] : 0);
    const int64_t head = (int64_t)h * a.head_dim * ES;
    const uint8_t* in = a.in[which] + (t0 + t) * a.in_stride[which] + head;
    uint8_t* out = a.out[which] + (t0 + t) * a.out_stride[which] + head;
    RopeRun<BF16, VEC> x0[UNITS], x1[UNITS];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int u = lane + i * lanes;
      if (!live || u >= units) continue;
      int e0, e1;
      runs(u, e0, e1);
      x0[i].load(in + e0 * ES);
      x1[i].load(in + e1 * ES);
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss = fmaf(x0[i].x[j], x0[i].x[j], fmaf(x1[i].x[j], x1[i].x[j], ss));
    }
    const float* w = a.norm[which];
    float f = 1.f;
    for (int m = lanes >> 1; m >= 1; m >>= 1) ss += __shfl_xor(ss, m);
    if (w) f = 1.0f / sqrtf(ss / (float)a.head_dim + a.eps);
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int u = lane + i * lanes;
      if (!live || u >= units) continue;
      int e0, e1;
      runs(u, e0, e1);
      if (w) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          x0[i].x[j] *= f * w[e0 + j];
          x1[i].x[j] *= f * w[e1 + j];
        }
      }
      if (u < pairs) {
        const float2* cs = turn + t * half;
        if constexpr (HALVES) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const float2 c = cs[u * VEC + j];
            const float p = x0[i].x[j], q = x1[i].x[j];
            x0[i].x[j] = fmaf(p, c.x, -(q * c.y));
            x1[i].x[j] = fmaf(p, c.y, q * c.x);
          }
        } else if constexpr (VEC == 1) {
          const float2 c = cs[u];
          const float p = x0[i].x[0], q = x1[i].x[0];
          x0[i].x[0] = fmaf(p, c.x, -(q * c.y));
          x1[i].x[0] = fmaf(p, c.y, q * c.x);
        } else {
          auto adjacent = [&](RopeRun<BF16, VEC>& r, int first) {
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) {
              const float2 c = cs[first + j];
              const float p = r.x[2 * j], q = r.x[2 * j + 1];
              r.x[2 * j] = fmaf(p, c.x, -(q * c.y));
              r.x[2 * j + 1] = fmaf(p, c.y, q * c.x);
            }
          };
          adjacent(x0[i], u * VEC);
          adjacent(x1[i], u * VEC + VEC / 2);
        }
      }
      x0[i].store(out + e0 * ES);
      x1[i].store(out + e1 * ES);
    }
  }
}

}  // namespace gqk
