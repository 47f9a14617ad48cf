// Reductions over the 64 lanes of a wave: four data-parallel-primitive steps
// within each row of 16 lanes, then the four rows through scalar registers.
// Every lane returns the result; the order of the sums is fixed. All 64 lanes
// have to be active.
#pragma once

#include "device_common.hpp"

namespace gqk {

// The value of the lane that a DPP control names: 0xB1 and 0x4E swap
// neighbours and pairs, 0x141 and 0x140 mirror 8 and 16 lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_word(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp_float(float v) {
  return __uint_as_float(dpp_word<CTRL>(__float_as_uint(v)));
}
__device__ __forceinline__ float lane_float(float v, int lane) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), lane));
}
__device__ __forceinline__ uint32_t lane_word(uint32_t v, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp_float<0xB1>(v));
  v = fmaxf(v, dpp_float<0x4E>(v));
  v = fmaxf(v, dpp_float<0x141>(v));
  v = fmaxf(v, dpp_float<0x140>(v));
  return fmaxf(fmaxf(lane_float(v, 0), lane_float(v, 16)), fmaxf(lane_float(v, 32), lane_float(v, 48)));
}

__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_float<0xB1>(v);
  v += dpp_float<0x4E>(v);
  v += dpp_float<0x141>(v);
  v += dpp_float<0x140>(v);
  return (lane_float(v, 0) + lane_float(v, 16)) + (lane_float(v, 32) + lane_float(v, 48));
}

__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) { return a > b ? a : b; }

}  // namespace gqk
