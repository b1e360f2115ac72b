// qmm_lanes.h -- exchanges and reductions between the lanes of a wave.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmm {

__device__ __forceinline__ float shfl_xor(float v, int m) { return __shfl_xor(v, m); }
__device__ __forceinline__ uint32_t shfl_xor(uint32_t v, int m) { return (uint32_t)__shfl_xor((int)v, m); }
__device__ __forceinline__ double shfl_xor(double v, int m) {
  const int2 a = __builtin_bit_cast(int2, v);
  return __builtin_bit_cast(double, int2{__shfl_xor(a.x, m), __shfl_xor(a.y, m)});
}

// Reductions over every L = 8, 16, 32 or 64 neighbouring lanes, the result on each
// of them (the same bits on all, where f is commutative: every lane joins the same
// pairs).
// Within a DPP row of 16: neighbours, pairs (quad_perm), the two quads (half
// mirror), the two halves (mirror); its four through scalars.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);  // every source lane is there
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) { return __uint_as_float(dpp<CTRL>(__float_as_uint(v))); }
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint2 a = __builtin_bit_cast(uint2, v);
  return __builtin_bit_cast(double, uint2{dpp<CTRL>(a.x), dpp<CTRL>(a.y)});
}
__device__ __forceinline__ uint32_t lane_of(uint32_t v, int i) { return __builtin_amdgcn_readlane(v, i); }
__device__ __forceinline__ float lane_of(float v, int i) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), i)); }
__device__ __forceinline__ double lane_of(double v, int i) {
  const uint2 a = __builtin_bit_cast(uint2, v);
  return __builtin_bit_cast(double, uint2{(uint32_t)__builtin_amdgcn_readlane(a.x, i), (uint32_t)__builtin_amdgcn_readlane(a.y, i)});
}
template <int L, typename T, typename F>
__device__ __forceinline__ T reduce(T v, F f) {
  v = f(v, dpp<0xB1>(v));
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x141>(v));
  if constexpr (L >= 16) v = f(v, dpp<0x140>(v));
  if constexpr (L == 32) v = f(v, shfl_xor(v, 16));
  if constexpr (L == 64) v = f(f(lane_of(v, 0), lane_of(v, 16)), f(lane_of(v, 32), lane_of(v, 48)));
  return v;
}

}  // namespace qmm
