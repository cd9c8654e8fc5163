// w4a4_wave.hpp — sums over a wave, and 16-byte accesses of rows that start
// anywhere.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "w4a4_common.hpp"

namespace w4a4 {

// The lanes of a group of 16, permuted: ctrl is a DPP control (quad permutation,
// mirror of 8 or of 16 lanes).
template <int CTRL>
__device__ __forceinline__ float lane_permuted(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}

// The sum over the wave, in every lane, always in the same order. In registers:
// shuffles through LDS take five times as long (a chain of six of about 100 cycles).
__device__ __forceinline__ float sum_of_16(float v) {   // over each 16 lanes
  v += lane_permuted<0xB1>(v);    // lane ^ 1
  v += lane_permuted<0x4E>(v);    // lane ^ 2
  v += lane_permuted<0x141>(v);   // the other 4 of 8
  v += lane_permuted<0x140>(v);   // the other 8 of 16
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
  v = sum_of_16(v);
  auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  v = __builtin_bit_cast(float, uint32_t(r[0])) + __builtin_bit_cast(float, uint32_t(r[1]));
  r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return __builtin_bit_cast(float, uint32_t(r[0])) + __builtin_bit_cast(float, uint32_t(r[1]));
}

// max(v, v of lane ^ 32); likewise the sum
__device__ __forceinline__ float other_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return fmaxf(__builtin_bit_cast(float, uint32_t(r[0])), __builtin_bit_cast(float, uint32_t(r[1])));
}
__device__ __forceinline__ float other_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return __builtin_bit_cast(float, uint32_t(r[0])) + __builtin_bit_cast(float, uint32_t(r[1]));
}

// 16 bytes on any 2-byte boundary, in one access: global memory takes them.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
__device__ __forceinline__ u32x4 load16_any(const uint16_t* p) { return *reinterpret_cast<const u32x4_any*>(p); }
__device__ __forceinline__ void store16_any(uint16_t* p, u32x4 v) { *reinterpret_cast<u32x4_any*>(p) = v; }

}  // namespace w4a4
