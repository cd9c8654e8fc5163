// w4a4_half.hpp — the two 16-bit types as bit patterns: widening to float32,
// rounding from it (nearest even) and their matrix instructions.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "w4a4_common.hpp"

namespace w4a4 {

template <bool F16>
__device__ __forceinline__ float widen(uint16_t b) {
  if constexpr (F16) return float(__builtin_bit_cast(_Float16, b));
  else return __builtin_bit_cast(float, uint32_t(b) << 16);
}

template <bool F16>
__device__ __forceinline__ uint16_t narrow(float v) {   // round to nearest even
  if constexpr (F16) return __builtin_bit_cast(uint16_t, _Float16(v));
  else return __builtin_bit_cast(uint16_t, __bf16(v));
}

// Two values rounded to one dword, `lo` in the low half.
template <bool F16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
  if constexpr (F16) {
    return __builtin_bit_cast(uint32_t, f16x2{_Float16(lo), _Float16(hi)});
  } else {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, bf16x2{__bf16(lo), __bf16(hi)});
  }
}

// D += A B over 16 (32x32 tile) or 32 (16x16 tile) of k, 8 values a lane.
template <bool F16>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  return lora_mfma<F16>(a, b, c);
}
template <bool F16>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

}  // namespace w4a4
