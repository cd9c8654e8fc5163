// w4a4_transpose.hpp — the transposing LDS read, which turns rows of 16-bit values
// into a matrix instruction's operand of their columns.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "w4a4_common.hpp"

namespace w4a4 {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Transposed read: the lanes of a group of 16 pass the addresses of 4 rows x 4
// runs of 4 values; lane i gets column i of the 4 rows.
__device__ __forceinline__ u32x2 read_transposed(const uint8_t* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (__attribute__((address_space(3))) s16x4*)p));
}

}  // namespace w4a4
