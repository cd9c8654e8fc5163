// w4a4_buffer.hpp — buffer descriptors and direct-to-LDS buffer loads, shared
// by the kernels that stream rows of a known extent: a read past the
// descriptor's range returns zeros, so ragged ends need no address clamp.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

namespace w4a4 {

// Descriptor of `bytes` bytes from `base` (both wave-uniform).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, int(bytes), 0x00020000);
}

// 16-byte direct-to-LDS load: lane l writes lds + 16 l (zeros past the range).
__device__ __forceinline__ void dma_rows(__amdgpu_buffer_rsrc_t rs, uint32_t voff, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)lds, 16, voff, 0, 0, 0);
}

}  // namespace w4a4
