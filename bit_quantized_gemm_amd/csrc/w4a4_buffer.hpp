// w4a4_buffer.hpp — direct-to-LDS buffer loads of rows of a known extent: a
// read past the descriptor's range returns zeros, so ragged ends need no
// address clamp.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "w4a4_common.hpp"

namespace w4a4 {

// A memory instruction takes scalar registers that a vector instruction wrote (a descriptor's, read from
// a lane) five cycles later at the earliest. The compiler sees no such instruction inside
// load_to_lds, so the wait is here: three, and the two before its load. (Once a descriptor: 2048 packed
// tokens of 4 heads on one 21.7 us, with it before each load 22.6.)
__device__ __forceinline__ void settle_desc(u32x4& d) { asm volatile("s_nop 2" : "+s"(d)); }

// Descriptor of `bytes` bytes from `base` (both wave-uniform), in scalar registers.
__device__ __forceinline__ u32x4 range_desc(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  u32x4 d{uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(a))),
          uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(a >> 32) & 0xFFFFu)),
          uint32_t(__builtin_amdgcn_readfirstlane(bytes)), 0x00020000u};
  settle_desc(d);
  return d;
}

// LDS byte address of a shared-memory pointer.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return uint32_t(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const uint8_t*)p));
}

// 16-byte load to LDS: lane l writes byte address lds + 16 l (zeros past the
// range). It has no register output; the caller waits for it (wait_vm) before
// the barrier that publishes the data. Written as an instruction because the
// compiler, where it knows of such a load, waits for all of them before every
// transposing LDS read, which leaves none in flight. M0, the LDS base, is set
// here, one idle cycle before the load takes it. The compiler reserves M0 and takes
// no note of it as clobbered, so a kernel that uses this may have no other
// instruction that sets or takes M0 (tests/test_block_asm.py reads the assembly).
__device__ __forceinline__ void load_to_lds(const u32x4& desc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(desc)
               : "memory");
}

}  // namespace w4a4
