// w4a4_page_index.hpp — the page of a key by a multiplication: for the host, which
// makes the multiplier, and the kernels that use it.
#pragma once

#include <stdint.h>

namespace w4a4 {

// key / page_size = high 32 bits of key * magic, >> shift, for keys below 2^31
struct PageIndex {
  uint32_t magic;
  int shift;
  constexpr int of(int key) const { return int(uint32_t((uint64_t(uint32_t(key)) * magic) >> 32) >> shift); }
};

// For pages of 9 keys or more: with 2^(n-1) < page_size <= 2^n the multiplier
// ceil(2^(31+n) / page_size) has 32 bits and is too large by less than 1, so that key * magic is
// too large by less than 2^31; the next page begins 2^(31+n) / page_size >= 2^31 or more further on.
constexpr PageIndex page_index(int page_size) {
  int n = 4;
  while ((int64_t(1) << n) < page_size) ++n;
  return PageIndex{uint32_t(((uint64_t(1) << (31 + n)) + uint64_t(page_size) - 1) / uint64_t(page_size)), n - 1};
}

}  // namespace w4a4
