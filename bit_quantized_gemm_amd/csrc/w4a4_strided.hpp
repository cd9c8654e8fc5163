// w4a4_strided.hpp — host checks of strided tensors of three outer dimensions
// with a dense run of elements inside.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace w4a4 {

// Whether dimensions of these sizes and strides (elements, run of `run`
// dense elements inside) give every index memory of its own.
template <int N>
inline bool strides_apart(const int (&size)[N], const int64_t (&stride)[N], int64_t run) {
  int order[N];
  for (int i = 0; i < N; ++i) order[i] = i;
  std::sort(order, order + N, [&](int a, int b) { return stride[a] < stride[b]; });
  int64_t span = run;
  for (int i : order) {
    if (size[i] <= 1) continue;
    if (stride[i] < span) return false;
    span = stride[i] * (size[i] - 1) + span;
  }
  return true;
}

// Elements from the first to the last of a strided tensor; -1 when that
// passes 2^62 or a stride is negative.
inline int64_t strided_extent(const int (&size)[3], const int64_t (&stride)[3], int64_t run) {
  const int64_t lim = int64_t(1) << 60;
  int64_t e = run;
  for (int i = 0; i < 3; ++i) {
    if (size[i] <= 1) continue;
    if (stride[i] < 0 || stride[i] > lim / size[i]) return -1;
    e += stride[i] * (size[i] - 1);
    if (e > lim) return -1;
  }
  return e;
}

}  // namespace w4a4
