// block_norm.hip — the norms after and before a block with its gate and
// residual in between (block_norm in gemm_w4a4.h):
//
//   z = post norm of y (or y itself)
//   r = residual_scale x + gate z
//   h = (norm(r) weight + bias) (1 + scale) + shift
//
// Bound by memory: x and y are read once, r and h written once, about 16 flops
// an element. 4096 x 3072, layer norm with gate, scale and shift: 16.4 us, 6.2 TB/s of
// reads and writes (a 1 GiB copy: 5.1); 4352 x 12288 82.9, 5.2 TB/s. A row's values stay in its lanes' registers from the loads to the
// stores, in float32; both norms' statistics are taken from them there (the
// variance from the differences to the mean, not from a difference of sums).
//
// A row is a wave's, or four waves' where the row is long or rows are few, or 16
// lanes' where it is short and rows are many. Rows of any width start on any 2-byte boundary; all accesses are 16 bytes, the last
// one of a width that is no multiple of 8 over the last 8 elements, the ones
// that it shares with its neighbour left out of the sums (both lanes store
// the same value for them).
#include <hip/hip_runtime.h>

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_w4a4.h"
#include "w4a4_common.hpp"
#include "w4a4_half.hpp"
#include "w4a4_host.hpp"
#include "w4a4_strided.hpp"
#include "w4a4_wave.hpp"

namespace w4a4 {

struct NormParams {
  const uint16_t *x, *y, *gate, *scale, *shift, *weight, *bias, *post_weight;
  uint16_t *out, *residual;
  int64_t xs[2], ys[2], gs[2], ss[2], hs[2], os[2], rs[2];   // batch, token
  int tokens, rows, width;
  float alpha, eps, width_f;
  int post;
};

// Statistics in use: a value v is normalised as (v pre - mean) rstd.
struct RowStats {
  float pre, mean, rstd;
};

// LANES lanes a row, CH runs of 8 elements a lane. TAIL: the width is no multiple of 8.
template <bool F16, bool LAYER, int LANES, int CH, bool TAIL>
__global__ __launch_bounds__(256) void block_norm_kernel(const NormParams p) {
  constexpr int WAVES = LANES / 64, ROWS = 256 / LANES;   // waves of a row (0: less than one); rows of a workgroup
  __shared__ float part[2][4];
  const int tid = threadIdx.x, wave = tid >> 6;
  const int lane = tid & (LANES - 1);
  const int64_t nth = (int64_t(blockIdx.y) * gridDim.x + blockIdx.x) * ROWS + tid / LANES;
  if (nth >= p.rows) return;   // (nothing below meets other rows' lanes)
  int row = int(nth);
  if constexpr (WAVES > 0) row = __builtin_amdgcn_readfirstlane(row);
  const int b = row / p.tokens, tok = row - b * p.tokens;
  const int C = p.width, runs = (C + 7) >> 3;

  // Run c of a lane, the runs dealt from the row's end: only a lane's first run can be the
  // one that is cut, so that only it needs masks (with the runs dealt from the row's
  // start every run did, and 150 to 370 of them were spilled).
  int at[CH], skip = 0;   // first element of a run, negative past the row's start; the cut run's elements that belong to the one before
  bool some[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int n = runs - 1 - (c * LANES + lane);
    some[c] = n >= 0;
    at[c] = n * 8;
  }
  if (TAIL && at[0] + 8 > C) {
    skip = at[0] - max(0, C - 8);
    at[0] = max(0, C - 8);
  }
  // (kept where no masks press: 4096 rows of 3072 16.4 us, 19.8 made anew each time)
  auto live = [&](int c) __attribute__((always_inline)) { return TAIL ? at[c] >= 0 : some[c]; };
  // (fewer than 8 elements: one by one, the rest zeros that `in` leaves out)
  auto load = [&](const uint16_t* from, int c) __attribute__((always_inline)) {
    if (!live(c)) return u32x4{0u, 0u, 0u, 0u};
    if (TAIL && c == 0 && C < 8) {
      u32x4 v{};
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < C) v[i >> 1] |= uint32_t(from[i]) << (16 * (i & 1));
      return v;
    }
    return load16_any(from + at[c]);
  };
  auto store = [&](uint16_t* to, int c, u32x4 v) __attribute__((always_inline)) {
    if (!live(c)) return;
    if (TAIL && c == 0 && C < 8) {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < C) to[i] = uint16_t(v[i >> 1] >> (16 * (i & 1)));
      return;
    }
    store16_any(to + at[c], v);
  };
  auto value = [](const u32x4& v, int i) __attribute__((always_inline)) { return widen<F16>(uint16_t(v[i >> 1] >> (16 * (i & 1)))); };
  // whether element i of run c counts in the sums
  auto in = [&](int c, int i) __attribute__((always_inline)) {
    return live(c) && (!TAIL || c > 0 || (i >= skip && at[0] + i < C));
  };
  int turn = 0;
  auto row_sum = [&](float v) __attribute__((always_inline)) {
    v = WAVES == 0 ? sum_of_16(v) : wave_sum(v);
    if constexpr (WAVES > 1) {
      // (two places in turn: a wave may still read the last sum's while another writes the next)
      if ((tid & 63) == 0) part[turn][wave] = v;
      __syncthreads();
      v = (part[turn][0] + part[turn][1]) + (part[turn][2] + part[turn][3]);
      turn ^= 1;
    }
    return v;
  };
  auto stats_with = [&](const float (&v)[CH][8], float pre, float eps) __attribute__((always_inline)) {
    // (the masks of the runs made anew: held from one step to the next, eight runs' were spilled)
    if constexpr (TAIL) {
      asm volatile("" : "+v"(skip));
#pragma unroll
      for (int c = 0; c < CH; ++c) asm volatile("" : "+v"(at[c]));
    }
    RowStats s{pre, 0.f, 0.f};
    if constexpr (LAYER) {
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += in(c, i) ? v[c][i] * pre : 0.f;
      s.mean = row_sum(sum) / p.width_f;   // (a rounded 1 / width would leave a difference in rows of one value)
    }
    float sq = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = in(c, i) ? v[c][i] * pre - s.mean : 0.f;
        sq += d * d;
      }
    s.rstd = 1.f / sqrtf(row_sum(sq) / p.width_f + eps);
    return s;
  };
  // Sums past float32's range (values from about 2^57 on): the same of values times
  // 2^-80, of which no sum is too large. Beside such values eps is nothing; 2^-100 in
  // its place keeps rows of one value at 0. A row with an infinity or a NaN comes
  // out the same both times.
  auto stats = [&](const float (&v)[CH][8]) __attribute__((always_inline)) {
    RowStats s = stats_with(v, 1.f, p.eps);
    if (!(s.rstd > 0.f) || !(fabsf(s.mean) < INFINITY)) s = stats_with(v, 0x1p-80f, 0x1p-100f);
    return s;
  };

  float r[CH][8];
  {
    const uint16_t* x = p.x + b * p.xs[0] + tok * p.xs[1];
    if (p.y) {
      const uint16_t* y = p.y + b * p.ys[0] + tok * p.ys[1];
      u32x4 xv[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const u32x4 yv = load(y, c);
        xv[c] = load(x, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[c][i] = value(yv, i);
      }
      if (p.post) {
        const RowStats s = stats(r);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const u32x4 wv = p.post_weight ? load(p.post_weight, c) : u32x4{};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            r[c][i] = (r[c][i] * s.pre - s.mean) * s.rstd;
            if (p.post_weight) r[c][i] *= value(wv, i);
          }
        }
      }
      if (p.gate) {
        const uint16_t* gate = p.gate + b * p.gs[0] + tok * p.gs[1];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const u32x4 gv = load(gate, c);
#pragma unroll
          for (int i = 0; i < 8; ++i) r[c][i] *= value(gv, i);
        }
      }
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) r[c][i] += value(xv[c], i) * p.alpha;
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const u32x4 xv = load(x, c);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[c][i] = value(xv, i);
      }
    }
  }
  const RowStats s = stats(r);
  // (x and y are read: either may be residual or out)
  if (p.residual) {
    uint16_t* res = p.residual + b * p.rs[0] + tok * p.rs[1];
#pragma unroll
    for (int c = 0; c < CH; ++c)
      store(res, c, u32x4{narrow2<F16>(r[c][0], r[c][1]), narrow2<F16>(r[c][2], r[c][3]), narrow2<F16>(r[c][4], r[c][5]),
                          narrow2<F16>(r[c][6], r[c][7])});
  }
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) r[c][i] = (r[c][i] * s.pre - s.mean) * s.rstd;
  if (p.weight)
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const u32x4 v = load(p.weight, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[c][i] *= value(v, i);
    }
  if (p.bias)
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const u32x4 v = load(p.bias, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[c][i] += value(v, i);
    }
  if (p.scale) {
    const uint16_t* scale = p.scale + b * p.ss[0] + tok * p.ss[1];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const u32x4 v = load(scale, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[c][i] += r[c][i] * value(v, i);
    }
  }
  if (p.shift) {
    const uint16_t* shift = p.shift + b * p.hs[0] + tok * p.hs[1];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const u32x4 v = load(shift, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[c][i] += value(v, i);
    }
  }
  uint16_t* out = p.out + b * p.os[0] + tok * p.os[1];
#pragma unroll
  for (int c = 0; c < CH; ++c)
    store(out, c, u32x4{narrow2<F16>(r[c][0], r[c][1]), narrow2<F16>(r[c][2], r[c][3]), narrow2<F16>(r[c][4], r[c][5]),
                        narrow2<F16>(r[c][6], r[c][7])});
}

// ------------------------------------------------------------------ host side

template <bool F16, bool LAYER, bool TAIL, int LANES>
static const void* norm_kernel_of(int ch) {
  if constexpr (LANES == 16)
    return reinterpret_cast<const void*>(block_norm_kernel<F16, LAYER, 16, 1, TAIL>);
  else
    return ch <= 1 ? reinterpret_cast<const void*>(block_norm_kernel<F16, LAYER, LANES, 1, TAIL>)
         : ch <= 2 ? reinterpret_cast<const void*>(block_norm_kernel<F16, LAYER, LANES, 2, TAIL>)
         : ch <= 4 ? reinterpret_cast<const void*>(block_norm_kernel<F16, LAYER, LANES, 4, TAIL>)
         : ch <= 6 ? reinterpret_cast<const void*>(block_norm_kernel<F16, LAYER, LANES, 6, TAIL>)
                   : reinterpret_cast<const void*>(block_norm_kernel<F16, LAYER, LANES, 8, TAIL>);
}

template <bool F16, bool LAYER, bool TAIL>
static const void* norm_kernel_of(int lanes, int ch) {
  return lanes == 16 ? norm_kernel_of<F16, LAYER, TAIL, 16>(ch)
       : lanes == 64 ? norm_kernel_of<F16, LAYER, TAIL, 64>(ch)
                     : norm_kernel_of<F16, LAYER, TAIL, 256>(ch);
}

static int block_norm_run(const block_norm_t* a, void* stream) {
  if (!a || a->batch < 0 || a->tokens < 0 || a->width < 1 || a->width > BLOCK_NORM_MAX_WIDTH) return GEMM_W4A4_EINVAL;
  if ((a->f16 | 1) != 1 || (a->layer | 1) != 1 || (a->post_norm | 1) != 1) return GEMM_W4A4_EINVAL;
  if (!(a->eps >= 1e-12f && a->eps <= 1.f) || !(fabsf(a->residual_scale) < INFINITY)) return GEMM_W4A4_EINVAL;
  if (int64_t(a->batch) * a->tokens >= (int64_t(1) << 31)) return GEMM_W4A4_EINVAL;
  if (a->batch == 0 || a->tokens == 0) return GEMM_W4A4_OK;   // (tensors without elements may have no address)
  if (!a->y && (a->gate || a->residual || a->post_norm || a->residual_scale != 1.f)) return GEMM_W4A4_EINVAL;
  if (a->post_weight && !a->post_norm) return GEMM_W4A4_EINVAL;
  const int C = a->width, size[3] = {a->batch, a->tokens, 1};
  struct Tensor {
    const void* p;
    const int64_t* stride;
    int64_t extent;
  };
  Tensor in[] = {{a->x, a->x_stride, 0}, {a->y, a->y_stride, 0}, {a->gate, a->gate_stride, 0},
                 {a->scale, a->scale_stride, 0}, {a->shift, a->shift_stride, 0}};
  Tensor out[] = {{a->out, a->out_stride, 0}, {a->residual, a->residual_stride, 0}};
  for (Tensor& t : in) {
    const int64_t st[3] = {t.stride[0], t.stride[1], 0};
    t.extent = t.p ? strided_extent(size, st, C) : 0;
    if (t.extent < 0) return GEMM_W4A4_EINVAL;
  }
  for (Tensor& t : out) {
    const int64_t st[3] = {t.stride[0], t.stride[1], 0};
    t.extent = t.p ? strided_extent(size, st, C) : 0;
    if (t.extent < 0 || (t.p && !strides_apart(size, st, C))) return GEMM_W4A4_EINVAL;
  }
  if (!a->x || !a->out) return GEMM_W4A4_EINVAL;
  uintptr_t all = uintptr_t(a->weight) | uintptr_t(a->bias) | uintptr_t(a->post_weight);
  for (const Tensor& t : in) all |= uintptr_t(t.p);
  for (const Tensor& t : out) all |= uintptr_t(t.p);
  if (all & 1u) return GEMM_W4A4_EALIGN;
  for (const Tensor& o : out) {
    for (int i = 0; i < 5; ++i) {
      // x or y itself, element for element, is in place
      bool same = i < 2 && o.p == in[i].p;
      for (int d = 0; d < 2; ++d) same = same && (size[d] == 1 || o.stride[d] == in[i].stride[d]);
      if (!same && overlaps(o.p, size_t(o.extent) * 2, in[i].p, size_t(in[i].extent) * 2)) return GEMM_W4A4_EOVERLAP;
    }
    for (const void* v : {a->weight, a->bias, a->post_weight})
      if (overlaps(o.p, size_t(o.extent) * 2, v, size_t(C) * 2)) return GEMM_W4A4_EOVERLAP;
  }
  if (overlaps(a->out, size_t(out[0].extent) * 2, a->residual, size_t(out[1].extent) * 2)) return GEMM_W4A4_EOVERLAP;
  const int dev_rc = check_device();
  if (dev_rc != GEMM_W4A4_OK) return dev_rc;

  NormParams p{};
  const auto bits = [](const void* v) { return static_cast<const uint16_t*>(v); };
  p.x = bits(a->x);
  p.y = bits(a->y);
  p.gate = bits(a->gate);
  p.scale = bits(a->scale);
  p.shift = bits(a->shift);
  p.weight = bits(a->weight);
  p.bias = bits(a->bias);
  p.post_weight = bits(a->post_weight);
  p.out = static_cast<uint16_t*>(a->out);
  p.residual = static_cast<uint16_t*>(a->residual);
  for (int d = 0; d < 2; ++d) {
    p.xs[d] = a->x_stride[d];
    p.ys[d] = a->y_stride[d];
    p.gs[d] = a->gate_stride[d];
    p.ss[d] = a->scale_stride[d];
    p.hs[d] = a->shift_stride[d];
    p.os[d] = a->out_stride[d];
    p.rs[d] = a->residual_stride[d];
  }
  p.tokens = a->tokens;
  p.rows = a->batch * a->tokens;
  p.width = C;
  p.alpha = a->residual_scale;
  p.eps = a->eps;
  p.width_f = float(C);
  p.post = a->post_norm;
  // Lanes of a row. All sides measured (us, with y, gate, scale and shift). 16 against 64: 98304 x 128 19.0 and
  // 42.8, 24672 x 115 7.5 and 16.3, 1100 x 128 3.1 and 3.5. 256 against 64: 8 x 3072 3.6 and 5.3, 600 x
  // 3072 5.4 and 6.3, 1100 x 4096 8.5 and 10.3, 2000 x 4096 12.8 and 14.5; 2000 x 2048 8.0 and 7.8, 4096 x 3072 20.1
  // and 17.1, 4096 x 1001 11.9 and 8.5.
  const bool few = p.rows < 4 * kNumCUs || (C > 2048 && p.rows <= 8 * kNumCUs);
  const int lanes = C > 4096 || few ? 256 : C <= 128 ? 16 : 64;
  const int ch = (C + 8 * lanes - 1) / (8 * lanes);
  const bool tail = C % 8 != 0;
  const void* k;
  if (a->f16)
    k = a->layer ? (tail ? norm_kernel_of<true, true, true>(lanes, ch) : norm_kernel_of<true, true, false>(lanes, ch))
                 : (tail ? norm_kernel_of<true, false, true>(lanes, ch) : norm_kernel_of<true, false, false>(lanes, ch));
  else
    k = a->layer ? (tail ? norm_kernel_of<false, true, true>(lanes, ch) : norm_kernel_of<false, true, false>(lanes, ch))
                 : (tail ? norm_kernel_of<false, false, true>(lanes, ch) : norm_kernel_of<false, false, false>(lanes, ch));
  void* args[] = {&p};
  // (a dimension of a launch holds fewer than 2^32 threads)
  const int64_t groups = (int64_t(p.rows) * lanes + 255) / 256, wide = std::min(groups, int64_t(1) << 20);
  const hipError_t e = hipLaunchKernel(k, dim3(unsigned(wide), unsigned((groups + wide - 1) / wide)), dim3(256), args, 0,
                                       static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GEMM_W4A4_OK : GEMM_W4A4_ELAUNCH;
}

}  // namespace w4a4

extern "C" int block_norm(const block_norm_t* args, void* stream) { return w4a4::block_norm_run(args, stream); }
