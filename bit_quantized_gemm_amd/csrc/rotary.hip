// rotary.hip — rotary positions over several axes on heads [batch, tokens,
// heads, head_dim] (rotary_axes in gemm_w4a4.h).
//
// Pair j of a head turns by t = positions[token, axis(j)] * inv_freq[j]:
// (u, w) -> (u cos t - w sin t, u sin t + w cos t). Bound by memory: 2 bytes
// read and 2 written an element against about 3 flops.
//
// A thread owns one unit of a head: V consecutive elements (interleaved: V/2
// pairs), or V pairs as two runs of V elements (halves), and walks the heads
// of its token, so the angles' sines and cosines, the only real arithmetic,
// are computed once per token and unit. V is 8 (16-byte accesses) where the
// head size, the strides and the addresses allow, else the widest that they
// do. 4096 tokens of 48 heads of 128: 18.2 us, 5.5 TB/s of reads and writes
// (a 1 GiB copy: 5.1).
#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include "gemm_w4a4.h"
#include "w4a4_common.hpp"
#include "w4a4_half.hpp"
#include "w4a4_host.hpp"
#include "w4a4_strided.hpp"

namespace w4a4 {

struct RotaryParams {
  const uint16_t* x;
  uint16_t* out;
  const int32_t* pos;
  const float* inv_freq;
  int64_t xs[3], os[3], ps[2];
  int tokens, heads, head_dim;
  int pairs;           // P
  int ends[3];         // first pair of axes 1, 2, 3 (P where there is none)
  int units;           // units of a head
  int rows;            // heads a workgroup's pass covers (threads / units)
  int token_groups;    // tokens a workgroup's pass covers, when rows > heads
  int inverse;
};

// cos and sin of pos * freq. The angle in turns is held in float64, whose rounding
// moves it by |pos * freq| / 2 pi * 2^-52 turns at most (2^-23 for a position of 2^31
// and a frequency of 1); its fraction, rounded to float32, by 2^-25 more. The sine
// and cosine instructions take turns.
__device__ __forceinline__ void turn(int pos, float freq, float& c, float& s) {
  const double t = double(pos) * (double(freq) * 0.15915494309189535);
  const float a = float(__builtin_amdgcn_fract(t));
  c = __builtin_amdgcn_cosf(a);
  s = __builtin_amdgcn_sinf(a);
}

template <int V>
struct Run {
  typedef uint16_t vec __attribute__((ext_vector_type(V)));
};
template <>
struct Run<1> {
  typedef uint16_t vec __attribute__((ext_vector_type(1)));
};

constexpr int kRotaryThreads = 256;   // most of a workgroup
constexpr int kHeads = 2;   // heads of a thread whose loads are in flight together

// V: elements of a run (interleaved: even). INTER: pairs are neighbours.
template <bool F16, bool INTER, int V>
__global__ __launch_bounds__(kRotaryThreads) void rotary_kernel(const RotaryParams p) {
  typedef typename Run<V>::vec vec;
  constexpr int NP = INTER ? V / 2 : V;   // pairs of a unit
  const int u = threadIdx.x % p.units, row = threadIdx.x / p.units;
  if (row >= p.rows) return;
  const int tok = blockIdx.x * p.token_groups + (p.token_groups > 1 ? row / p.heads : 0);
  if (tok >= p.tokens) return;
  const int h0 = p.token_groups > 1 ? row % p.heads : row;
  const int step = p.token_groups > 1 ? p.heads : p.rows;
  const int b = blockIdx.y;
  const uint16_t* x = p.x + int64_t(b) * p.xs[0] + int64_t(tok) * p.xs[1];
  uint16_t* out = p.out + int64_t(b) * p.os[0] + int64_t(tok) * p.os[1];
  const int32_t* pos = p.pos + int64_t(b) * p.ps[0] + int64_t(tok) * p.ps[1];
  // halves: units past the pairs copy a run of V elements
  const int pair_units = INTER ? p.units : p.pairs / V;
  const bool copy = !INTER && u >= pair_units;
  const int e0 = copy ? 2 * p.pairs + (u - pair_units) * V : u * V;
  // The heads of a pass, kHeads at a time: their loads are asked for together,
  // the first ones before the angles are worked out.
  vec lo[kHeads], hi[kHeads];
  auto load = [&](int h0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const uint16_t* xh = x + int64_t(min(h0 + i * step, p.heads - 1)) * p.xs[2] + e0;
      lo[i] = *reinterpret_cast<const vec*>(xh);
      if constexpr (!INTER)
        if (!copy) hi[i] = *reinterpret_cast<const vec*>(xh + p.pairs);
    }
  };
  load(h0);
  float c[NP], s[NP];
  if (!copy) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int j = INTER ? u * NP + i : e0 + i;
      c[i] = 1.f;
      s[i] = 0.f;
      if (j < p.pairs) {
        const int a = int(j >= p.ends[0]) + int(j >= p.ends[1]) + int(j >= p.ends[2]);
        turn(pos[a], p.inv_freq[j], c[i], s[i]);
        if (p.inverse) s[i] = -s[i];
      }
    }
  }
  for (int hb = h0; hb < p.heads; hb += kHeads * step) {
    if (hb != h0) load(hb);
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int h = hb + k * step;
      if (h >= p.heads) break;
      uint16_t* oh = out + int64_t(h) * p.os[2] + e0;
      const vec a = lo[k];
      if (copy) {
        *reinterpret_cast<vec*>(oh) = a;
      } else if constexpr (INTER) {
        vec r = a;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          if (u * NP + i < p.pairs) {   // elements past the pairs keep their bits
            const float x0 = widen<F16>(a[2 * i]), x1 = widen<F16>(a[2 * i + 1]);
            r[2 * i] = narrow<F16>(x0 * c[i] - x1 * s[i]);
            r[2 * i + 1] = narrow<F16>(x0 * s[i] + x1 * c[i]);
          }
        }
        *reinterpret_cast<vec*>(oh) = r;
      } else {
        const vec w = hi[k];
        vec r0, r1;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const float x0 = widen<F16>(a[i]), x1 = widen<F16>(w[i]);
          r0[i] = narrow<F16>(x0 * c[i] - x1 * s[i]);
          r1[i] = narrow<F16>(x0 * s[i] + x1 * c[i]);
        }
        *reinterpret_cast<vec*>(oh) = r0;
        *reinterpret_cast<vec*>(oh + p.pairs) = r1;
      }
    }
  }
}

// ------------------------------------------------------------------ host side

template <bool F16, bool INTER>
const void* rotary_kernel_of(int v) {
  switch (v) {
    case 8: return reinterpret_cast<const void*>(rotary_kernel<F16, INTER, 8>);
    case 4: return reinterpret_cast<const void*>(rotary_kernel<F16, INTER, 4>);
    case 2: return reinterpret_cast<const void*>(rotary_kernel<F16, INTER, 2>);
    default: return INTER ? nullptr : reinterpret_cast<const void*>(rotary_kernel<F16, false, 1>);
  }
}

static int rotary_run(const rotary_axes_t* a, void* stream) {
  if (!a || a->batch < 0 || a->tokens < 0 || a->heads < 0) return GEMM_W4A4_EINVAL;
  if (a->head_dim < 1 || a->head_dim > ROTARY_MAX_HEAD_DIM) return GEMM_W4A4_EINVAL;
  if (a->axes < 1 || a->axes > ROTARY_AXES_MAX || a->batch > 65535) return GEMM_W4A4_EINVAL;
  if ((a->f16 | 1) != 1 || (a->interleaved | 1) != 1 || (a->inverse | 1) != 1) return GEMM_W4A4_EINVAL;
  int P = 0, ends[4];
  for (int i = 0; i < ROTARY_AXES_MAX; ++i) {
    if (i < a->axes) {
      if (a->sections[i] < 0 || a->sections[i] > a->head_dim / 2) return GEMM_W4A4_EINVAL;
      P += a->sections[i];
    }
    ends[i] = i < a->axes - 1 ? P : ROTARY_MAX_HEAD_DIM;
  }
  if (2 * P > a->head_dim || (a->interleaved && a->head_dim % 2 != 0)) return GEMM_W4A4_EINVAL;
  const int size[3] = {a->batch, a->tokens, a->heads};
  const int64_t xe = strided_extent(size, a->x_stride, a->head_dim), oe = strided_extent(size, a->out_stride, a->head_dim);
  if (xe < 0 || oe < 0 || !strides_apart(size, a->out_stride, a->head_dim)) return GEMM_W4A4_EINVAL;
  const int psize[3] = {a->batch, a->tokens, 1};
  const int64_t pst[3] = {a->pos_stride[0], a->pos_stride[1], 0};
  const int64_t pe = strided_extent(psize, pst, a->axes);
  if (pe < 0) return GEMM_W4A4_EINVAL;
  if (a->batch == 0 || a->tokens == 0 || a->heads == 0) return GEMM_W4A4_OK;
  if (!a->x || !a->out || !a->positions || (P > 0 && !a->inv_freq)) return GEMM_W4A4_EINVAL;
  if ((uintptr_t(a->x) | uintptr_t(a->out)) & 1u) return GEMM_W4A4_EALIGN;
  if ((uintptr_t(a->positions) | uintptr_t(a->inv_freq)) & 3u) return GEMM_W4A4_EALIGN;
  bool same = a->x == a->out;
  for (int i = 0; i < 3; ++i) same = same && (size[i] == 1 || a->x_stride[i] == a->out_stride[i]);
  if ((!same && overlaps(a->out, size_t(oe) * 2, a->x, size_t(xe) * 2)) ||
      overlaps(a->out, size_t(oe) * 2, a->positions, size_t(pe) * 4) ||
      overlaps(a->out, size_t(oe) * 2, a->inv_freq, size_t(P) * 4))
    return GEMM_W4A4_EOVERLAP;
  // widest run that the sizes, the strides and the addresses allow
  int v = 8;
  const bool inter = a->interleaved != 0;
  auto fits = [&](int w) {
    bool ok = a->head_dim % w == 0 && (inter || P % w == 0) && ((uintptr_t(a->x) | uintptr_t(a->out)) & (2 * w - 1)) == 0;
    for (int i = 0; i < 3; ++i)
      ok = ok && (size[i] == 1 || (a->x_stride[i] % w == 0 && a->out_stride[i] % w == 0));
    return ok;
  };
  while (v > 1 && !fits(v)) v /= 2;
  if (inter && v < 2) return GEMM_W4A4_EALIGN;
  const int dev_rc = check_device();
  if (dev_rc != GEMM_W4A4_OK) return dev_rc;
  RotaryParams p{};
  p.x = static_cast<const uint16_t*>(a->x);
  p.out = static_cast<uint16_t*>(a->out);
  p.pos = a->positions;
  p.inv_freq = a->inv_freq;
  for (int i = 0; i < 3; ++i) {
    p.xs[i] = a->x_stride[i];
    p.os[i] = a->out_stride[i];
    p.ends[i] = ends[i];
  }
  p.ps[0] = a->pos_stride[0];
  p.ps[1] = a->pos_stride[1];
  p.tokens = a->tokens;
  p.heads = a->heads;
  p.head_dim = a->head_dim;
  p.pairs = P;
  p.inverse = a->inverse;
  p.units = inter ? a->head_dim / v : P / v + (a->head_dim - 2 * P) / v;
  // One wave a workgroup where a head's units fit (measured against 128, 256 and
  // 512 threads at 4096 tokens: 48 of 72 heads of 128 18.2 us against 18.3, 20.1
  // and 22.2; 24 heads, halves, 11.7 against 13.7, 17.1 and 21.8).
  const int threads = p.units <= kWave ? kWave : kRotaryThreads;
  p.rows = threads / p.units;
  p.token_groups = p.rows >= 2 * a->heads ? p.rows / a->heads : 1;
  p.rows = p.token_groups > 1 ? p.token_groups * a->heads : std::min(p.rows, a->heads);
  const void* k = a->f16 ? (inter ? rotary_kernel_of<true, true>(v) : rotary_kernel_of<true, false>(v))
                         : (inter ? rotary_kernel_of<false, true>(v) : rotary_kernel_of<false, false>(v));
  void* args[] = {&p};
  const unsigned grid = unsigned((int64_t(a->tokens) + p.token_groups - 1) / p.token_groups);
  const hipError_t e = hipLaunchKernel(k, dim3(grid, a->batch), dim3(threads), args, 0, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GEMM_W4A4_OK : GEMM_W4A4_ELAUNCH;
}

}  // namespace w4a4

extern "C" int rotary_axes(const rotary_axes_t* args, void* stream) { return w4a4::rotary_run(args, stream); }
