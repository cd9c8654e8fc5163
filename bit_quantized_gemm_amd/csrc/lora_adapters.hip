// lora_adapters.hip — low-rank adapters of many requests beside a shared
// projection (lora_adapters in gemm_w4a4.h): row m with adapter a,
//
//   out[m] = y[m] + scaling[a] (x[m] down[a]^T) up[a]
//
// in two launches, since all of K has to be summed before the first column:
//
//   shrink   low[m] = x[m] down[a]^T, K over the waves of a workgroup and, where
//            rows are few, over workgroups (slices), float32 sums to the workspace
//   expand   adds the slices up, multiplies by up[a] and adds y
//
// Both are bound by memory: many rows by y and out, few rows by the adapters
// in use. Rows are taken in tiles as they come; a tile goes through the distinct
// adapters of its rows one by one, so rows of a request, which are neighbours, share
// the adapter's operands, and no order of rows is wrong. Columns of the products belong
// to rows, so rows of other adapters in the tile are computed along and not stored.
// With few rows each distinct adapter of a tile has a workgroup of its own.
//
// low is held in float32. For the second product, whose matrix instruction takes
// 16 bits, it is split into two 16-bit parts, high and low, so that
// nothing past 2^-16 of it is lost; the instructions are hidden behind the
// memory. In binary16 a row is first scaled by a power of two, so that no size
// of low passes the type's range.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "gemm_w4a4.h"
#include "w4a4_common.hpp"
#include "w4a4_half.hpp"
#include "w4a4_host.hpp"
#include "w4a4_strided.hpp"
#include "w4a4_transpose.hpp"
#include "w4a4_wave.hpp"

namespace w4a4 {

struct AdaptParams {
  const uint16_t *x, *y, *down, *up;
  uint16_t* out;
  const int32_t *adapter, *ranks;
  const float* scaling;
  float* low;              // [slices][rows][padded rank]
  int64_t xs, ys, os;      // row strides
  int rows, K, N, adapters, R, Rp;
  int slices;
  int in_place;
};

// The rank of adapter a, 0 where it is none.
__device__ __forceinline__ int rank_of(const AdaptParams& p, int a) {
  if (a < 0 || a >= p.adapters) return 0;
  return p.ranks ? min(max(p.ranks[a], 0), p.R) : p.R;
}

// Calls f(adapter, its rank, mask of its rows) for the distinct adapters of up to 64 rows
// from row0 on, in order of their first rows: for number `slot` and every `slots`-th
// after it. Adapter -1: rows without one.
template <class F>
__device__ __forceinline__ void each_adapter(const AdaptParams& p, int row0, int rows, int slot, int slots, F&& f) {
  const int lane = threadIdx.x & 63, row = row0 + lane;
  const bool live = lane < rows && row < p.rows;
  int id = live ? p.adapter[row] : -1;
  const int rank = live ? rank_of(p, id) : 0;
  if (rank == 0) id = -1;
  uint64_t left = __builtin_amdgcn_ballot_w64(live);
  for (int n = 0; left; ++n) {
    const int first = __builtin_ctzll(left);
    const int a = __builtin_amdgcn_readlane(id, first), r = __builtin_amdgcn_readlane(rank, first);
    const uint64_t mask = __builtin_amdgcn_ballot_w64(live && id == a);
    left &= ~mask;
    if (n % slots == slot) f(a, r, mask);
  }
}

// RT: tiles of 16 ranks at most; XT: tiles of 16 rows. blockIdx: row tile, slice of K, slot.
template <bool F16, int RT, int XT>
__global__ __launch_bounds__(256) void adapters_shrink_kernel(const AdaptParams p) {
  constexpr int WAVES = 4, STEPS = 2;   // 32-wide steps of k in flight a wave
  __shared__ f32x4 part[WAVES][RT * XT * 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int row0 = blockIdx.x * 16 * XT, slice = blockIdx.y;
  const int units = (p.K + 32 * STEPS - 1) / (32 * STEPS);
  const int u0 = int(int64_t(units) * slice / p.slices), u1 = int(int64_t(units) * (slice + 1) / p.slices);
  each_adapter(p, row0, 16 * XT, blockIdx.z, gridDim.z, [&](int a, int rank, uint64_t mask) __attribute__((always_inline)) {
    if (a < 0) return;
    const int nt = (rank + 15) >> 4;
    const uint16_t *xr[XT], *dr[RT];
    bool have[RT];   // this lane's rank is one of the adapter's
#pragma unroll
    for (int t = 0; t < XT; ++t) xr[t] = p.x + int64_t(min(row0 + 16 * t + l16, p.rows - 1)) * p.xs;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      have[t] = 16 * t + l16 < rank;
      dr[t] = p.down + (int64_t(a) * p.R + min(16 * t + l16, rank - 1)) * p.K;
    }
    f32x4 acc[RT][XT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < XT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 xv[2][STEPS][XT], dv[2][STEPS][RT];
    auto load = [&](int u, int at) __attribute__((always_inline)) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int k = (u * STEPS + s) * 32 + 8 * g, kc = min(k, p.K - 8);
        const bool in = k < p.K;
#pragma unroll
        for (int t = 0; t < XT; ++t) {
          xv[at][s][t] = *reinterpret_cast<const u32x4*>(xr[t] + kc);
          if (!in) xv[at][s][t] = u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int t = 0; t < RT; ++t)
          if (t < nt) {
            dv[at][s][t] = *reinterpret_cast<const u32x4*>(dr[t] + kc);
            if (!in || !have[t]) dv[at][s][t] = u32x4{0u, 0u, 0u, 0u};
          }
      }
    };
    auto multiply = [&](int at) __attribute__((always_inline)) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int t = 0; t < RT; ++t)
          if (t < nt)
#pragma unroll
            for (int j = 0; j < XT; ++j) acc[t][j] = mfma16<F16>(dv[at][s][t], xv[at][s][j], acc[t][j]);
    };
    int u = u0 + wave;
    if (u < u1) load(u, 0);
    for (; u < u1; u += 2 * WAVES) {
      if (u + WAVES < u1) load(u + WAVES, 1);
      multiply(0);
      if (u + 2 * WAVES < u1) load(u + 2 * WAVES, 0);
      if (u + WAVES < u1) multiply(1);
    }
    // the waves' sums meet in LDS, in order
    __syncthreads();
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int j = 0; j < XT; ++j) part[wave][(t * XT + j) * 64 + lane] = acc[t][j];
    __syncthreads();
    for (int i = tid; i < nt * XT * 64; i += 256) {
      const int t = i / (XT * 64), j = i / 64 % XT, r = i & 15, q = (i >> 4) & 3;
      f32x4 v = part[0][i];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) v += part[w][i];
      const int at = 16 * t + 4 * q;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (at + e >= rank) v[e] = 0.f;   // (an infinity of x times nothing)
      if (mask >> (16 * j + r) & 1)
        *reinterpret_cast<f32x4*>(p.low + (int64_t(slice) * p.rows + row0 + 16 * j + r) * p.Rp + at) = v;
    }
  });
}

// Two 16-bit parts of eight values: high the nearest, low the nearest to the rest.
template <bool F16>
__device__ __forceinline__ void split8(const float (&v)[8], u32x4& high, u32x4& low) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = narrow2<F16>(v[2 * i], v[2 * i + 1]);
    const float h0 = widen<F16>(uint16_t(h)), h1 = widen<F16>(uint16_t(h >> 16));
    high[i] = h;
    low[i] = narrow2<F16>(fabsf(h0) < INFINITY ? v[2 * i] - h0 : 0.f, fabsf(h1) < INFINITY ? v[2 * i + 1] - h1 : 0.f);
  }
}

// A wave: 64 columns of up to 64 rows. up[a]'s tile passes through LDS of the wave's own
// to be transposed: D[column][row] = up^T low^T, so that a row is a lane. The
// matrix instruction's columns are dealt so that a lane's values are runs of 8
// neighbours (16-byte accesses of y and out, 128 bytes a row and wave).
// KT: steps of 16 ranks at most. TAIL: N is no multiple of 8. blockIdx: 4 waves of columns,
// row tile, slot.
template <bool F16, int KT, bool TAIL>
__global__ __launch_bounds__(256) void adapters_expand_kernel(const AdaptParams p) {
  constexpr int ROWB = 128;
  __shared__ __attribute__((aligned(16))) uint8_t smem[4][KT * 16 * ROWB];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int n0 = (blockIdx.x * 4 + wave) * 64;
  if (n0 >= p.N) return;
  uint8_t* tile = smem[wave];
  const int row0 = blockIdx.y * 64;
  // 8 columns from n on of a row; those past N are zeros and are not stored
  auto load8 = [&](const uint16_t* row, int n) __attribute__((always_inline)) {
    u32x4 v{0u, 0u, 0u, 0u};
    if (n + (TAIL ? 7 : 0) < p.N) {
      v = load16_any(row + n);
    } else if (TAIL) {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (n + i < p.N) v[i >> 1] |= uint32_t(row[n + i]) << (16 * (i & 1));
    }
    return v;
  };
  auto store8 = [&](uint16_t* row, int n, u32x4 v) __attribute__((always_inline)) {
    if (n + (TAIL ? 7 : 0) < p.N) {
      store16_any(row + n, v);
    } else if (TAIL) {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (n + i < p.N) row[n + i] = uint16_t(v[i >> 1] >> (16 * (i & 1)));
    }
  };
  each_adapter(p, row0, 64, blockIdx.z, gridDim.z, [&](int a, int rank, uint64_t mask) __attribute__((always_inline)) {
    if (a < 0 && p.in_place) return;
    const int nt = (rank + 15) >> 4;
    u32x4 up[2][KT];
    float factor = 1.f;
    if (a >= 0) {
      const uint16_t* from = p.up + int64_t(a) * p.R * p.N;
      u32x4 in[2 * KT];
#pragma unroll
      for (int i = 0; i < 2 * KT; ++i)
        if (i < 2 * nt) {
          const int r = 8 * i + (lane >> 3);
          in[i] = r < rank ? load8(from + int64_t(r) * p.N, n0 + 8 * (lane & 7)) : u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
      for (int i = 0; i < 2 * KT; ++i)
        if (i < 2 * nt) {
          const int r = 8 * i + (lane >> 3), c = (lane & 7) ^ ((r >> 1 & 1) << 2);
          *reinterpret_cast<u32x4*>(tile + r * ROWB + c * 16) = in[i];
        }
      if (p.scaling) factor = p.scaling[a];
#pragma unroll
      for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int k = 0; k < KT; ++k)
          if (k < nt) {
            const int r = 16 * k + 4 * h + ((lane & 15) >> 2);
            // runs of 4 columns in the order 0 2 1 3 of each 16
            const int run = 8 * d + 4 * ((lane >> 4) & 1) + ((lane & 1) << 1 | (lane >> 1 & 1));
            const uint8_t* v = tile + r * ROWB + (((run >> 1) ^ ((r >> 1 & 1) << 2)) * 16) + (run & 1) * 8;
            const u32x2 lo = read_transposed(v), hi = read_transposed(v + 8 * ROWB);
            up[d][k] = u32x4{lo.x, lo.y, hi.x, hi.y};
          }
    }
#pragma unroll 1
    for (int sub = 0; sub < 2; ++sub) {
      const uint32_t mine = uint32_t(mask >> (32 * sub));
      if (mine == 0) continue;
      const int row = min(row0 + 32 * sub + l32, p.rows - 1);
      const bool store = mine >> l32 & 1;
      const uint16_t* yr = p.y + int64_t(row) * p.ys;
      uint16_t* outr = p.out + int64_t(row) * p.os;
      u32x4 yv[2][2];
#pragma unroll
      for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int b = 0; b < 2; ++b) yv[d][b] = load8(yr, n0 + 32 * d + 16 * b + 8 * h);
      if (a >= 0) {
        float low[KT][8];
        const float* lr = p.low + int64_t(row) * p.Rp + 4 * h;
#pragma unroll
        for (int k = 0; k < KT; ++k)
          if (k < nt) {
            f32x4 v0 = *reinterpret_cast<const f32x4*>(lr + 16 * k), v1 = *reinterpret_cast<const f32x4*>(lr + 16 * k + 8);
            for (int s = 1; s < p.slices; ++s) {
              const float* other = lr + int64_t(s) * p.rows * p.Rp + 16 * k;
              v0 += *reinterpret_cast<const f32x4*>(other);
              v1 += *reinterpret_cast<const f32x4*>(other + 8);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              low[k][e] = v0[e] * factor;
              low[k][4 + e] = v1[e] * factor;
            }
          }
        float back = 1.f;
        if constexpr (F16) {
          float top = 0.f;
#pragma unroll
          for (int k = 0; k < KT; ++k)
            if (k < nt)
#pragma unroll
              for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(low[k][e]));
          top = other_max(top);
          if (top > 0.f && top < INFINITY) {
            const int ex = max(__builtin_amdgcn_frexp_expf(top), -100) - 15;   // the largest to 2^14 .. 2^15
            const float to = __builtin_amdgcn_ldexpf(1.f, -ex);
            back = __builtin_amdgcn_ldexpf(1.f, ex);
#pragma unroll
            for (int k = 0; k < KT; ++k)
              if (k < nt)
#pragma unroll
                for (int e = 0; e < 8; ++e) low[k][e] *= to;
          }
        }
        f32x16 acc[2] = {};
#pragma unroll
        for (int k = 0; k < KT; ++k)
          if (k < nt) {
            u32x4 lh, ll;
            split8<F16>(low[k], lh, ll);
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              acc[d] = mfma32<F16>(up[d][k], lh, acc[d]);
              acc[d] = mfma32<F16>(up[d][k], ll, acc[d]);
            }
          }
#pragma unroll
        for (int d = 0; d < 2; ++d)
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t w = yv[d][b][i];
              yv[d][b][i] = narrow2<F16>(widen<F16>(uint16_t(w)) + acc[d][8 * b + 2 * i] * back,
                                         widen<F16>(uint16_t(w >> 16)) + acc[d][8 * b + 2 * i + 1] * back);
            }
      }
      if (store)
#pragma unroll
        for (int d = 0; d < 2; ++d)
#pragma unroll
          for (int b = 0; b < 2; ++b) store8(outr, n0 + 32 * d + 16 * b + 8 * h, yv[d][b]);
    }
  });
}

// ------------------------------------------------------------------ host side

struct AdaptPlan {
  int row_tiles;        // of 16 rows
  int tiles, slots, slices;
  int out_tiles, out_slots;
  int Rp;
  int64_t bytes;
};

static bool adapt_sizes_ok(const lora_adapters_t* a) {
  return a && a->rows >= 0 && a->rows <= LORA_ADAPTERS_MAX_ROWS && a->N >= 1 && a->N <= 1 << 30 && a->K >= 8 && a->K <= 1 << 30 && a->K % 8 == 0 &&
         a->rank >= 1 && a->rank <= LORA_ADAPTERS_MAX_RANK && a->adapters >= 1;
}

// Row tiles of 16 rows where there are few, else 32. Up to two workgroups a compute
// unit, first by distinct adapters (few rows), then by slices of K of at least 256.
static AdaptPlan adapt_plan(const lora_adapters_t* a) {
  constexpr int kWorkgroups = 2 * kNumCUs;
  AdaptPlan pl{};
  pl.Rp = (a->rank + 15) / 16 * 16;
  pl.row_tiles = a->rows <= 256 ? 1 : 2;
  const int per = 16 * pl.row_tiles;
  pl.tiles = (a->rows + per - 1) / per;
  const int most = std::min(std::min(a->adapters, a->rows), per);   // distinct adapters of a tile
  pl.slots = std::max(1, std::min(kWorkgroups / std::max(1, pl.tiles), most));
  pl.slices = std::max(1, std::min(std::min(kWorkgroups / std::max(1, pl.tiles * pl.slots), (a->K + 255) / 256), 8));
  pl.out_tiles = (a->rows + 63) / 64;
  const int64_t groups = (int64_t(a->N) + 255) / 256 * std::max(1, pl.out_tiles);
  // (one more than the adapters: the rows without one)
  pl.out_slots = int(std::max<int64_t>(1, std::min<int64_t>(2 * kWorkgroups / groups, std::min(std::min(a->adapters + 1, a->rows), 64))));
  pl.bytes = int64_t(pl.slices) * a->rows * pl.Rp * 4;
  return pl;
}

template <bool F16>
static const void* shrink_of(int ranks, int row_tiles) {
  if (row_tiles == 1)
    return ranks <= 16 ? reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 1, 1>)
         : ranks <= 32 ? reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 2, 1>)
         : ranks <= 64 ? reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 4, 1>)
                       : reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 8, 1>);
  return ranks <= 16 ? reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 1, 2>)
       : ranks <= 32 ? reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 2, 2>)
       : ranks <= 64 ? reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 4, 2>)
                     : reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 8, 2>);
}

template <bool F16, bool TAIL>
static const void* expand_of(int ranks) {
  return ranks <= 32 ? reinterpret_cast<const void*>(adapters_expand_kernel<F16, 2, TAIL>)
       : ranks <= 64 ? reinterpret_cast<const void*>(adapters_expand_kernel<F16, 4, TAIL>)
                     : reinterpret_cast<const void*>(adapters_expand_kernel<F16, 8, TAIL>);
}

static int lora_adapters_run(const lora_adapters_t* a, void* stream) {
  if (!adapt_sizes_ok(a) || (a->f16 | 1) != 1) return GEMM_W4A4_EINVAL;
  const int64_t lim = int64_t(1) << 60;
  const int xsz[3] = {a->rows, 1, 1};
  const int64_t xst[3] = {a->x_stride, 0, 0}, yst[3] = {a->y_stride, 0, 0}, ost[3] = {a->out_stride, 0, 0};
  const int64_t xe = strided_extent(xsz, xst, a->K), ye = strided_extent(xsz, yst, a->N), oe = strided_extent(xsz, ost, a->N);
  if (xe < 0 || ye < 0 || oe < 0 || !strides_apart(xsz, ost, a->N)) return GEMM_W4A4_EINVAL;
  if (a->rows > 1 && (a->x_stride & 7)) return GEMM_W4A4_EINVAL;
  const int64_t widest = std::max(a->K, a->N);
  if (int64_t(a->adapters) * a->rank > lim / widest) return GEMM_W4A4_EINVAL;
  if (a->rows == 0) return GEMM_W4A4_OK;
  if (!a->x || !a->y || !a->down || !a->up || !a->out || !a->adapter) return GEMM_W4A4_EINVAL;
  if ((uintptr_t(a->x) | uintptr_t(a->down)) & 15u) return GEMM_W4A4_EALIGN;
  if ((uintptr_t(a->y) | uintptr_t(a->up) | uintptr_t(a->out)) & 1u) return GEMM_W4A4_EALIGN;
  if ((uintptr_t(a->adapter) | uintptr_t(a->ranks) | uintptr_t(a->scaling)) & 3u) return GEMM_W4A4_EALIGN;
  const AdaptPlan pl = adapt_plan(a);
  if (!a->workspace || a->workspace_bytes < pl.bytes) return GEMM_W4A4_ESCRATCH;
  if (uintptr_t(a->workspace) & 15u) return GEMM_W4A4_EALIGN;
  const bool same = a->out == a->y && (a->rows == 1 || a->out_stride == a->y_stride);
  const size_t weights = size_t(a->adapters) * a->rank * 2;
  const struct { const void* p; size_t n; } outs[] = {{a->out, size_t(oe) * 2}, {a->workspace, size_t(pl.bytes)}},
      ins[] = {{a->y, size_t(ye) * 2}, {a->x, size_t(xe) * 2}, {a->down, weights * a->K}, {a->up, weights * a->N},
               {a->adapter, size_t(a->rows) * 4}, {a->ranks, size_t(a->adapters) * 4}, {a->scaling, size_t(a->adapters) * 4}};
  for (int o = 0; o < 2; ++o)
    for (int i = 0; i < 7; ++i)
      if (!(o == 0 && i == 0 && same) && overlaps(outs[o].p, outs[o].n, ins[i].p, ins[i].n)) return GEMM_W4A4_EOVERLAP;
  if (overlaps(outs[0].p, outs[0].n, outs[1].p, outs[1].n)) return GEMM_W4A4_EOVERLAP;
  const int dev_rc = check_device();
  if (dev_rc != GEMM_W4A4_OK) return dev_rc;
  AdaptParams p{};
  p.x = static_cast<const uint16_t*>(a->x);
  p.y = static_cast<const uint16_t*>(a->y);
  p.down = static_cast<const uint16_t*>(a->down);
  p.up = static_cast<const uint16_t*>(a->up);
  p.out = static_cast<uint16_t*>(a->out);
  p.adapter = a->adapter;
  p.ranks = a->ranks;
  p.scaling = a->scaling;
  p.low = static_cast<float*>(a->workspace);
  p.xs = a->x_stride;
  p.ys = a->y_stride;
  p.os = a->out_stride;
  p.rows = a->rows;
  p.K = a->K;
  p.N = a->N;
  p.adapters = a->adapters;
  p.R = a->rank;
  p.Rp = pl.Rp;
  p.slices = pl.slices;
  p.in_place = same;
  void* args[] = {&p};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = hipLaunchKernel(a->f16 ? shrink_of<true>(a->rank, pl.row_tiles) : shrink_of<false>(a->rank, pl.row_tiles),
                                 dim3(unsigned(pl.tiles), unsigned(pl.slices), unsigned(pl.slots)), dim3(256), args, 0, st);
  const bool tail = a->N % 8 != 0;
  const void* expand = a->f16 ? (tail ? expand_of<true, true>(a->rank) : expand_of<true, false>(a->rank))
                              : (tail ? expand_of<false, true>(a->rank) : expand_of<false, false>(a->rank));
  if (e == hipSuccess)
    e = hipLaunchKernel(expand,
                        dim3(unsigned((a->N + 255) / 256), unsigned(pl.out_tiles), unsigned(pl.out_slots)), dim3(256), args, 0, st);
  return e == hipSuccess ? GEMM_W4A4_OK : GEMM_W4A4_ELAUNCH;
}

}  // namespace w4a4

extern "C" int lora_adapters(const lora_adapters_t* args, void* stream) { return w4a4::lora_adapters_run(args, stream); }

extern "C" int64_t lora_adapters_workspace(const lora_adapters_t* args) {
  return w4a4::adapt_sizes_ok(args) ? w4a4::adapt_plan(args).bytes : GEMM_W4A4_EINVAL;
}
