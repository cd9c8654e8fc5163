// lora_adapters.hip — low-rank adapters of many requests beside a shared
// projection (lora_adapters in gemm_w4a4.h): row m with adapter a,
//
//   out[m] = y[m] + scaling[a] (x[m] down[a]^T) up[a]
//
// in launches of their own, since all of K has to be summed before the first column:
//
//   shrink   low[m] = scaling[a] x[m] down[a]^T, K over the waves of a workgroup and over
//            workgroups (slices)
//   expand   multiplies low by up[a] and adds y
//
// Both are bound by memory: many rows by y and out, few rows by the adapters
// in use. Columns of the products belong to rows, so the rows of a tile only have to share an
// adapter, and lie anywhere. Few rows are taken as they come: a tile goes through the
// distinct adapters of its rows, each of which has a workgroup of its own while there are
// compute units, and expand adds the slices and splits the sums (below) itself. Many rows are
// first grouped, a launch of one workgroup: tiles of 64 rows of one adapter. (Tiles as
// they come take 60 us in place of 47 for 4352 rows of 12 requests and 12288 columns: the last
// tiles, of short requests, go through six adapters one after the other.) There the slices are
// added and split between the two products, once for all columns.
//
// low is summed in float32. For the second product, whose matrix instruction takes
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
  float* low;              // [slices][rows][Rp]
  u32x4* parts;            // joined: the two parts in the order of the second product's operand,
                           // [tile of 32 rows][16 ranks][part][lane][8],
  float* back;             // and, binary16, each row's factor
  int64_t xs, ys, os;      // row strides
  int rows, K, N, adapters, R, Rp;   // Rp: 16 rank_steps(R)
  int slices;
  int in_place;
  // many rows: the groups' tiles, and the rows of tile t from order[64 t] on
  struct AdaptTile* group;
  int32_t* order;
  int tiles;               // most tiles there can be
};

struct AdaptTile {
  int adapter, rank;       // rank 0: rows without an adapter
  int rows;                // 0: no tile
  float scaling;
};

// The rank of adapter a, 0 where it is none.
__device__ __forceinline__ int rank_of(const AdaptParams& p, int a) {
  if (a < 0 || a >= p.adapters) return 0;
  return p.ranks ? min(max(p.ranks[a], 0), p.R) : p.R;
}

// Steps of 16 ranks that both launches go through for a rank: a power of two, each of which
// has code of its own. low is zeros from the rank on.
constexpr int kAdaptSlices = 4;   // most slices of K, whose loads expand has in flight together
__host__ __device__ __forceinline__ int rank_steps(int rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }

// Lane n: the place of the n-th set bit of `mask` (n below their number; past it, those of the
// bits that are not set).
__device__ __forceinline__ int nth_bits(uint64_t mask) {
  const int lane = threadIdx.x & 63;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  const int set = __builtin_popcountll(mask & below);
  const int to = mask >> lane & 1 ? set : __builtin_popcountll(mask) + lane - set;
  return __builtin_amdgcn_ds_permute(to * 4, lane);
}
// What lane n holds (all lanes take part: one that does not is read as 0).
__device__ __forceinline__ int of_lane(int v, int n) { return __builtin_amdgcn_ds_bpermute(n * 4, v); }

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

// Rows by adapter, in tiles of 64. The order of rows within an adapter's tiles goes by the order
// in which the waves come by; no result depends on it.
constexpr int kGroupThreads = 1024, kGroupAdapters = 4096;   // most adapters it takes
__global__ __launch_bounds__(kGroupThreads) void adapters_group_kernel(const AdaptParams p) {
  __shared__ int next[kGroupAdapters + 1];   // rows of an adapter (the last: of none), then the next place in its tiles
  __shared__ int total[kGroupThreads / 64];
  constexpr int ROUNDS = 8;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, A = p.adapters;
  for (int a = tid; a <= A; a += kGroupThreads) next[a] = 0;
  __syncthreads();
  // The adapters of the next rows, all loads in flight together; up to 8192 rows they
  // stay in the registers for both passes.
  int id[ROUNDS];
  auto look = [&](int row0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) id[i] = p.adapter[min(row0 + i * kGroupThreads + tid, p.rows - 1)];
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i)
      if (id[i] < 0 || id[i] > A) id[i] = A;
  };
  // f(row, adapter, mask of the wave's lanes whose rows have it) for the distinct adapters of each wave
  auto each = [&](bool again, auto&& f) __attribute__((always_inline)) {
    for (int row0 = 0; row0 < p.rows; row0 += ROUNDS * kGroupThreads) {
      if (!again || p.rows > ROUNDS * kGroupThreads) look(row0);
#pragma unroll
      for (int i = 0; i < ROUNDS; ++i) {
        const int row = row0 + i * kGroupThreads + tid;
        uint64_t left = __builtin_amdgcn_ballot_w64(row < p.rows);
        while (left) {
          const int a = __builtin_amdgcn_readlane(id[i], __builtin_ctzll(left));
          const uint64_t mask = __builtin_amdgcn_ballot_w64(row < p.rows && id[i] == a);
          left &= ~mask;
          f(row, a, mask);
        }
      }
    }
  };
  each(false, [&](int, int a, uint64_t mask) __attribute__((always_inline)) {
    if (lane == 0) atomicAdd(&next[a], __builtin_popcountll(mask));
  });
  __syncthreads();
  // the first tile of each adapter: a thread takes a run of them, and the sums before it
  const int run = A / kGroupThreads + 1, from = tid * run, to = min(from + run, A + 1);
  int tiles = 0;
  for (int a = from; a < to; ++a) tiles += (next[a] + 63) >> 6;
  int upto = tiles;   // of the wave's lanes up to this one
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int v = __shfl_up(upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 63) total[wave] = upto;
  __syncthreads();
  int at = upto - tiles, all = 0;
#pragma unroll
  for (int w = 0; w < kGroupThreads / 64; ++w) {
    at += w < wave ? total[w] : 0;
    all += total[w];
  }
  for (int a = from; a < to; ++a) {
    const int n = next[a];
    next[a] = at * 64;
    const AdaptTile tile{a, rank_of(p, a), 64, a < A && p.scaling ? p.scaling[a] : 1.f};
    for (int i = 0; i < n; i += 64, ++at) {
      p.group[at] = tile;
      if (n - i < 64) p.group[at].rows = n - i;
    }
  }
  for (int i = all + tid; i < p.tiles; i += kGroupThreads) p.group[i].rows = 0;
  __syncthreads();
  each(true, [&](int row, int a, uint64_t mask) __attribute__((always_inline)) {
    int place = 0;
    if (lane == 0) place = atomicAdd(&next[a], __builtin_popcountll(mask));
    place = __builtin_amdgcn_readfirstlane(place);
    if (mask >> lane & 1) p.order[place + __builtin_popcountll(mask & ((uint64_t(1) << lane) - 1))] = row;
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

// binary16: the power of two by which a row whose largest finite value is `top` is multiplied
// before the split, which takes that to 2^14 .. 2^15, and its inverse. (An infinity stays
// one under any factor, and may not leave the row's other values past the type's range:
// opposite infinities would be a NaN.)
__device__ __forceinline__ float finite_size(float v) { return fabsf(v) < INFINITY ? fabsf(v) : 0.f; }
__device__ __forceinline__ void row_factor(float top, float& to, float& back) {
  to = back = 1.f;
  if (top > 0.f) {
    const int e = max(__builtin_amdgcn_frexp_expf(top), -100) - 15;
    to = __builtin_amdgcn_ldexpf(1.f, -e);
    back = __builtin_amdgcn_ldexpf(1.f, e);
  }
}

// low of 16 XT rows (XT > 1: of a group's tile) and a slice of K, in float32. RT: tiles of 16 ranks
// at most. The waves split
// the slice, so that its loads, of both operands straight to the matrix instruction's
// registers, are in flight at once. blockIdx: row tile, slice, slot.
template <bool F16, int RT, int XT, int WAVES>
__global__ __launch_bounds__(WAVES * 64, 2) void adapters_shrink_kernel(const AdaptParams p) {
  constexpr int STEPS = XT == 1 && RT < 8 ? 2 : 1, UNIT = 32 * STEPS;   // k of a wave's turn
  __shared__ f32x4 part[WAVES][RT * XT * 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  constexpr int DEPTH = XT == 1 ? 2 : 4;   // turns whose loads are in flight together
  constexpr int PER = 64 / (16 * XT);   // workgroups of a group's tile
  const int row0 = XT > 1 ? 0 : blockIdx.x * 16, slice = blockIdx.y;
  const int units = (p.K + UNIT - 1) / UNIT;
  // a wave's turns lie one after the other in the row
  const int nth = slice * WAVES + wave, all = p.slices * WAVES;
  const int u0 = int(int64_t(units) * nth / all), u1 = int(int64_t(units) * (nth + 1) / all);
  // NT: the adapter's rank tiles, and NX: tiles of its rows, so that every load is certain (with
  // loads that depend on the rank the compiler waits for each)
  auto sums = [&]<int NT, int NX>(int a, int rank, int places, int count) __attribute__((always_inline)) {
    const uint16_t *xr[NX], *dr[NT];
#pragma unroll
    for (int j = 0; j < NX; ++j) xr[j] = p.x + int64_t(row0 + of_lane(places, min(16 * j + l16, count - 1))) * p.xs;
    // (ranks past the last repeat it: their sums are columns of their own, made zeros below)
#pragma unroll
    for (int t = 0; t < NT; ++t) dr[t] = p.down + (int64_t(a) * p.R + min(16 * t + l16, rank - 1)) * p.K;
    f32x4 acc[NT][NX];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < NX; ++j) acc[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 xv[DEPTH][STEPS][NX], dv[DEPTH][STEPS][NT];
    auto load = [&](int u, int at) __attribute__((always_inline)) {   // (past the last unit: the last again)
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        const int k = min(max(min(u, u1 - 1), 0) * UNIT + 32 * s + 8 * g, p.K - 8);
#pragma unroll
        for (int j = 0; j < NX; ++j) xv[at][s][j] = *reinterpret_cast<const u32x4*>(xr[j] + k);
#pragma unroll
        for (int t = 0; t < NT; ++t) dv[at][s][t] = *reinterpret_cast<const u32x4*>(dr[t] + k);
      }
    };
    auto multiply = [&](int u, int at) __attribute__((always_inline)) {
      if ((u + 1) * UNIT > p.K) {   // what lies past K: nothing
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
          if (u * UNIT + 32 * s + 8 * g >= p.K) {
#pragma unroll
            for (int j = 0; j < NX; ++j) xv[at][s][j] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int t = 0; t < NT; ++t) dv[at][s][t] = u32x4{0u, 0u, 0u, 0u};
          }
      }
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < NX; ++j) acc[t][j] = mfma16<F16>(dv[at][s][t], xv[at][s][j], acc[t][j]);
    };
    for (int u = u0; u < u1; u += DEPTH) {
#pragma unroll
      for (int i = 0; i < DEPTH; ++i) load(u + i, i);
#pragma unroll
      for (int i = 0; i < DEPTH; ++i)
        if (u + i < u1) multiply(u + i, i);
    }
    __syncthreads();   // (the last adapter's part is read)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < NX; ++j) part[wave][(t * XT + j) * 64 + lane] = acc[t][j];
  };
  auto adapter = [&](int a, int rank, float factor, int places, int count) __attribute__((always_inline)) {
    const int nt = rank_steps(rank);
    auto with = [&]<int NT>() __attribute__((always_inline)) {
      if (count <= 16) sums.template operator()<NT, 1>(a, rank, places, count);
      else sums.template operator()<NT, XT>(a, rank, places, count);
    };
    if (nt == 1) with.template operator()<1>();
    else if (nt == 2) with.template operator()<(RT < 2 ? RT : 2)>();
    else if (nt == 4) with.template operator()<(RT < 4 ? RT : 4)>();
    else with.template operator()<RT>();
    // the waves' sums meet in LDS, in order; a thread takes 8 ranks of a row
    __syncthreads();
    const int nx = (count + 15) >> 4;
    const int items = nt * nx * 32;
    for (int i0 = 0; i0 < items; i0 += WAVES * 64) {
      // (every lane stays in: others read its `places`)
      const int i = min(i0 + tid, items - 1), r = i & 15, half = (i >> 4) & 1, j = (i >> 5) % nx, t = (i >> 5) / nx;
      const int at = (t * XT + j) * 64 + 32 * half + r;
      const int row = row0 + of_lane(places, min(16 * j + r, count - 1));
      f32x4 s0 = part[0][at], s1 = part[0][at + 16];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) {
        s0 += part[w][at];
        s1 += part[w][at + 16];
      }
      const int left = rank - (16 * t + 8 * half);   // ranks from the last on are zeros
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s0[e] = e < left ? s0[e] * factor : 0.f;
        s1[e] = 4 + e < left ? s1[e] * factor : 0.f;
      }
      if (i0 + tid < items && 16 * j + r < count) {
        f32x4* to = reinterpret_cast<f32x4*>(p.low + (int64_t(slice) * p.rows + row) * p.Rp + 16 * t + 8 * half);
        to[0] = s0;
        to[1] = s1;
      }
    }
  };
  if constexpr (XT > 1) {
    const AdaptTile g = p.group[blockIdx.x / PER];
    const int first = int(blockIdx.x) % PER * 16 * XT, count = min(g.rows - first, 16 * XT);
    if (g.rank > 0 && count > 0) {
      const int row = p.order[blockIdx.x / PER * 64 + first + min(lane, count - 1)];
      adapter(g.adapter, g.rank, g.scaling, row, count);
    }
  } else {
    each_adapter(p, row0, 16, blockIdx.z, gridDim.z, [&](int a, int rank, uint64_t mask) __attribute__((always_inline)) {
      if (a >= 0) adapter(a, rank, p.scaling ? p.scaling[a] : 1.f, nth_bits(mask), __builtin_popcountll(mask));
    });
  }
}

// The slices' sums of 32 rows, added in order and split: once for all columns. A wave per 16
// ranks, a lane per 8 of them of a row. (Rows without an adapter, and what lies past the steps of
// a row's own, are whatever the workspace holds; nothing reads them.)
template <bool F16>
__global__ __launch_bounds__(512) void adapters_join_kernel(const AdaptParams p) {
  __shared__ uint32_t top[32];
  const int tid = threadIdx.x, lane = tid & 63, t = tid >> 6, r = lane & 31;
  const int row = min(int(blockIdx.x) * 32 + r, p.rows - 1);
  const float* from = p.low + int64_t(row) * p.Rp + 16 * t + 8 * (lane >> 5);
  f32x4 s0{}, s1{};
  for (int s = 0; s < p.slices; s += 8) {   // eight slices' loads in flight together
    f32x4 v[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const f32x4* at = reinterpret_cast<const f32x4*>(from + int64_t(min(s + i, p.slices - 1)) * p.rows * p.Rp);
      v[i][0] = at[0];
      v[i][1] = at[1];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (s + i < p.slices) {
        s0 += v[i][0];
        s1 += v[i][1];
      }
  }
  float v[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
  if constexpr (F16) {
    // the row's largest, over the ranks of its own adapter
    const int steps = rank_steps(rank_of(p, p.adapter[row]));
    float m = 0.f, to, back;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, finite_size(v[e]));
    if (tid < 32) top[tid] = 0;
    __syncthreads();
    if (t < steps) atomicMax(&top[r], __builtin_bit_cast(uint32_t, m));   // (of magnitudes, in any order the same)
    __syncthreads();
    row_factor(__builtin_bit_cast(float, top[r]), to, back);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= to;
    if (tid < 32 && int(blockIdx.x) * 32 + r < p.rows) p.back[row] = back;
  }
  u32x4 hi, lo;
  split8<F16>(v, hi, lo);
  u32x4* to = p.parts + (int64_t(blockIdx.x) * (p.Rp >> 4) + t) * 128 + lane;
  to[0] = hi;
  to[64] = lo;
}

// A wave: 64 columns of up to 64 rows. up[a]'s tile passes through LDS of the wave's own
// to be transposed, D[column][row] = up^T low^T, and D through the same LDS back to rows,
// so that y and out are read and written 128 bytes a row (straight from the
// accumulators, 32 bytes a row at a time, 4352 x 12288 columns took 99 us).
// KT: steps of 16 ranks at most. SLICED: low as the slices' sums.
// blockIdx: 4 waves of columns, row tile, slot.
enum class Tail {
  kNone,     // N is a multiple of 8
  kShift,
  kNarrow,   // N is below 8
};
template <bool F16, int KT, Tail TAIL, bool SLICED>
__global__ __launch_bounds__(256, KT > 4 ? (SLICED ? 1 : 2) : SLICED ? 2 : KT > 2 ? 3 : 4) void adapters_expand_kernel(const AdaptParams p) {
  constexpr int ROWB = 128, PITCH = 68;   // bytes of a row of up's tile; floats of a row of D
  constexpr int BYTES = KT * 16 * ROWB > 32 * PITCH * 4 ? KT * 16 * ROWB : 32 * PITCH * 4;
  __shared__ __attribute__((aligned(16))) uint8_t smem[4][BYTES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int n0 = (blockIdx.x * 4 + wave) * 64;
  if (n0 >= p.N) return;
  uint8_t* tile = smem[wave];
  float* sums = reinterpret_cast<float*>(tile);
  const int row0 = SLICED ? blockIdx.y * 64 : 0;
  const int r8 = lane >> 3, c8 = lane & 7, n = n0 + 8 * c8;   // accesses of rows: 8 lanes a row
  // Columns n .. n + 7 of a row; those past N are not stored, and whatever the row holds. The loads of
  // the last columns end with the row and are moved down afterwards (`settle`), so that every load is
  // one access, and certain.
  auto load8 = [&](const uint16_t* row) __attribute__((always_inline)) {
    if constexpr (TAIL == Tail::kNarrow) {
      u32x4 v{0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (n + i < p.N) v[i >> 1] |= uint32_t(row[n + i]) << (16 * (i & 1));
      return v;
    } else {
      return load16_any(row + min(n, p.N - 8));
    }
  };
  const bool last = TAIL == Tail::kShift && n0 + 64 > p.N;   // the wave holds the row's end
  auto settle = [&](u32x4& v) __attribute__((always_inline)) {
    if constexpr (TAIL == Tail::kShift) {
      const int by = max(n + 8 - p.N, 0);
      if (by & 1) v = u32x4{v.x >> 16 | v.y << 16, v.y >> 16 | v.z << 16, v.z >> 16 | v.w << 16, v.w >> 16};
      if (by & 2) v = u32x4{v.y, v.z, v.w, 0u};
      if (by & 4) v = u32x4{v.z, v.w, 0u, 0u};
    }
  };
  auto store8 = [&](uint16_t* row, u32x4 v) __attribute__((always_inline)) {
    if (n + 8 <= p.N) store16_any(row + n, v);
    else if constexpr (TAIL != Tail::kNone)
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (n + i < p.N) row[n + i] = uint16_t(v[i >> 1] >> (16 * (i & 1)));
  };
  // NT: the adapter's steps of 16 ranks; 0: rows without one
  auto rows = [&]<int NT>(int a, int rank, int places, int count) __attribute__((always_inline)) {
    constexpr int NT1 = NT > 0 ? NT : 1;
    u32x4 up[2][NT1];
    if constexpr (NT > 0) {
      const uint16_t* from = p.up + int64_t(a) * p.R * p.N;
      u32x4 in[2 * NT];
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) in[i] = load8(from + int64_t(min(8 * i + r8, rank - 1)) * p.N);
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) {
        const int r = 8 * i + r8;
        if (last) settle(in[i]);
        if (r >= rank) in[i] = u32x4{0u, 0u, 0u, 0u};
        *reinterpret_cast<u32x4*>(tile + r * ROWB + (c8 ^ ((r >> 1 & 1) << 2)) * 16) = in[i];
      }
#pragma unroll
      for (int d = 0; d < 2; ++d)
#pragma unroll
        for (int k = 0; k < NT; ++k) {
          const int r = 16 * k + 8 * h + ((lane & 15) >> 2), run = 8 * d + 4 * ((lane >> 4) & 1) + (lane & 3);
          const uint8_t* v = tile + r * ROWB + ((run >> 1) ^ ((r >> 1 & 1) << 2)) * 16 + (run & 1) * 8;
          const u32x2 lo = read_transposed(v), hi = read_transposed(v + 4 * ROWB);
          up[d][k] = u32x4{lo.x, lo.y, hi.x, hi.y};
        }
    }
#pragma unroll 1
    for (int base = 0; base < count; base += 32) {
      int64_t at[4];   // rows of this lane's accesses
      u32x4 yv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        at[i] = row0 + of_lane(places, min(base + 8 * i + r8, count - 1));
        yv[i] = load8(p.y + at[i] * p.ys);
      }
      if constexpr (NT == 0) {
        if (last)
#pragma unroll
          for (int i = 0; i < 4; ++i) settle(yv[i]);
      } else {
        f32x16 acc[2] = {};
        float back = 1.f;
        const int row = row0 + of_lane(places, min(base + l32, count - 1));   // of this lane's column of D
        if constexpr (SLICED) {
          float low[NT][8];
#pragma unroll
          for (int k = 0; k < NT; ++k) {
            const float* lr = p.low + int64_t(row) * p.Rp + 16 * k + 8 * h;
            f32x4 v[kAdaptSlices][2];
#pragma unroll
            for (int s = 0; s < kAdaptSlices; ++s) {
              const f32x4* from = reinterpret_cast<const f32x4*>(lr + int64_t(min(s, p.slices - 1)) * p.rows * p.Rp);
              v[s][0] = from[0];
              v[s][1] = from[1];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              low[k][e] = v[0][e >> 2][e & 3];
#pragma unroll
              for (int s = 1; s < kAdaptSlices; ++s) low[k][e] += s < p.slices ? v[s][e >> 2][e & 3] : 0.f;
            }
          }
          if constexpr (F16) {
            float top = 0.f, to;
#pragma unroll
            for (int k = 0; k < NT; ++k)
#pragma unroll
              for (int e = 0; e < 8; ++e) top = fmaxf(top, finite_size(low[k][e]));
            row_factor(other_max(top), to, back);
#pragma unroll
            for (int k = 0; k < NT; ++k)
#pragma unroll
              for (int e = 0; e < 8; ++e) low[k][e] *= to;
          }
#pragma unroll
          for (int k = 0; k < NT; ++k) {
            u32x4 lh, ll;
            split8<F16>(low[k], lh, ll);
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              acc[d] = mfma32<F16>(up[d][k], lh, acc[d]);
              acc[d] = mfma32<F16>(up[d][k], ll, acc[d]);
            }
          }
        } else {
          u32x4 lv[NT][2];
          const u32x4* from = p.parts + int64_t(row >> 5) * (p.Rp >> 4) * 2 * 64 + 32 * h + (row & 31);
#pragma unroll
          for (int k = 0; k < NT; ++k) {
            lv[k][0] = from[k * 128];
            lv[k][1] = from[k * 128 + 64];
          }
          if constexpr (F16) back = p.back[row];
#pragma unroll
          for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              acc[d] = mfma32<F16>(up[d][k], lv[k][0], acc[d]);
              acc[d] = mfma32<F16>(up[d][k], lv[k][1], acc[d]);
            }
        }
        if (last)
#pragma unroll
          for (int i = 0; i < 4; ++i) settle(yv[i]);
        // D to rows (a wave's LDS accesses keep their order)
#pragma unroll
        for (int d = 0; d < 2; ++d)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<f32x4*>(sums + l32 * PITCH + 32 * d + 2 * i + 4 * h) =
                f32x4{acc[d][i] * back, acc[d][i + 1] * back, acc[d][i + 2] * back, acc[d][i + 3] * back};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 s0 = *reinterpret_cast<const f32x4*>(sums + (8 * i + r8) * PITCH + 8 * c8);
          const f32x4 s1 = *reinterpret_cast<const f32x4*>(sums + (8 * i + r8) * PITCH + 8 * c8 + 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t w = yv[i][j];
            const float a0 = j < 2 ? s0[2 * j & 3] : s1[2 * j & 3], a1 = j < 2 ? s0[(2 * j + 1) & 3] : s1[(2 * j + 1) & 3];
            yv[i][j] = narrow2<F16>(widen<F16>(uint16_t(w)) + a0, widen<F16>(uint16_t(w >> 16)) + a1);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (base + 8 * i + r8 < count) store8(p.out + at[i] * p.os, yv[i]);
    }
  };
  // places: lane n's row, from row0, of the adapter's n-th
  auto adapter = [&](int a, int rank, int places, int count) __attribute__((always_inline)) {
    const int nt = rank_steps(rank);
    if (a < 0) {
      if (!p.in_place) rows.template operator()<0>(a, rank, places, count);
    } else if (nt == 1) {
      rows.template operator()<1>(a, rank, places, count);
    } else if (nt == 2) {
      rows.template operator()<KT < 2 ? 1 : 2>(a, rank, places, count);
    } else if (nt == 4) {
      rows.template operator()<KT < 4 ? KT : 4>(a, rank, places, count);
    } else {
      rows.template operator()<KT>(a, rank, places, count);
    }
  };
  if constexpr (SLICED) {
    each_adapter(p, row0, 64, blockIdx.z, gridDim.z, [&](int a, int rank, uint64_t mask) __attribute__((always_inline)) {
      adapter(a, rank, nth_bits(mask), __builtin_popcountll(mask));
    });
  } else {
    const AdaptTile g = p.group[blockIdx.y];
    if (g.rows == 0) return;
    const int row = p.order[64 * blockIdx.y + min(lane, g.rows - 1)];
    adapter(g.rank > 0 ? g.adapter : -1, g.rank, row, g.rows);
  }
}

// ------------------------------------------------------------------ host side

struct AdaptPlan {
  bool many;            // grouped
  int tiles, slots, slices;
  int out_tiles, out_slots;
  int Rp;
  int64_t low_bytes, parts_bytes, back_bytes, group_bytes, bytes;
};

static bool adapt_sizes_ok(const lora_adapters_t* a) {
  return a && a->rows >= 0 && a->rows <= LORA_ADAPTERS_MAX_ROWS && a->N >= 1 && a->N <= 1 << 30 && a->K >= 8 && a->K <= 1 << 30 && a->K % 8 == 0 &&
         a->rank >= 1 && a->rank <= LORA_ADAPTERS_MAX_RANK && a->adapters >= 1;
}

// Few or many by rows x rank x columns, since few rows split low anew for every 64 columns. Both
// measured (us, few against many), up to 2^26: 800 rows, rank 16, 1024 columns 10.3 and 16.0, 431,
// 32, 2746 10.3 and 17.4, 1200, 16, 3072 16.1 and 18.7, 512, 32, 3072 18.7 and 17.9; past it 260, 64, 7822
// 21.6 and 20.1, 300, 64, 9216 28.8 and 19.6, 512, 32, 12288 25.6 and 21.3, 150, 128, 12288 32 and 25.
// Few rows: workgroups of 16 rows, one for each distinct adapter, and slices of K of at least
// 512 (a turn for each wave) while there are fewer workgroups than compute units. Many: the
// groups' tiles (of 64 ranks and 64 rows the operands are loaded once for 16 products; past rank
// 64 two workgroups of 32 rows a tile), slices of about 512, all of whose loads are in flight at once,
// up to two workgroups a compute unit.
static AdaptPlan adapt_plan(const lora_adapters_t* a) {
  constexpr int64_t kFewWork = int64_t(1) << 26;
  AdaptPlan pl{};
  pl.Rp = 16 * rank_steps(a->rank);
  pl.many = a->rows > 64 && int64_t(a->rows) * pl.Rp * a->N > kFewWork && a->adapters <= kGroupAdapters;
  if (pl.many) {
    pl.out_tiles = a->rows / 64 + std::min(a->adapters + 1, a->rows);
    pl.out_slots = 1;
    pl.tiles = pl.out_tiles * (a->rank <= 64 ? 1 : 2);
    pl.slots = 1;
    const int likely = (a->rows + 63) / 64 * (a->rank <= 64 ? 1 : 2);
    pl.slices = std::max(1, std::min(std::min(2 * kNumCUs / likely, (a->K + 511) / 512), 8));
  } else {
    pl.tiles = (a->rows + 15) / 16;
    const int tiles = std::max(1, pl.tiles);
    pl.slots = std::max(1, std::min(2 * kNumCUs / tiles, std::min(std::min(a->adapters, a->rows), 16)));
    pl.slices = std::max(1, std::min(std::min(kNumCUs / (tiles * pl.slots), a->K / 512), kAdaptSlices));
    pl.out_tiles = (a->rows + 63) / 64;
    const int64_t groups = (int64_t(a->N) + 255) / 256 * std::max(1, pl.out_tiles);
    // (one more than the adapters: the rows without one)
    pl.out_slots = int(std::max<int64_t>(1, std::min({4 * kNumCUs / groups, int64_t(a->adapters) + 1, int64_t(a->rows), int64_t(64)})));
  }
  pl.bytes = pl.low_bytes = int64_t(pl.slices) * a->rows * pl.Rp * 4;
  if (pl.many) {
    pl.parts_bytes = (int64_t(a->rows) + 31) / 32 * 32 * pl.Rp * 4;
    pl.back_bytes = a->f16 ? (int64_t(a->rows) + 3) / 4 * 16 : 0;
    pl.group_bytes = int64_t(pl.out_tiles) * int64_t(sizeof(AdaptTile));
    pl.bytes += pl.parts_bytes + pl.back_bytes + pl.group_bytes + int64_t(pl.out_tiles) * 64 * 4;
  }
  return pl;
}

template <bool F16>
static const void* shrink_of(bool many, int ranks) {
  if (many)
    return ranks <= 16 ? reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 1, 4, 4>)
         : ranks <= 32 ? reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 2, 4, 4>)
         : ranks <= 64 ? reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 4, 4, 4>)
                       : reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 8, 2, 4>);
  return ranks <= 16 ? reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 1, 1, 8>)
       : ranks <= 32 ? reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 2, 1, 8>)
       : ranks <= 64 ? reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 4, 1, 8>)
                     : reinterpret_cast<const void*>(adapters_shrink_kernel<F16, 8, 1, 8>);
}

template <bool F16, Tail TAIL, bool SLICED>
static const void* expand_of(int ranks) {
  return ranks <= 16 ? reinterpret_cast<const void*>(adapters_expand_kernel<F16, 1, TAIL, SLICED>)
       : ranks <= 32 ? reinterpret_cast<const void*>(adapters_expand_kernel<F16, 2, TAIL, SLICED>)
       : ranks <= 64 ? reinterpret_cast<const void*>(adapters_expand_kernel<F16, 4, TAIL, SLICED>)
                     : reinterpret_cast<const void*>(adapters_expand_kernel<F16, 8, TAIL, SLICED>);
}

template <bool F16, bool SLICED>
static const void* expand_of(int ranks, int N) {
  if (N < 8) return reinterpret_cast<const void*>(adapters_expand_kernel<F16, 8, Tail::kNarrow, SLICED>);
  return N % 8 == 0 ? expand_of<F16, Tail::kNone, SLICED>(ranks) : expand_of<F16, Tail::kShift, SLICED>(ranks);
}

template <bool F16>
static const void* expand_of(int ranks, int N, bool sliced) {
  return sliced ? expand_of<F16, true>(ranks, N) : expand_of<F16, false>(ranks, N);
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
  p.parts = reinterpret_cast<u32x4*>(p.low + pl.low_bytes / 4);
  p.back = p.low + (pl.low_bytes + pl.parts_bytes) / 4;
  p.group = reinterpret_cast<AdaptTile*>(p.back + pl.back_bytes / 4);
  p.order = reinterpret_cast<int32_t*>(p.group + pl.out_tiles);
  p.tiles = pl.out_tiles;
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
  hipError_t e = hipSuccess;
  if (pl.many) e = hipLaunchKernel(reinterpret_cast<const void*>(adapters_group_kernel), dim3(1), dim3(kGroupThreads), args, 0, st);
  if (e == hipSuccess)
    e = hipLaunchKernel(a->f16 ? shrink_of<true>(pl.many, a->rank) : shrink_of<false>(pl.many, a->rank),
                        dim3(unsigned(pl.tiles), unsigned(pl.slices), unsigned(pl.slots)), dim3(pl.many ? 256 : 512), args, 0, st);
  if (e == hipSuccess && pl.many)
    e = hipLaunchKernel(a->f16 ? reinterpret_cast<const void*>(adapters_join_kernel<true>) : reinterpret_cast<const void*>(adapters_join_kernel<false>),
                        dim3(unsigned((a->rows + 31) / 32)), dim3(pl.Rp * 4), args, 0, st);
  if (e == hipSuccess)
    e = hipLaunchKernel(a->f16 ? expand_of<true>(a->rank, a->N, !pl.many) : expand_of<false>(a->rank, a->N, !pl.many),
                        dim3(unsigned((a->N + 255) / 256), unsigned(pl.out_tiles), unsigned(pl.out_slots)), dim3(256), args, 0, st);
  return e == hipSuccess ? GEMM_W4A4_OK : GEMM_W4A4_ELAUNCH;
}

}  // namespace w4a4

extern "C" int lora_adapters(const lora_adapters_t* args, void* stream) { return w4a4::lora_adapters_run(args, stream); }

extern "C" int64_t lora_adapters_workspace(const lora_adapters_t* args) {
  return w4a4::adapt_sizes_ok(args) ? w4a4::adapt_plan(args).bytes : GEMM_W4A4_EINVAL;
}
