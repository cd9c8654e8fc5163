// attention.hip — attention of q to keys and values of another length
// (cross_attention in gemm_w4a4.h):
//
//   out[i] = sum_j exp(s_ij - m_i) v_j / sum_j exp(s_ij - m_i),  s_ij = scale q_i . k_j
//
// in one pass over the keys with a running maximum m and sum, kept in float32.
//
// Many rows are bound by the matrix cores and the exponentials (4 D flops and
// one exponential a score), few rows by reading K and V.
//
// The scores are computed transposed, S^T = K Q^T, in 32x32 tiles: a lane holds
// 16 keys of one query (the other 16 are in lane ^ 32), so the maximum and the
// sum over keys run inside the lane, and the exponentials, rounded to 16 bits,
// are the B operand of O^T = V^T P^T as they stand: the accumulator's key order
// (4 keys of each half in turn) is matched by reading V's rows in that order,
// with the transposing LDS read. Every factor of a query is one value a lane.
//
// K and V go to LDS by direct-to-LDS buffer loads. The
// descriptors end with the sequence's last key, so keys past kv_lens and the
// padding of head sizes to DP read as zeros, whatever memory holds there.
// 16-byte chunks are XOR-swizzled by row so that no read meets a bank twice (K:
// reads of 16 rows at one chunk; V: transposing reads of 4 rows at four).
//
// That rounding is what the matrix instruction costs: it takes 16-bit operands, and
// weights in float32 (or as two 16-bit parts) would run the second product at an
// eighth (half) of its rate. A weight is off by half a unit of the 16-bit type, out
// 1.2 to 1.4 times as far from 64 bits as with float32 weights (bfloat16 0.0021 to 0.0023 of its
// size against 0.0017, f16 0.00029 against 0.00021); the sum that divides is of
// the unrounded weights.
//
// Rows of a (sequence, key head) are (token, query head of the group) pairs, so
// heads that share keys share a tile. Few rows: the waves of a workgroup take
// different keys for the same 32 rows and join in LDS, and the keys of
// tiles that would fill no round of the compute units are cut into parts, a
// workgroup each, which a second launch joins, in order.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_w4a4.h"
#include "w4a4_buffer.hpp"
#include "w4a4_common.hpp"
#include "w4a4_half.hpp"
#include "w4a4_host.hpp"
#include "w4a4_strided.hpp"
#include "w4a4_transpose.hpp"
#include "w4a4_wave.hpp"

namespace w4a4 {

struct AttnParams {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  float* lse;
  const int32_t* kv_lens;
  float* part_o;       // the cut tiles' [tile][part][row of the tile][D] sums and
  float* part_ms;      // [tile][part][row of the tile][2] maximum (log2 units) and sum
  int64_t qs[3], ks[3], vs[3], os[3];   // batch, token, head
  int q_len, kv_len, kv_heads, D, group;   // group: query heads of a key head
  int rows;            // q_len * group
  int pairs;           // batch * kv_heads
  int whole;           // the first tiles are done whole; the keys of the cut tiles
  int cut, parts;      // after them in so many parts, a workgroup each
  int batch, per_seq;  // sequences; tiles of a sequence (row tiles x key heads)
  int even;            // 1: all tiles are cut, into parts of even length over the sequences
  float c;             // scale * log2(e)
};

// What a workgroup does: keys first .. first + len - 1 for row tile `tile` of
// (sequence, key head) `pair`. KT: keys are divided in multiples of it.
struct Share {
  int pair, tile, b, kvh;
  int first, len;
  int slot;            // of a cut tile: its part's place in the workspace; else -1
  bool idle;           // nothing to do
};

// Keys of sequence b in use.
__device__ __forceinline__ int keys_of(const AttnParams& p, int b) {
  return p.kv_lens ? min(max(p.kv_lens[b], 0), p.kv_len) : p.kv_len;
}

// Cutting sequences of uneven length into parts of even length: with T units of
// kUnit keys in a sequence and `per_seq` tiles of each, parts are Q units, the
// fewest with which all parts fit `parts` * `cut` workgroups, and a tile of the
// sequence has ceil(T / Q) of them. Their places in the workspace go by sequence,
// tile and part; workgroups take a sequence's tiles before its next part, so that
// the heads of the same keys, neighbours in memory, are read together (8 sequences
// of 0 to 8191 keys of 8 heads 31.8 to 31.4 us, 4 of 24 heads 45.5 to 44.5). Every lane of a wave looks at its own sequences (there are fewer than
// 256: every one has a tile, and tiles that fill a round are not cut).
constexpr int kUnit = 128;
struct EvenParts {
  int b, start, count, units;   // sequence, number of its first part, parts of a tile, units of a part
};

// The sequence of part number `at` (b < 0: past the last), or of sequence `want`.
__device__ __forceinline__ EvenParts even_parts(const AttnParams& p, int at, int want) {
  const int lane = threadIdx.x & 63;
  int64_t sum = 0;
  for (int c = lane; c < p.batch; c += 64) sum += (keys_of(p, c) + kUnit - 1) / kUnit;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
  const int64_t room = int64_t(p.cut) * p.parts - int64_t(p.per_seq) * p.batch;   // parts past one a tile
  EvenParts e;
  e.units = int(max(int64_t(2), (sum * p.per_seq + room - 1) / room));
  int base = 0;
  for (int c = 0; c < p.batch; c += 64) {
    const int b = c + lane;
    const int n = b < p.batch ? ((keys_of(p, b) + kUnit - 1) / kUnit + e.units - 1) / e.units : 0;
    int upto = n;   // of the lanes up to this one
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    const int start = base + p.per_seq * (upto - n);
    const uint64_t hit = __builtin_amdgcn_ballot_w64(want >= 0 ? b == want : at >= start && at < start + p.per_seq * n);
    if (hit) {
      const int from = __builtin_ctzll(hit);
      e.b = c + from;
      e.start = __builtin_amdgcn_readlane(start, from);
      e.count = __builtin_amdgcn_readlane(n, from);
      return e;
    }
    base += p.per_seq * __builtin_amdgcn_readlane(upto, 63);
  }
  e.b = -1;
  e.start = e.count = 0;
  return e;
}

template <int KT>
__device__ __forceinline__ Share share_of(const AttnParams& p) {
  Share w;
  const int idx = blockIdx.x;
  w.idle = false;
  if (p.even) {
    const EvenParts e = even_parts(p, idx, -1);
    w.idle = e.b < 0;
    if (w.idle) return w;
    const int part = (idx - e.start) / p.per_seq, nth = (idx - e.start) - part * p.per_seq;
    w.slot = e.start + nth * e.count + part;
    w.b = e.b;
    w.kvh = nth % p.kv_heads;
    w.tile = nth / p.kv_heads;
    w.pair = w.b * p.kv_heads + w.kvh;
    w.first = part * e.units * kUnit;
    w.len = __builtin_amdgcn_readfirstlane(min(keys_of(p, w.b) - w.first, e.units * kUnit));
    return w;
  }
  const bool cut = idx >= p.whole;
  const int part = cut ? (idx - p.whole) / p.cut : 0, nth = cut ? (idx - p.whole) % p.cut : 0;
  const int id = cut ? p.whole + nth : idx;
  w.slot = cut ? nth * p.parts + part : -1;
  w.pair = id % p.pairs;
  w.tile = id / p.pairs;
  w.b = w.pair / p.kv_heads;
  w.kvh = w.pair - w.b * p.kv_heads;
  const int len = __builtin_amdgcn_readfirstlane(keys_of(p, w.b));
  w.first = 0;
  w.len = len;
  if (cut) {
    const int64_t all = (len + KT - 1) / KT;
    w.first = int(all * part / p.parts) * KT;
    w.len = max(0, min(len, int(all * (part + 1) / p.parts) * KT) - w.first);
  }
  return w;
}

// Few rows: DP, the head size padded to 64, 96 or 128.
template <int DP_>
struct FewAttn {
  static constexpr int DP = DP_, WAVES = 4, THREADS = WAVES * kWave, ROWS = 32;
  static constexpr int KT = 32;                            // keys of a wave's tile
  static constexpr int ROWB = DP > 64 ? 256 : 128;         // bytes of a key's row in LDS
  static constexpr int CH = ROWB / 16;                     // 16-byte chunks of a row
  static constexpr int TILE = KT * ROWB;
  static constexpr int RPL = 1024 / ROWB;                  // rows a wave's load covers
  static constexpr int LOADS = KT / RPL;                   // loads of a tile
  static constexpr int SWZ = 16 / RPL;                     // loads after which the swizzles repeat
  static constexpr int LDS = WAVES * 2 * TILE;
  static constexpr int MERGE = (WAVES - 1) * 32 * (DP + 4) * 4;   // join of the waves' parts
  static_assert(MERGE <= LDS && 2 * LDS <= kLdsLimit, "two workgroups a compute unit");
};

// Position of chunk c of row r.
template <class C>
__device__ __forceinline__ int k_chunk(int r, int c) { return c ^ (C::CH == 16 ? r & 15 : (r >> 1) & 7); }
template <class C>
__device__ __forceinline__ int v_chunk(int r, int c) { return c ^ (C::CH == 16 ? (r & 3) << 2 : ((r >> 1) & 1) << 2); }

// A weight is exp2(s c - m), s c in one fma with the rounded maximum m, so that
// the top score's own is 2^r, r the rounding of its product: at most 1 up to this
// magnitude of m, and scores whose weights no longer fit a float32 (r = 128), or 16
// bits (r = 16), 2^8 or 2^4 times past it. Beyond it s c is rounded before m is taken
// away: the maximum's weight is 1, as it is in float32 scores.
constexpr float kFar = 16777216.f;
// (kept from being contracted into what it is subtracted from)
__device__ __forceinline__ float rounded_product(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}

// A row's result from its sums o (values 8 (i / 4) + 4 h + i % 4 of each 32),
// maximum m and sum l, or its part of them. r: the row in its tile.
template <bool F16, class C>
__device__ __forceinline__ void store_row(const AttnParams& p, const f32x16 (&o)[C::DP / 32], float m, float l,
                                          const Share& w, int r, int tok, int hq, int h) {
  constexpr int DT = C::DP / 32;
  const int D = p.D;
  if (w.slot >= 0) {
    const int64_t at = int64_t(w.slot) * C::ROWS + r;
    float* po = p.part_o + at * D;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int e = 32 * d + 2 * i + 4 * h;
        if (e < D) *reinterpret_cast<f32x4*>(po + e) = f32x4{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
      }
    if (h == 0) {
      p.part_ms[at * 2] = m;
      p.part_ms[at * 2 + 1] = l;
    }
    return;
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;   // a NaN sum stays one
  // 8 values a lane: the halves of a row swap runs of 4
  uint16_t* out = p.out + int64_t(w.b) * p.os[0] + int64_t(tok) * p.os[1] + int64_t(hq) * p.os[2];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
      const auto a = __builtin_amdgcn_permlane32_swap(narrow2<F16>(o[d][i] * inv, o[d][i + 1] * inv),
                                                      narrow2<F16>(o[d][i + 4] * inv, o[d][i + 5] * inv), false, false);
      const auto c = __builtin_amdgcn_permlane32_swap(narrow2<F16>(o[d][i + 2] * inv, o[d][i + 3] * inv),
                                                      narrow2<F16>(o[d][i + 6] * inv, o[d][i + 7] * inv), false, false);
      const int e = 32 * d + 2 * i + 8 * h;
      if (e < D) *reinterpret_cast<u32x4*>(out + e) = u32x4{uint32_t(a[0]), uint32_t(c[0]), uint32_t(a[1]), uint32_t(c[1])};
    }
  if (p.lse && h == 0)
    p.lse[(int64_t(w.b) * p.kv_heads * p.group + hq) * p.q_len + tok] =
        l == 0.f ? -INFINITY : (m + __builtin_log2f(l)) * 0.6931471805599453f;
}

// ------------------------------------------------------------------ few rows
//
// Bound by reading K and V. The waves of a workgroup take 32-key tiles of its
// share in turn, each through LDS of its own and without meeting the others: K
// of the next tile is asked for as soon as this one's scores have been read
// from it, V after the products, so that each of the 8 waves of a compute unit
// keeps 8 to 16 KiB in flight. They join in LDS at the end. 64 sequences of 8192
// keys, one token: 5.9 TB/s; 8 of 0 to 8191: 37 us, 3.6 TB/s, 5 of them the join.
template <bool F16, class C>
__global__ __launch_bounds__(C::THREADS, 2) void attention_few_kernel(const AttnParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::LDS];
  constexpr int DK = C::DP / 16, DT = C::DP / 32;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const Share w = share_of<C::KT * C::WAVES>(p);
  if (w.idle) return;
  const int b = w.b, kvh = w.kvh, len = w.len, D = p.D;
  const int nt = (len + C::KT - 1) / C::KT;

  // this lane's query row
  const int row = w.tile * C::ROWS + l32;
  const int rowc = min(row, p.rows - 1);
  const int tok = rowc / p.group, hq = kvh * p.group + rowc % p.group;
  u32x4 qv[DK];
  {
    const uint16_t* q = p.q + int64_t(b) * p.qs[0] + int64_t(tok) * p.qs[1] + int64_t(hq) * p.qs[2];
#pragma unroll
    for (int s = 0; s < DK; ++s) {
      const int d = 16 * s + 8 * h;
      qv[s] = d < D ? *reinterpret_cast<const u32x4*>(q + d) : u32x4{0u, 0u, 0u, 0u};
    }
  }

  // load u of a tile covers rows u RPL ..; lane -> (row, chunk position);
  // chunks past D are out of every range and read zeros
  const int dr = lane / C::CH, dp = lane % C::CH;
  const uint32_t kst = uint32_t(p.ks[1]) * 2u, vst = uint32_t(p.vs[1]) * 2u;   // token strides in bytes
  uint32_t koff[C::SWZ], voff[C::SWZ];
#pragma unroll
  for (int u = 0; u < C::SWZ; ++u) {
    const int r = u * C::RPL + dr, kc = k_chunk<C>(r, dp), vc = v_chunk<C>(r, dp);
    koff[u] = kc * 8 < D ? uint32_t(r) * kst + uint32_t(kc) * 16u : 0xFFFFFFF0u;
    voff[u] = vc * 8 < D ? uint32_t(r) * vst + uint32_t(vc) * 16u : 0xFFFFFFF0u;
  }
  const uint8_t* kb = reinterpret_cast<const uint8_t*>(p.k + int64_t(b) * p.ks[0] + int64_t(kvh) * p.ks[2] + int64_t(w.first) * p.ks[1]);
  const uint8_t* vb = reinterpret_cast<const uint8_t*>(p.v + int64_t(b) * p.vs[0] + int64_t(kvh) * p.vs[2] + int64_t(w.first) * p.vs[1]);
  const uint8_t* kt = smem + wave * 2 * C::TILE;
  const uint8_t* vt = kt + C::TILE;
  // the 16 rows from `half` on of tile t (an empty range past the last key: the
  // same loads, which read nothing, so that every wait counts alike)
  auto load = [&](const uint8_t* base, uint32_t stride, const uint32_t (&off)[C::SWZ], int t, uint32_t to) __attribute__((always_inline)) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r0 = t * C::KT + 16 * half, rows = min(len - r0, 16);
      const uint32_t any = uint32_t(-rows >> 31);   // all ones where rows > 0
      const u32x4 rs = range_desc(base + int64_t(r0) * stride, (uint32_t(rows - 1) * stride + uint32_t(D) * 2u) & any);
#pragma unroll
      for (int u = 0; u < C::SWZ; ++u) load_to_lds(rs, off[u], to + (half * C::SWZ + u) * 1024);
    }
  };
  const uint32_t kto = lds_address(kt), vto = lds_address(vt);
  const bool shared_memory = vst < uint32_t(D) * 2u;   // rows of v that overlap in memory

  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;   // maximum in log2 units; this lane's part of the sum

  if (wave < nt) {
    load(kb, kst, koff, wave, kto);
    load(vb, vst, voff, wave, vto);
  }
  for (int t = wave; t < nt; t += C::WAVES) {
    wait_vm<C::LOADS>();   // K of tile t; V's loads are younger
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    f32x16 sc;
#pragma unroll
    for (int s = 0; s < DK; ++s) {
      const u32x4 a = *reinterpret_cast<const u32x4*>(kt + l32 * C::ROWB + k_chunk<C>(l32, 2 * s + h) * 16);
      sc = mfma32<F16>(a, qv[s], s == 0 ? f32x16{} : sc);
    }
    __builtin_amdgcn_sched_barrier(0);
    wait_vm_lgkm0<63>();   // K is read
    load(kb, kst, koff, t + C::WAVES, kto);
    if ((t + 1) * C::KT > len) {   // the keys end in this tile
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (t * C::KT + 8 * (i >> 2) + 4 * h + (i & 3) >= len) sc[i] = -INFINITY;
    }
    float top = sc[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, sc[i]);
    top = other_max(top) * p.c;
    const float mn = fmaxf(m, top);
    const float ms = mn == -INFINITY ? 0.f : mn;   // no key yet, or none with weight
    if (__builtin_amdgcn_ballot_w64(mn != m)) {
      const float alpha = __builtin_amdgcn_exp2f(m - ms);
      l *= alpha;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= alpha;
    }
    m = mn;
    float cs = p.c;
    if (__builtin_amdgcn_ballot_w64(fabsf(ms) > kFar)) {
      const bool far = fabsf(ms) > kFar;
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[i] = far ? rounded_product(sc[i], p.c) : sc[i];
      cs = far ? 1.f : cs;
    }
    u32x4 pv[2];
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], cs, -ms));
      const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i + 1], cs, -ms));
      l += e0 + e1;
      pv[i >> 3][(i >> 1) & 3] = narrow2<F16>(e0, e1);
    }
    wait_vm<C::LOADS>();   // V of tile t; the next K's loads are younger
    asm volatile("" ::: "memory");
    if (shared_memory && (t + 1) * C::KT > len) {
      // rows past the last key have weight 0, but where rows overlap they are in
      // the descriptor's range and may hold an infinity: make them zeros
      for (int i = lane; i < C::TILE / 16; i += kWave)
        if (t * C::KT + i / C::CH >= len) *reinterpret_cast<u32x4*>(smem + (wave * 2 + 1) * C::TILE + i * 16) = u32x4{};
      wait_vm_lgkm0<63>();
      asm volatile("" ::: "memory");
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const int r = 16 * j + 4 * h + ((lane & 15) >> 2), run = 8 * d + 4 * ((lane >> 4) & 1) + (lane & 3);
        const uint8_t* v = vt + r * C::ROWB + v_chunk<C>(r, run >> 1) * 16 + (run & 1) * 8;
        const u32x2 lo = read_transposed(v), hi = read_transposed(v + 8 * C::ROWB);
        o[d] = mfma32<F16>(u32x4{lo.x, lo.y, hi.x, hi.y}, pv[j], o[d]);
      }
    __builtin_amdgcn_sched_barrier(0);
    wait_vm_lgkm0<63>();   // V is read
    load(vb, vst, voff, t + C::WAVES, vto);
  }
  wait_vm<0>();
  l = other_sum(l);

  // join the waves' keys: the others write their sums, maximum and sum; wave 0
  // adds them in order
  float* mg = reinterpret_cast<float*>(smem);
  constexpr int S = C::DP + 4;
  __syncthreads();
  if (wave != 0) {
    float* mine = mg + ((wave - 1) * 32 + l32) * S;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<f32x4*>(mine + 32 * d + 2 * i + 4 * h) = f32x4{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
    if (h == 0) {
      mine[C::DP] = m;
      mine[C::DP + 1] = l;
    }
  }
  __syncthreads();
  if (wave != 0) return;
  float mm = m;
#pragma unroll
  for (int v = 0; v < C::WAVES - 1; ++v) mm = fmaxf(mm, mg[(v * 32 + l32) * S + C::DP]);
  const float ms = mm == -INFINITY ? 0.f : mm;
  const float f0 = __builtin_amdgcn_exp2f(m - ms);
  l *= f0;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] *= f0;
#pragma unroll
  for (int v = 0; v < C::WAVES - 1; ++v) {
    const float* other = mg + (v * 32 + l32) * S;
    const float f = __builtin_amdgcn_exp2f(other[C::DP] - ms);
    l += other[C::DP + 1] * f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const f32x4 w4 = *reinterpret_cast<const f32x4*>(other + 32 * d + 2 * i + 4 * h);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][i + e] += w4[e] * f;
      }
  }
  if (row >= p.rows) return;
  store_row<F16, C>(p, o, mm, l, w, l32, tok, hq, h);
}

// ------------------------------------------------------------------ many rows
//
// 32 rows a wave, 4 waves a workgroup, two workgroups a compute unit, and each
// wave's own instructions overlapped: step j runs, all independent of each
// other, the score MFMAs of the 32 keys j + 1, the softmax of the 32 keys j on
// the vector ALU and the product MFMAs of the 32 keys j - 1. The step is
// written out MFMA by MFMA (products and scores in turn), each with its share
// of the softmax and of the operand reads of four MFMAs on, fenced so that the
// order stays.
//
// Rings of four 32-key tiles of K and of V, loaded two steps before they are
// read, one meeting of the workgroup a step. 4352 x 4608 keys, 24 heads of 128:
// 246 to 282 us from card to card, 873 to 1003 TFLOP/s of the 1228 that a large
// product reaches; the matrix cores, the exponentials and the LDS reads share the
// issue slots. 4096 x 512 keys: 34 to 39 us, 661 to 750 TFLOP/s, with 768 tiles for
// 512 places.
//
// The sums are rescaled only when a row's maximum has grown by more than
// kSlack (in powers of two) past the one its weights are taken against; until
// then weights are at most 2^kSlack, which float32 sums and the 16-bit types
// hold without loss.
constexpr float kSlack = 8.f;

template <int DP_>
struct WideAttn {
  static constexpr int DP = DP_, WAVES = 4, KT = 32, RING = 4;
  static constexpr int THREADS = WAVES * kWave;
  static constexpr int ROWS = WAVES * 32;
  static constexpr int ROWB = DP > 64 ? 256 : 128;
  static constexpr int CH = ROWB / 16;
  static constexpr int TILE = KT * ROWB;
  static constexpr int RPR = THREADS * 16 / ROWB;   // rows a round of loads covers
  static constexpr int ROUNDS = KT / RPR;           // rounds of a tile
  static constexpr int LDS = 2 * RING * TILE;       // K tiles, then V tiles
  static_assert(KT % RPR == 0 && ROUNDS >= 1 && RPR % 16 == 0, "whole rounds; the swizzles repeat every 16 rows");
  static_assert(2 * LDS <= kLdsLimit, "two workgroups a compute unit");
};

template <bool F16, class C>
__global__ __launch_bounds__(C::THREADS, 2) void attention_wide_kernel(const AttnParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::LDS];
  constexpr int DK = C::DP / 16, DT = C::DP / 32, VOFF = C::RING * C::TILE;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  // Two workgroups share a compute unit; the second of them (256 on) goes first
  // where both can issue, so that the two do not run in step and wait for the
  // same units (4352 x 4608 keys, 24 heads of 128: 265 to 256 us).
  if (blockIdx.x & 256) __builtin_amdgcn_s_setprio(2);
  const Share w = share_of<C::KT>(p);
  const int b = w.b, kvh = w.kvh, len = w.len, D = p.D;
  const int n = (len + C::KT - 1) / C::KT;

  const int row = w.tile * C::ROWS + wave * 32 + l32;
  const int rowc = min(row, p.rows - 1);
  const int tok = rowc / p.group, hq = kvh * p.group + rowc % p.group;
  u32x4 qv[DK];
  {
    const uint16_t* q = p.q + int64_t(b) * p.qs[0] + int64_t(tok) * p.qs[1] + int64_t(hq) * p.qs[2];
#pragma unroll
    for (int s = 0; s < DK; ++s) {
      const int d = 16 * s + 8 * h;
      qv[s] = d < D ? *reinterpret_cast<const u32x4*>(q + d) : u32x4{0u, 0u, 0u, 0u};
    }
  }

  // loads: round u covers rows u RPR .. of a tile; lane -> (row, chunk
  // position); chunks past D are out of every range and read zeros
  const int dr = tid / C::CH, dp = tid % C::CH;
  const int kc = k_chunk<C>(dr, dp), vc = v_chunk<C>(dr, dp);
  const uint32_t kst = uint32_t(p.ks[1]) * 2u, vst = uint32_t(p.vs[1]) * 2u;
  const bool klive = kc * 8 < D, vlive = vc * 8 < D;
  const uint32_t koff = klive ? uint32_t(dr) * kst + uint32_t(kc) * 16u : 0xFFFFFFF0u, kstep = klive ? C::RPR * kst : 0u;
  const uint32_t voff = vlive ? uint32_t(dr) * vst + uint32_t(vc) * 16u : 0xFFFFFFF0u, vstep = vlive ? C::RPR * vst : 0u;
  const uint8_t* kb = reinterpret_cast<const uint8_t*>(p.k + int64_t(b) * p.ks[0] + int64_t(kvh) * p.ks[2] + int64_t(w.first) * p.ks[1]);
  const uint8_t* vb = reinterpret_cast<const uint8_t*>(p.v + int64_t(b) * p.vs[0] + int64_t(kvh) * p.vs[2] + int64_t(w.first) * p.vs[1]);
  const uint32_t lds0 = lds_address(smem) + wave * 1024;
  // Tile t of K (to ring place t % RING) or V; tiles past the last key are
  // empty ranges: zeros (by a mask and no branch, so that a step stays one block).
  auto load = [&](const uint8_t* base, uint32_t stride, uint32_t off, uint32_t step, int t, uint32_t to) __attribute__((always_inline)) {
    const int rows = min(len - t * C::KT, C::KT);
    const uint32_t any = uint32_t(-rows >> 31);   // all ones where rows > 0
    const u32x4 rs = range_desc(base + int64_t(t * C::KT) * stride, (uint32_t(rows - 1) * stride + uint32_t(D) * 2u) & any);
#pragma unroll
    for (int u = 0; u < C::ROUNDS; ++u) load_to_lds(rs, off + u * step, lds0 + to + u * C::RPR * C::ROWB);
  };
  auto load_k = [&](int t, int ring) __attribute__((always_inline)) { load(kb, kst, koff, kstep, t, ring * C::TILE); };
  auto load_v = [&](int t, int ring) __attribute__((always_inline)) { load(vb, vst, voff, vstep, t, VOFF + ring * C::TILE); };

  // this lane's LDS addresses in the rings' first tiles, by slot
  uint32_t kaddr[DK], vaddr[DT];
#pragma unroll
  for (int i = 0; i < DK; ++i) kaddr[i] = l32 * C::ROWB + k_chunk<C>(l32, 2 * i + h) * 16;
#pragma unroll
  for (int d = 0; d < DT; ++d) {
    const int r = 4 * h + ((lane & 15) >> 2), run = 8 * d + 4 * ((lane >> 4) & 1) + (lane & 3);
    vaddr[d] = VOFF + r * C::ROWB + v_chunk<C>(r, run >> 1) * 16 + (run & 1) * 8;
  }
  // K operand of score slot i (16 of D); V operand of product slot i: 16 keys
  // i / DT, 32 of D i % DT
  auto read_k = [&](int ring, int i) __attribute__((always_inline)) {
    return *reinterpret_cast<const u32x4*>(smem + kaddr[i] + ring * C::TILE);
  };
  auto read_v = [&](int ring, int i) __attribute__((always_inline)) {
    const uint8_t* v = smem + vaddr[i % DT] + (ring * C::TILE + i / DT * 16 * C::ROWB);
    const u32x2 lo = read_transposed(v), hi = read_transposed(v + 8 * C::ROWB);
    return u32x4{lo.x, lo.y, hi.x, hi.y};
  };

  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;
  f32x16 sc[2];         // scores, by key tile's parity
  u32x4 pv[2][2];       // weights, likewise
  u32x4 ka[2], va[2];   // operands of the next two score and product slots

  // The softmax of a step in parts: the maximum by quarters and what follows
  // from it, then the weights one key at a time.
  constexpr int FIN = 8, PARTS = FIN + 16;
  float alpha, ms, top, grown, drop, lold, e[4];
  auto soft = [&]<bool TAIL>(int part, f32x16& s, u32x4 (&wt)[2], int key0) __attribute__((always_inline)) {
    if (part < 4) {
      if constexpr (TAIL) {
#pragma unroll
        for (int i = 4 * part; i < 4 * part + 4; ++i)
          if (key0 + 8 * (i >> 2) + 4 * h + (i & 3) >= len) s[i] = -INFINITY;
      }
      float t = part == 0 ? s[0] : top;
#pragma unroll
      for (int i = 4 * part; i < 4 * part + 4; ++i) t = fmaxf(t, s[i]);
      top = t;
    } else if (part == 4) {
      top = other_max(top);
    } else if (part == 5) {
      // the maximum in use grows, or stays and alpha, the factor of what was
      // summed before, is 1 (the first keys: m is -inf)
      top *= p.c;
      grown = top - m > kSlack ? top : m;
    } else if (part == 6) {
      drop = m == grown ? 0.f : m - grown;
      ms = grown == -INFINITY ? 0.f : grown;
      m = grown;
    } else if (part == 7) {
      alpha = __builtin_amdgcn_exp2f(drop);
      l *= alpha;
      lold = l;
    } else {
      // an exponential is used one part after it was asked for
      const int i = part - FIN;
      if (i > 0) l += e[(i - 1) & 3];
      if (i > 0 && i % 2 == 0) wt[(i - 2) >> 3][((i - 2) >> 1) & 3] = narrow2<F16>(e[(i - 2) & 3], e[(i - 1) & 3]);
      e[i & 3] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], p.c, -ms));
      if (i == 15) {
        l += e[3];
        wt[1][3] = narrow2<F16>(e[2], e[3]);
      }
    }
  };
  // Where each part goes: in proportion to cycles, counting the latency of
  // chained instructions, after a lead in which the last scores come in.
  constexpr int kLead = 40, kMaxCost = 20, kFinCost = 28, kKeyCost = 18, MFMAS = 2 * DK;
  constexpr auto cost_before = [](int part) {
    int c = kLead;
    for (int i = 0; i < part; ++i) c += i < 4 ? kMaxCost : i < FIN ? kFinCost : kKeyCost;
    return c;
  };
  constexpr auto first_part = [=](int mfma) {   // the first part at or after MFMA `mfma`'s share
    int i = 0;
    while (i < PARTS && cost_before(i) * MFMAS < cost_before(PARTS) * mfma) ++i;
    return i;
  };
  // Step j; R: j % RING. Reads K tile j + 1 and V tile j - 1 and, at its end,
  // the first operands of step j + 1 (K tile j + 2, V tile j). In its second
  // half, after the workgroup has met, K tile j + 4 and V tile j + 2 go to LDS, over
  // K tile j and V tile j - 2, which every wave last read in step j - 1: that meeting
  // is all that keeps the loads behind those reads. The loads are waited for at the
  // meeting of step j + 2 (only those of step j + 1 are younger), which publishes
  // them; K tile j + 4 and V tile j + 2 are first read at that step's end.
  auto step = [&]<bool TAIL, int R>(int j) __attribute__((always_inline)) {
    constexpr int P = R & 1;
    static_for<0, MFMAS>([&]<int I>() __attribute__((always_inline)) {
      constexpr int i = I / 2;
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (I == MFMAS / 2) {
        wait_vm<2 * C::ROUNDS>();
        wg_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (I % 2 == 0) {
        o[i % DT] = mfma32<F16>(va[i % 2], pv[1 - P][i / DT], o[i % DT]);
        va[i % 2] = i + 2 < DK ? read_v((R + 3) & 3, i + 2) : read_v(R, i + 2 - DK);
      } else {
        sc[1 - P] = mfma32<F16>(ka[i % 2], qv[i], i == 0 ? f32x16{} : sc[1 - P]);
        ka[i % 2] = i + 2 < DK ? read_k((R + 1) & 3, i + 2) : read_k((R + 2) & 3, i + 2 - DK);
      }
      static_for<first_part(I), first_part(I + 1)>([&]<int PART>() __attribute__((always_inline)) {
        soft.template operator()<TAIL>(PART, sc[P], pv[P], j * C::KT);
      });
      if constexpr (I == MFMAS / 2) load_k(j + 4, R);
      if constexpr (I == MFMAS / 2 + 1) load_v(j + 2, (R + 2) & 3);
    });
    __builtin_amdgcn_sched_barrier(0);
    // (the compiler would move the weights past the branch, away from the MFMAs)
    asm volatile("" : "+v"(pv[P][0]), "+v"(pv[P][1]), "+v"(l));
    if (__builtin_amdgcn_ballot_w64(alpha != 1.f || fabsf(ms) > kFar)) {
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= alpha;
      if (fabsf(ms) > kFar) {   // these rows' weights and sum again, scores rounded first
        l = lold;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float e0 = __builtin_amdgcn_exp2f(rounded_product(sc[P][i], p.c) - ms);
          const float e1 = __builtin_amdgcn_exp2f(rounded_product(sc[P][i + 1], p.c) - ms);
          l += e0 + e1;
          pv[P][i >> 3][(i >> 1) & 3] = narrow2<F16>(e0, e1);
        }
      }
    }
  };
  static_assert(C::RING == 4 && MFMAS >= 8, "the step above");

  if (n > 0) {
    // zeros stand in for the values before the first
    for (int i = tid * 16; i < C::TILE; i += C::THREADS * 16) *reinterpret_cast<u32x4*>(smem + VOFF + 3 * C::TILE + i) = u32x4{0u, 0u, 0u, 0u};
    load_k(0, 0);
    load_k(1, 1);
    load_v(0, 0);
    load_k(2, 2);
    load_v(1, 1);
    load_k(3, 3);
    wait_vm_lgkm0<4 * C::ROUNDS>();
    wg_barrier();
#pragma unroll
    for (int i = 0; i < DK; ++i) sc[0] = mfma32<F16>(read_k(0, i), qv[i], i == 0 ? f32x16{} : sc[0]);
    pv[1][0] = pv[1][1] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ka[i] = read_k(1, i);
      va[i] = read_v(3, i);
    }
    const int full = len / C::KT;
    int j = 0;
    for (; j + 4 <= full; j += 4) {
      step.template operator()<false, 0>(j);
      step.template operator()<false, 1>(j + 1);
      step.template operator()<false, 2>(j + 2);
      step.template operator()<false, 3>(j + 3);
    }
    if (j < n) step.template operator()<true, 0>(j);
    if (j + 1 < n) step.template operator()<true, 1>(j + 1);
    if (j + 2 < n) step.template operator()<true, 2>(j + 2);
    if (j + 3 < n) step.template operator()<true, 3>(j + 3);
    wait_vm<0>();
    // products of the last 32 keys
    const int last = (n - 1) & 3;
    const bool odd = last & 1;
    const u32x4 w0 = odd ? pv[1][0] : pv[0][0], w1 = odd ? pv[1][1] : pv[0][1];
#pragma unroll
    for (int i = 0; i < DK; ++i)
      o[i % DT] = mfma32<F16>(i < 2 ? va[i] : read_v(last, i), i / DT == 0 ? w0 : w1, o[i % DT]);
  }

  if (row >= p.rows) return;
  l = other_sum(l);
  store_row<F16, C>(p, o, m, l, w, wave * 32 + l32, tok, hq, h);
}

// Joins the parts of the cut tiles' rows, in order: one thread per 4 values,
// blockIdx.y the cut tile.
template <bool F16>
__global__ __launch_bounds__(256) void attention_join_kernel(const AttnParams p, int tile_rows) {
  const int per = p.D / 4, nth = blockIdx.y, id = p.whole + nth;
  int pair = id % p.pairs, tile = id / p.pairs, parts = p.parts;
  int64_t slot = int64_t(nth) * p.parts;
  if (p.even) {   // nth: (sequence, row tile, key head)
    const EvenParts e = even_parts(p, -1, nth / p.per_seq);
    const int in = nth % p.per_seq;
    pair = e.b * p.kv_heads + in % p.kv_heads;
    tile = in / p.kv_heads;
    parts = e.count;
    slot = e.start + int64_t(in) * parts;
  }
  const int i = blockIdx.x * 256 + threadIdx.x, r = i / per, row = tile * tile_rows + r;
  if (r >= tile_rows || row >= p.rows) return;
  const int e = (i - r * per) * 4;
  const int64_t at = slot * tile_rows + r;
  const float* ms = p.part_ms + at * 2;
  const float* po = p.part_o + at * p.D + e;
  // eight parts at a time, their loads in flight together
  float mm = -INFINITY, l = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = 0; s0 < parts; s0 += 8) {
    float pm[8], pl[8];
    f32x4 po8[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t s = min(s0 + k, parts - 1);
      pm[k] = s0 + k < parts ? ms[s * tile_rows * 2] : -INFINITY;
      pl[k] = ms[s * tile_rows * 2 + 1];
      po8[k] = *reinterpret_cast<const f32x4*>(po + s * tile_rows * p.D);
    }
    float mn = mm;
#pragma unroll
    for (int k = 0; k < 8; ++k) mn = fmaxf(mn, pm[k]);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float f0 = __builtin_amdgcn_exp2f(mm - base);
    l *= f0;
    o *= f0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s0 + k < parts) {
        const float f = __builtin_amdgcn_exp2f(pm[k] - base);
        l += pl[k] * f;
        o += po8[k] * f;
      }
    mm = mn;
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  const int b = pair / p.kv_heads, tok = row / p.group, hq = (pair - b * p.kv_heads) * p.group + row % p.group;
  uint16_t* out = p.out + int64_t(b) * p.os[0] + int64_t(tok) * p.os[1] + int64_t(hq) * p.os[2];
  *reinterpret_cast<u32x2*>(out + e) = u32x2{narrow2<F16>(o.x * inv, o.y * inv), narrow2<F16>(o.z * inv, o.w * inv)};
  if (p.lse && e == 0)
    p.lse[(int64_t(b) * p.kv_heads * p.group + hq) * p.q_len + tok] = l == 0.f ? -INFINITY : (mm + __builtin_log2f(l)) * 0.6931471805599453f;
}

// ------------------------------------------------------------------ host side

struct AttnPlan {
  bool few;      // 32-row tiles, waves over the keys
  int rows, tiles, pairs, rows_all;
  int64_t whole;
  int cut, parts;
  bool even;
  int64_t o_bytes, bytes;
};

static bool attn_sizes_ok(const cross_attention_t* a) {
  if (!a || a->batch < 0 || a->q_len < 0 || a->kv_len < 0 || a->q_heads < 0 || a->kv_heads < 1) return false;
  if (a->q_heads % a->kv_heads != 0) return false;
  if (a->head_dim < 8 || a->head_dim > CROSS_ATTENTION_MAX_HEAD_DIM || a->head_dim % 8 != 0) return false;
  // Rows and keys are counted in int, rounded up to tiles and, for loads asked for
  // ahead, a few tiles past the end.
  const int64_t lim = int64_t(1) << 31, most = lim - CROSS_ATTENTION_PAST_END;
  return int64_t(a->q_len) * a->q_heads <= most && a->kv_len <= most && int64_t(a->batch) * a->kv_heads < lim / 256 &&
         int64_t(a->batch) * a->q_len * a->q_heads < lim;
}

// Tiles and which of them are cut. Up to 32 rows (token, query head of the
// group) a pair, or rows of v that overlap in memory (which only that kernel
// masks): the few-row kernel; else 128-row tiles; two workgroups a compute unit.
// Both measured (us, 32-row tiles against 128-row ones): 32 rows, 512 pairs of 1024
// keys 53.0 and 54.9, 128 pairs of 0 to 8191 of head size 64 41.8 and 49.8, 24 pairs
// of 512 10.2 and 11.6; 33 rows 88.4 and 55.8, 79.9 and 51.3, 10.3 and 11.7; 128 rows
// 164 and 63.6, 96.7 and 56.4, 12.3 and 14.8. Past 32 rows 32-row tiles read the keys
// more than once, which costs up to three times where the tiles fill the chip and gains
// up to 1.4 times where they do not (32 pairs of 4096 keys, 128 rows: 26.8 and 38.0).
// Tiles that fill no whole round of the compute
// units are cut into the parts that would fill it, of at least kMinPart keys;
// where sequences have lengths of their own and few rows, into parts of even
// length (8 sequences of 0 to 8191 keys, one token: 41.2 to 37.0 us).
static AttnPlan attn_plan(const cross_attention_t* a) {
  constexpr int kMinPart = 256;
  AttnPlan pl{};
  const int group = a->q_heads / a->kv_heads;
  pl.rows_all = a->q_len * group;
  pl.pairs = a->batch * a->kv_heads;
  pl.few = pl.rows_all <= 32 || (a->kv_len > 1 && a->v_stride[1] < a->head_dim);
  pl.rows = pl.few ? 32 : 128;
  pl.tiles = (pl.rows_all + pl.rows - 1) / pl.rows;
  pl.whole = int64_t(pl.tiles) * pl.pairs;
  pl.parts = 1;
  const int left = int(pl.whole % kNumCUs);
  if (left > 0) {
    const int slots = pl.whole < kNumCUs ? 2 * kNumCUs : kNumCUs;
    const int parts = std::min(slots / left, a->kv_len / kMinPart);
    if (parts > 1) {
      pl.parts = parts;
      pl.cut = left;
      pl.whole -= left;
      // (a sequence's part count follows its length on the device)
      pl.even = pl.few && pl.whole == 0 && a->kv_lens && a->batch > 1;
      const int64_t n = int64_t(left) * parts * pl.rows;
      pl.o_bytes = n * a->head_dim * 4;
      pl.bytes = pl.o_bytes + n * 8;
    }
  }
  return pl;
}

template <bool F16>
static const void* attention_of(bool few, int D) {
  if (few)
    return D <= 64 ? reinterpret_cast<const void*>(attention_few_kernel<F16, FewAttn<64>>)
         : D <= 96 ? reinterpret_cast<const void*>(attention_few_kernel<F16, FewAttn<96>>)
                   : reinterpret_cast<const void*>(attention_few_kernel<F16, FewAttn<128>>);
  return D <= 64 ? reinterpret_cast<const void*>(attention_wide_kernel<F16, WideAttn<64>>)
       : D <= 96 ? reinterpret_cast<const void*>(attention_wide_kernel<F16, WideAttn<96>>)
                 : reinterpret_cast<const void*>(attention_wide_kernel<F16, WideAttn<128>>);
}

static int attention_run(const cross_attention_t* a, void* stream) {
  if (!attn_sizes_ok(a) || (a->f16 | 1) != 1 || !(a->scale > 0.f && a->scale <= 1e30f)) return GEMM_W4A4_EINVAL;
  const int qsz[3] = {a->batch, a->q_len, a->q_heads}, ksz[3] = {a->batch, a->kv_len, a->kv_heads};
  const int D = a->head_dim;
  const int64_t qe = strided_extent(qsz, a->q_stride, D), ke = strided_extent(ksz, a->k_stride, D),
                ve = strided_extent(ksz, a->v_stride, D), oe = strided_extent(qsz, a->out_stride, D);
  if (qe < 0 || ke < 0 || ve < 0 || oe < 0 || !strides_apart(qsz, a->out_stride, D)) return GEMM_W4A4_EINVAL;
  const bool keys = a->kv_len > 0;
  for (int i = 0; i < 3; ++i) {
    if (qsz[i] > 1 && ((a->q_stride[i] | a->out_stride[i]) & 7)) return GEMM_W4A4_EINVAL;
    if (ksz[i] > 1 && ((a->k_stride[i] | a->v_stride[i]) & 7)) return GEMM_W4A4_EINVAL;
  }
  if (a->kv_len > 1 && (a->k_stride[1] >= (int64_t(1) << 23) || a->v_stride[1] >= (int64_t(1) << 23))) return GEMM_W4A4_EINVAL;
  if (a->batch == 0 || a->q_len == 0 || a->q_heads == 0) return GEMM_W4A4_OK;
  if (!a->q || !a->out || (keys && (!a->k || !a->v))) return GEMM_W4A4_EINVAL;
  if ((uintptr_t(a->q) | uintptr_t(a->out) | (keys ? uintptr_t(a->k) | uintptr_t(a->v) : 0u)) & 15u) return GEMM_W4A4_EALIGN;
  if ((uintptr_t(a->lse) | uintptr_t(a->kv_lens)) & 3u) return GEMM_W4A4_EALIGN;
  const AttnPlan pl = attn_plan(a);
  if (pl.bytes > 0) {
    if (!a->workspace || a->workspace_bytes < pl.bytes) return GEMM_W4A4_ESCRATCH;
    if (uintptr_t(a->workspace) & 15u) return GEMM_W4A4_EALIGN;
  }
  const struct { const void* p; size_t n; } outs[] = {
      {a->out, size_t(oe) * 2}, {a->lse, size_t(a->batch) * size_t(a->q_heads) * size_t(a->q_len) * 4},
      {pl.bytes > 0 ? a->workspace : nullptr, size_t(pl.bytes)}};
  const struct { const void* p; size_t n; } ins[] = {
      {a->q, size_t(qe) * 2}, {keys ? a->k : nullptr, size_t(ke) * 2}, {keys ? a->v : nullptr, size_t(ve) * 2},
      {a->kv_lens, size_t(a->batch) * 4}};
  for (int x = 0; x < 3; ++x) {
    for (const auto& in : ins)
      if (overlaps(outs[x].p, outs[x].n, in.p, in.n)) return GEMM_W4A4_EOVERLAP;
    for (int y = x + 1; y < 3; ++y)
      if (overlaps(outs[x].p, outs[x].n, outs[y].p, outs[y].n)) return GEMM_W4A4_EOVERLAP;
  }
  const int dev_rc = check_device();
  if (dev_rc != GEMM_W4A4_OK) return dev_rc;

  AttnParams p{};
  p.q = static_cast<const uint16_t*>(a->q);
  p.k = static_cast<const uint16_t*>(a->k);
  p.v = static_cast<const uint16_t*>(a->v);
  p.out = static_cast<uint16_t*>(a->out);
  p.lse = a->lse;
  p.kv_lens = a->kv_lens;
  p.part_o = static_cast<float*>(a->workspace);
  p.part_ms = pl.bytes > 0 ? p.part_o + pl.o_bytes / 4 : nullptr;
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = a->q_stride[i];
    p.ks[i] = a->k_stride[i];
    p.vs[i] = a->v_stride[i];
    p.os[i] = a->out_stride[i];
  }
  if (a->kv_len <= 1) p.ks[1] = p.vs[1] = D;   // the stride of a single key is not the caller's to keep
  p.q_len = a->q_len;
  p.kv_len = a->kv_len;
  p.kv_heads = a->kv_heads;
  p.D = D;
  p.group = a->q_heads / a->kv_heads;
  p.rows = pl.rows_all;
  p.pairs = pl.pairs;
  p.whole = int(std::min<int64_t>(pl.whole, INT32_MAX));
  p.cut = pl.cut;
  p.batch = a->batch;
  p.per_seq = pl.tiles * a->kv_heads;
  p.even = pl.even;
  p.parts = pl.parts;
  p.c = a->scale * 1.4426950408889634f;
  int tile_rows = pl.rows;
  void* args[] = {&p, &tile_rows};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t grid = pl.whole + int64_t(pl.cut) * pl.parts;
  if (grid >= (int64_t(1) << 31)) return GEMM_W4A4_EINVAL;
  hipError_t e = hipLaunchKernel(a->f16 ? attention_of<true>(pl.few, D) : attention_of<false>(pl.few, D),
                                 dim3(unsigned(grid)), dim3(256), args, 0, st);
  if (e == hipSuccess && pl.cut > 0) {
    const int rows = std::min(pl.rows, pl.rows_all);
    e = hipLaunchKernel(a->f16 ? reinterpret_cast<const void*>(attention_join_kernel<true>)
                               : reinterpret_cast<const void*>(attention_join_kernel<false>),
                        dim3(unsigned((rows * (D / 4) + 255) / 256), unsigned(pl.cut)), dim3(256), args, 0, st);
  }
  return e == hipSuccess ? GEMM_W4A4_OK : GEMM_W4A4_ELAUNCH;
}

}  // namespace w4a4

extern "C" int cross_attention(const cross_attention_t* args, void* stream) { return w4a4::attention_run(args, stream); }

extern "C" int64_t cross_attention_workspace(const cross_attention_t* args) {
  return w4a4::attn_sizes_ok(args) ? w4a4::attn_plan(args).bytes : GEMM_W4A4_EINVAL;
}
