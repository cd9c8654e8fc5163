// w4a4_attention.hpp — the attention kernels, shared by cross_attention
// (attention.hip), packed_attention (packed_attention.hip) and paged_attention
// (paged_attention.hip): their mathematics and layouts stand in attention.hip. What the
// three differ in is where rows and keys lie and which keys a row sees.
#pragma once

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
#include "w4a4_page_index.hpp"
#include "w4a4_strided.hpp"
#include "w4a4_transpose.hpp"
#include "w4a4_wave.hpp"

namespace w4a4 {

// Where rows and keys lie.
enum class Attend {
  kDense,    // sequences one stride apart, keys of another length for all rows
  kPacked,   // sequences one after the other in one run of tokens, their own keys; causal or not
  kPaged,    // keys in pages; the rows are each sequence's newest tokens
};

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
  // packed: sequence s is the tokens starts[s] .. starts[s + 1] - 1 of q_len
  const int32_t* starts;
  int seqs, causal;
  // paged: page table[b][i] holds keys i page_size .. of sequence b; ks[0], vs[0]: stride of pages
  const int32_t* table;
  int64_t table_stride;
  int page_size, pages;
  PageIndex page_index;
};

// The parameters, read once more: what only the end of a kernel needs and would be kept over
// its main loop (where the scalar registers are spilled) if it were taken from `p`.
__device__ __forceinline__ const AttnParams& params_again() {
  auto at = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(at));
  return *(const AttnParams*)at;
}

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

// Sum over the wave, in every lane.
__device__ __forceinline__ int wave_sum_int(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, true);
  auto r = __builtin_amdgcn_permlane16_swap(uint32_t(v), uint32_t(v), false, false);
  v = int(uint32_t(r[0]) + uint32_t(r[1]));
  r = __builtin_amdgcn_permlane32_swap(uint32_t(v), uint32_t(v), false, false);
  return __builtin_amdgcn_readfirstlane(int(uint32_t(r[0]) + uint32_t(r[1])));
}

// First token and tokens of packed sequence s; starts that fall or leave 0 .. q_len are
// taken to the nearest that do not.
__device__ __forceinline__ int packed_start(const AttnParams& p, int s) { return min(max(p.starts[s], 0), p.q_len); }
__device__ __forceinline__ int packed_len(const AttnParams& p, int s) { return max(packed_start(p, s + 1) - packed_start(p, s), 0); }

// Packed sequences: workgroups take key heads, and for each the row tiles of all sequences
// by their place in the sequence, the last ones first: with the mask these have the most
// keys, so that the longest work begins first. With F(t) tiles at place t or later, tile
// number n of all is at the last place t with F(t) > n, and there the one of the
// (n - F(t + 1))-th sequence that has a tile at that place.
//
// Up to 64 sequences a lane of each wave has one; past that a thread of the workgroup has
// kSeqs, and the waves' sums meet in LDS.
constexpr int kSeqs = 16;
static_assert(kSeqs * 256 == PACKED_ATTENTION_MAX_SEQS, "a place for every sequence");
struct PackedTile {
  int seq, tile, start, len;   // seq < 0: past the last
};
template <int ROWS, bool MANY>
__device__ __forceinline__ PackedTile packed_tile(const AttnParams& p, int n) {
  constexpr int SEQS = MANY ? kSeqs : 1, WAVES = 4;
  __shared__ int meet[2][WAVES];
  __shared__ int found;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int own[SEQS];   // tiles of this thread's sequences
#pragma unroll
  for (int i = 0; i < SEQS; ++i) {
    const int s = MANY ? tid + 256 * i : lane;
    own[i] = s < p.seqs ? int((int64_t(packed_len(p, s)) * p.group + ROWS - 1) / ROWS) : 0;
  }
  int turn = 0;
  auto sum = [&](int v) __attribute__((always_inline)) {
    v = wave_sum_int(v);
    if constexpr (MANY) {
      // (two places in turn: a wave may still read the last sum's while another writes the next)
      if (lane == 0) meet[turn][wave] = v;
      __syncthreads();
      v = __builtin_amdgcn_readfirstlane(meet[turn][0] + meet[turn][1] + meet[turn][2] + meet[turn][3]);
      turn ^= 1;
    }
    return v;
  };
  auto from = [&](int t) __attribute__((always_inline)) {
    int f = 0;
#pragma unroll
    for (int i = 0; i < SEQS; ++i) f += max(own[i] - t, 0);
    return sum(f);
  };
  PackedTile w{-1, 0, 0, 0};
  if (n >= from(0)) return w;
  int lo = 0, hi = int((int64_t(p.q_len) * p.group + ROWS - 1) / ROWS);   // F(hi) = 0
  if constexpr (MANY) {   // (their longest is mostly far shorter: 400 of 8 tokens 49 us, 59 without; 100 of 100 27 and 29)
    int most = own[0];
#pragma unroll
    for (int i = 1; i < SEQS; ++i) most = max(most, own[i]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) most = max(most, __shfl_xor(most, d));
    if (lane == 0) meet[turn][wave] = most;
    __syncthreads();
    hi = __builtin_amdgcn_readfirstlane(max(max(meet[turn][0], meet[turn][1]), max(meet[turn][2], meet[turn][3])));
    turn ^= 1;
  }
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (from(mid) > n) lo = mid;
    else hi = mid;
  }
  const int nth = n - from(lo + 1);   // among the sequences with a tile at this place
  if constexpr (!MANY) {
    const uint64_t has = __builtin_amdgcn_ballot_w64(own[0] > lo);
    const int rank = __builtin_popcountll(has & ((uint64_t(1) << lane) - 1));
    const uint64_t hit = __builtin_amdgcn_ballot_w64((has >> lane & 1) && rank == nth);
    if (hit == 0) return w;
    w.seq = __builtin_ctzll(hit);
  } else {
    // by thread, and for a thread by its own order
    int mine = 0;
#pragma unroll
    for (int i = 0; i < SEQS; ++i) mine += own[i] > lo;
    int upto = mine;   // of the wave's lanes up to this one
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(upto, d);
      if (lane >= d) upto += v;
    }
    if (lane == 63) meet[turn][wave] = upto;
    if (tid == 0) found = -1;
    __syncthreads();
    int before = upto - mine;
    for (int v = 0; v < wave; ++v) before += meet[turn][v];
#pragma unroll
    for (int i = 0; i < SEQS; ++i)
      if (own[i] > lo && before++ == nth) found = tid + 256 * i;
    __syncthreads();
    w.seq = __builtin_amdgcn_readfirstlane(found);
    if (w.seq < 0) return w;
  }
  w.tile = lo;
  w.start = __builtin_amdgcn_readfirstlane(packed_start(p, w.seq));
  w.len = __builtin_amdgcn_readfirstlane(packed_len(p, w.seq));
  return w;
}

template <class C, Attend A, int KT>
__device__ __forceinline__ Share share_of(const AttnParams& p, int& rows, int& origin) {
  Share w;
  const int idx = blockIdx.x;
  w.idle = false;
  if constexpr (A == Attend::kPacked) {
    const int n = idx / p.kv_heads;
    const PackedTile at = p.seqs <= 64 ? packed_tile<C::ROWS, false>(p, n) : packed_tile<C::ROWS, true>(p, n);
    w.idle = at.seq < 0;
    if (w.idle) return w;
    rows = at.len * p.group;
    origin = at.start;
    w.b = w.pair = 0;
    w.kvh = idx - n * p.kv_heads;
    w.tile = at.tile;
    w.first = 0;
    w.slot = -1;
    w.len = p.causal ? min(at.len, (min(rows, (at.tile + 1) * C::ROWS) - 1) / p.group + 1) : at.len;
    return w;
  }
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
  if constexpr (A == Attend::kPaged) w.tile = p.per_seq / p.kv_heads - 1 - w.tile;   // the last rows see the most keys
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

// Paged: the table's entries page0 .. page0 + 63 of sequence b, one a lane.
struct Pages {
  const AttnParams& p;
  int b, page0 = 0, entries = -1;
  __device__ __forceinline__ void look(int from) {
    page0 = from;
    const int64_t at = int64_t(from) + (threadIdx.x & 63);
    entries = at * p.page_size < p.kv_len ? p.table[int64_t(b) * p.table_stride + at] : -1;
  }
  __device__ __forceinline__ int place_of(int key) const { return p.page_index.of(key); }
  // the page that holds key `key` of the sequence: its number in the cache, -1 where there is none
  __device__ __forceinline__ int page_of(int key) {
    const int i = place_of(key);
    if (i < page0 || i >= page0 + 64) look(i);
    return held(key);
  }
  // likewise of a key whose entry is held
  __device__ __forceinline__ int held(int key) const {
    const int e = __builtin_amdgcn_readlane(entries, place_of(key) - page0);
    return e >= 0 && e < p.pages ? e : -1;
  }
  // the bytes from a cache's start to that key, `stride` a token
  __device__ __forceinline__ int64_t key_at(int key, int page, int64_t page_stride, uint32_t stride) const {
    const int i = place_of(key);
    return int64_t(page) * page_stride * 2 + int64_t(key - i * p.page_size) * stride;
  }
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

// A lane's row again, key by key, leaving out the keys that it does not see: its sums o, maximum m
// and (in the lower half of the wave) sum of weights l. In the matrix product those keys have weight 0, which
// is not enough where a value is an infinity or a NaN: 0 times it is NaN. Taken when a sum is one
// and a value that some row does not see is one; slow (some 300 instructions a key).
// m and l come from the scores used here: theirs are summed in another order than the matrix
// instruction's, and of large ones a weight would differ by any factor from the one in l.
// `keys` calls its argument with every key's index and the addresses of its k and v rows.
template <bool F16, class C, class F>
__device__ __forceinline__ void careful_sums(f32x16 (&o)[C::DP / 32], const u32x4 (&qv)[C::DP / 16], int D, float c, float& m, float& l,
                                                       int lim, F&& keys) {
  constexpr int DK = C::DP / 16, DT = C::DP / 32;
  const int h = (threadIdx.x & 63) >> 5;
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  keys([&](int j, const uint16_t* k, const uint16_t* v) __attribute__((always_inline)) {
    int Dk = D;
    asm volatile("" : "+s"(Dk));   // (the masks of the head size made here: kept over the keys they were spilled)
    __builtin_amdgcn_sched_barrier(0);
    float s = 0.f;
#pragma unroll
    for (int t = 0; t < DK; ++t) {
      const int e = 16 * t + 8 * h;
      const u32x4 a = e < Dk ? *reinterpret_cast<const u32x4*>(k + e) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s += widen<F16>(uint16_t(a[i])) * widen<F16>(uint16_t(qv[t][i])) +
             widen<F16>(uint16_t(a[i] >> 16)) * widen<F16>(uint16_t(qv[t][i] >> 16));
      __builtin_amdgcn_sched_barrier(0);   // (one load at a time: registers)
    }
    s = other_sum(s);
    const float far = rounded_product(s, c), mn = j < lim ? fmaxf(m, far) : m;
    const float ms = mn == -INFINITY ? 0.f : mn;
    if (__builtin_amdgcn_ballot_w64(mn != m)) {
      const float alpha = __builtin_amdgcn_exp2f(m - ms);
      l *= alpha;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= alpha;
    }
    m = mn;
    const float e0 = __builtin_amdgcn_exp2f(fabsf(ms) > kFar ? far - ms : __builtin_fmaf(s, c, -ms));
    const float w = widen<F16>(narrow<F16>(e0));
    if (j < lim) {
      l += h == 0 ? e0 : 0.f;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const int e = 32 * d + 2 * i + 4 * h;
          const u32x2 a = e < Dk ? *reinterpret_cast<const u32x2*>(v + e) : u32x2{0u, 0u};
          o[d][i] += w * widen<F16>(uint16_t(a.x));
          o[d][i + 1] += w * widen<F16>(uint16_t(a.x >> 16));
          o[d][i + 2] += w * widen<F16>(uint16_t(a.y));
          o[d][i + 3] += w * widen<F16>(uint16_t(a.y >> 16));
          __builtin_amdgcn_sched_barrier(0);
        }
    }
  });
}

// Whether v holds an infinity or a NaN for the keys first .. last - 1 (`at`: a key's row).
template <bool F16, class F>
__device__ __forceinline__ bool keys_not_finite(int first, int last, int D, F&& at) {
  const int e = 2 * (threadIdx.x & 63);
  float z = 0.f;
  for (int j = first; j < last; ++j) {
    const uint16_t* v = at(j);
    if (v && e < D) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(v + e);
      z += widen<F16>(uint16_t(w)) * 0.f + widen<F16>(uint16_t(w >> 16)) * 0.f;
    }
  }
  return __builtin_amdgcn_ballot_w64(!(z == 0.f)) != 0;
}

// Whether a sum of the wave's rows is an infinity or a NaN.
template <int DT>
__device__ __forceinline__ bool any_not_finite(const f32x16 (&o)[DT]) {
  float z = 0.f;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) z += o[d][i] * 0.f;
  return __builtin_amdgcn_ballot_w64(!(z == 0.f)) != 0;
}

// A wave's rows again whose sums are no numbers, if a value that some row does not see is
// none. The wave's keys: every WAVES-th tile of the share from `wave` on.
template <bool F16, class C, Attend A, int WAVES>
__device__ __forceinline__ void see_again(f32x16 (&o)[C::DP / 32], const u32x4 (&qv)[C::DP / 16], const AttnParams& p, const Share& w,
                                          int origin, float& m, float& l, int lim, int lim0, int wave) {
  int len = __builtin_amdgcn_readfirstlane(w.len);
  asm volatile("" : "+s"(len));
  Pages pages{p, w.b};
  const uint16_t *k = p.k + int64_t(w.kvh) * p.ks[2], *v = p.v + int64_t(w.kvh) * p.vs[2];
  if constexpr (A == Attend::kPaged) pages.look(w.first / p.page_size);
  // key j of the share, nullptr on a page that is none
  auto row = [&](const uint16_t* x, const int64_t (&stride)[3], int j) __attribute__((always_inline)) -> const uint16_t* {
    if constexpr (A == Attend::kPaged) {
      const int page = pages.page_of(w.first + j);
      return page < 0 ? nullptr : x + pages.key_at(w.first + j, page, stride[0], uint32_t(stride[1]) * 2u) / 2;
    } else {
      return x + int64_t(origin + w.first + j) * stride[1];
    }
  };
  if (!keys_not_finite<F16>(max(lim0, 0), len, p.D, [&](int j) __attribute__((always_inline)) { return row(v, p.vs, j); })) return;
  careful_sums<F16, C>(o, qv, p.D, p.c, m, l, lim, [&](auto&& key) __attribute__((always_inline)) {
    for (int t = wave; t * C::KT < len; t += WAVES)
#pragma unroll 1
      for (int j = t * C::KT; j < min(len, (t + 1) * C::KT); ++j) {
        const uint16_t* at = row(k, p.ks, j);
        if (at) key(j, at, row(v, p.vs, j));
      }
  });
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
//
// Paged: a load covers 16 keys, which lie in one page. A wave keeps the table's next 64
// entries in a register, one a lane. Entries outside the cache read nothing, and
// their keys have no weight.
template <bool F16, class C, Attend A>
__global__ __launch_bounds__(C::THREADS, 2) void attention_few_kernel(const AttnParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::LDS];
  constexpr int DK = C::DP / 16, DT = C::DP / 32;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  int rows = p.rows, origin = 0;   // rows of the sequence; packed: its first token
  const Share w = share_of<C, A, C::KT * C::WAVES>(p, rows, origin);
  if (w.idle) return;
  const int b = w.b, kvh = w.kvh, len = w.len, D = p.D;
  const int nt = (len + C::KT - 1) / C::KT;

  // this lane's query row
  const int row = w.tile * C::ROWS + l32;
  const int rowc = min(row, rows - 1);
  const int tok = origin + rowc / p.group, hq = kvh * p.group + rowc % p.group;
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
  const uint16_t *kh = p.k + int64_t(kvh) * p.ks[2], *vh = p.v + int64_t(kvh) * p.vs[2];
  if constexpr (A != Attend::kPaged) {
    kh += int64_t(b) * p.ks[0] + int64_t(origin + w.first) * p.ks[1];
    vh += int64_t(b) * p.vs[0] + int64_t(origin + w.first) * p.vs[1];
  }
  const uint8_t *kb = reinterpret_cast<const uint8_t*>(kh), *vb = reinterpret_cast<const uint8_t*>(vh);
  Pages pages{p, b};
  if constexpr (A == Attend::kPaged) pages.look(w.first / p.page_size);
  const uint8_t* kt = smem + wave * 2 * C::TILE;
  const uint8_t* vt = kt + C::TILE;
  // the 16 rows from `half` on of tile t (an empty range past the last key: the
  // same loads, which read nothing, so that every wait counts alike)
  auto load = [&](const uint8_t* base, int64_t page_stride, uint32_t stride, const uint32_t (&off)[C::SWZ], int t, uint32_t to) __attribute__((always_inline)) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r0 = t * C::KT + 16 * half, rows = min(len - r0, 16);
      uint32_t any = uint32_t(-rows >> 31);   // all ones where rows > 0
      int64_t at = int64_t(r0) * stride;
      if constexpr (A == Attend::kPaged) {
        const int page = rows > 0 ? pages.page_of(w.first + r0) : 0;
        at = pages.key_at(w.first + r0, page, page_stride, stride);
        if (page < 0) any = 0;
      }
      const u32x4 rs = range_desc(base + at, (uint32_t(rows - 1) * stride + uint32_t(D) * 2u) & any);
#pragma unroll
      for (int u = 0; u < C::SWZ; ++u) load_to_lds(rs, off[u], to + (half * C::SWZ + u) * 1024);
    }
  };
  const uint32_t kto = lds_address(kt), vto = lds_address(vt);
  const bool shared_memory = A == Attend::kDense && vst < uint32_t(D) * 2u;   // rows of v that overlap in memory
  // keys of the share that this lane's row sees, and the fewest of the tile's rows
  int lim = len, lim0 = len;
  if constexpr (A == Attend::kPacked)
    if (p.causal) {
      lim = min(len, tok - origin + 1);
      lim0 = min(len, w.tile * C::ROWS / p.group + 1);
    }
  if constexpr (A == Attend::kPaged) {
    const int before = keys_of(p, b) - p.q_len + 1 - w.first;   // (the sum of all keys and new tokens is below 2^31)
    lim = min(len, before + tok);
    lim0 = __builtin_amdgcn_readfirstlane(min(len, before + w.tile * C::ROWS / p.group));
  }

  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;   // maximum in log2 units; this lane's part of the sum

  if (wave < nt) {
    load(kb, p.ks[0], kst, koff, wave, kto);
    load(vb, p.vs[0], vst, voff, wave, vto);
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
    load(kb, p.ks[0], kst, koff, t + C::WAVES, kto);
    if ((t + 1) * C::KT > lim0) {   // the keys end in this tile
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (t * C::KT + 8 * (i >> 2) + 4 * h + (i & 3) >= lim) sc[i] = -INFINITY;
    }
    if constexpr (A == Attend::kPaged) {   // keys of a page that is none
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int key = w.first + t * C::KT + 16 * half;
        if (key - w.first < len && pages.page_of(key) < 0)
#pragma unroll
          for (int i = 8 * half; i < 8 * half + 8; ++i) sc[i] = -INFINITY;
      }
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
    load(vb, p.vs[0], vst, voff, t + C::WAVES, vto);
  }
  wait_vm<0>();
  const AttnParams& pe = A == Attend::kDense ? p : params_again();
  if constexpr (A != Attend::kDense)
    if (lim0 < len && any_not_finite(o)) see_again<F16, C, A, C::WAVES>(o, qv, pe, w, origin, m, l, lim, lim0, wave);
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
    // (the compiler would otherwise read all waves' sums first and add them behind the branch below)
    if constexpr (A == Attend::kPacked)
#pragma unroll
      for (int d = 0; d < DT; ++d) asm volatile("" : "+v"(o[d]));
  }
  if (row >= rows) return;
  store_row<F16, C>(pe, o, mm, l, w, l32, tok, hq, h);
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
// 246 to 282 us from card to card, 873 to 1003 TFLOP/s of the 1228 to 1386 that a large
// product reaches; the matrix cores, the exponentials and the LDS reads share the
// issue slots. 4096 x 512 keys: 34 to 40 us, 644 to 750 TFLOP/s, with 768 tiles for
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

//
// Packed sequences with the mask: a row sees the keys up to its own; a tile's steps end
// with its last row's, and only the steps past its first row's are masked.
//
// Paged: likewise; a wave's load of 4 or 8 keys lies in 16 of one page. A sequence with an
// entry outside the cache masks every step.
template <bool F16, class C, Attend A>
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
  int rows = p.rows, origin = 0;   // rows of the sequence; packed: its first token
  Share w = share_of<C, A, C::KT>(p, rows, origin);
  if (w.idle) return;
  const int b = w.b, kvh = w.kvh, D = p.D;
  int before = 0;   // paged: keys of the share that the sequence's first new token sees (with those up to it)
  if constexpr (A == Attend::kPaged) {
    before = __builtin_amdgcn_readfirstlane(keys_of(p, b)) - p.q_len + 1 - w.first;   // (all keys and new tokens are fewer than 2^31)
    w.len = max(0, min(w.len, before + (min(rows, (w.tile + 1) * C::ROWS) - 1) / p.group));
  }
  const int len = w.len;
  const int n = (len + C::KT - 1) / C::KT;

  const int row = w.tile * C::ROWS + wave * 32 + l32;
  const int rowc = min(row, rows - 1);
  const int tok = origin + rowc / p.group, hq = kvh * p.group + rowc % p.group;
  // keys that this lane's row sees, and the fewest of the tile's rows
  int lim = len, lim0 = len;
  if constexpr (A == Attend::kPacked)
    if (p.causal) {
      lim = tok - origin + 1;
      lim0 = w.tile * C::ROWS / p.group + 1;
    }
  Pages pages{p, b};
  bool holes = false;   // paged: an entry of the share's keys is no page
  if constexpr (A == Attend::kPaged) {
    lim = min(len, before + tok);
    lim0 = max(0, min(len, before + w.tile * C::ROWS / p.group));
    const int first = w.first / p.page_size;
    for (int i = first; int64_t(i) * p.page_size < int64_t(w.first) + len; i += 64) {
      pages.look(i);
      holes |= __builtin_amdgcn_ballot_w64(int64_t(i + lane) * p.page_size < int64_t(w.first) + len &&
                                           (pages.entries < 0 || pages.entries >= p.pages)) != 0;
    }
    if (pages.page0 != first) pages.look(first);
    if (holes) lim0 = 0;
  }
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
  const int in = A == Attend::kPaged ? dr & 15 : dr;   // row of what the load's range holds
  const uint32_t koff = klive ? uint32_t(in) * kst + uint32_t(kc) * 16u : 0xFFFFFFF0u, kstep = klive ? C::RPR * kst : 0u;
  const uint32_t voff = vlive ? uint32_t(in) * vst + uint32_t(vc) * 16u : 0xFFFFFFF0u, vstep = vlive ? C::RPR * vst : 0u;
  const uint16_t *kh = p.k + int64_t(kvh) * p.ks[2], *vh = p.v + int64_t(kvh) * p.vs[2];
  if constexpr (A != Attend::kPaged) {
    kh += int64_t(b) * p.ks[0] + int64_t(origin + w.first) * p.ks[1];
    vh += int64_t(b) * p.vs[0] + int64_t(origin + w.first) * p.vs[1];
  }
  const uint8_t *kb = reinterpret_cast<const uint8_t*>(kh), *vb = reinterpret_cast<const uint8_t*>(vh);
  const uint32_t lds0 = lds_address(smem) + wave * 1024;
  // Tile t of K (to ring place t % RING) or V; tiles past the last key are
  // empty ranges: zeros (by a mask and no branch, so that a step stays one block).
  auto load = [&](const uint8_t* base, int64_t page_stride, uint32_t stride, uint32_t off, uint32_t step, int t, uint32_t to) __attribute__((always_inline)) {
    if constexpr (A == Attend::kPaged) {
#pragma unroll
      for (int u = 0; u < C::ROUNDS; ++u) {
        const int r0 = t * C::KT + (C::RPR == 16 ? 16 * u : 16 * (wave >> 1)), rows = min(len - r0, 16);
        const int page = pages.held(w.first + r0);
        const uint32_t any = uint32_t(~(page >> 31)) & uint32_t(-rows >> 31);
        const u32x4 rs = range_desc(base + pages.key_at(w.first + r0, max(page, 0), page_stride, stride),
                                    (uint32_t(rows - 1) * stride + uint32_t(D) * 2u) & any);
        load_to_lds(rs, off, uint32_t(__builtin_amdgcn_readfirstlane(lds0 + to + u * C::RPR * C::ROWB)));
      }
      return;
    }
    const int rows = min(len - t * C::KT, C::KT);
    const uint32_t any = uint32_t(-rows >> 31);   // all ones where rows > 0
    const u32x4 rs = range_desc(base + int64_t(t * C::KT) * stride, (uint32_t(rows - 1) * stride + uint32_t(D) * 2u) & any);
#pragma unroll
    for (int u = 0; u < C::ROUNDS; ++u) load_to_lds(rs, off + u * step, lds0 + to + u * C::RPR * C::ROWB);
  };
  // Paged: the ranges that steps j .. j + 3 load, j a multiple of 4, made by a lane each: 16 keys
  // of K by lanes 0 .. 7, of V by 8 .. 15 (by scalar instructions in each step 2048 tokens over 8000
  // keys take 279 us, and with a branch for the table's next entries 360; so 221).
  uint32_t range_low = 0, range_high = 0, range_bytes = 0;
  auto ranges = [&](int j) __attribute__((always_inline)) {
    if (pages.place_of(w.first + (j + 8) * C::KT) >= pages.page0 + 64) pages.look(pages.place_of(w.first + j * C::KT));
    const bool val = lane & 8;
    const int r0 = (j + (val ? 2 : 4)) * C::KT + 16 * (lane & 7), key = w.first + r0, i = pages.place_of(key), rows = min(len - r0, 16);
    const int e = __builtin_amdgcn_ds_bpermute((i - pages.page0) * 4, pages.entries);
    const bool any = rows > 0 && e >= 0 && e < p.pages;
    const uint32_t stride = val ? vst : kst;
    const uint64_t at = reinterpret_cast<uint64_t>(val ? vb : kb) + pages.key_at(key, any ? e : 0, val ? p.vs[0] : p.ks[0], stride);
    range_low = uint32_t(at);
    range_high = uint32_t(at >> 32) & 0xFFFFu;
    range_bytes = any ? uint32_t(rows - 1) * stride + uint32_t(D) * 2u : 0u;
  };
  auto load_range = [&](int from, uint32_t off, uint32_t to) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < C::ROUNDS; ++u) {
      const int at = from + (C::RPR == 16 ? u : wave >> 1);
      u32x4 rs{uint32_t(__builtin_amdgcn_readlane(range_low, at)), uint32_t(__builtin_amdgcn_readlane(range_high, at)),
               uint32_t(__builtin_amdgcn_readlane(range_bytes, at)), 0x00020000u};
      settle_desc(rs);
      load_to_lds(rs, off, uint32_t(__builtin_amdgcn_readfirstlane(lds0 + to + u * C::RPR * C::ROWB)));
    }
  };
  auto load_k = [&](int t, int ring) __attribute__((always_inline)) { load(kb, p.ks[0], kst, koff, kstep, t, ring * C::TILE); };
  auto load_v = [&](int t, int ring) __attribute__((always_inline)) { load(vb, p.vs[0], vst, voff, vstep, t, VOFF + ring * C::TILE); };

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
          if (key0 + 8 * (i >> 2) + 4 * h + (i & 3) >= lim) s[i] = -INFINITY;
        if constexpr (A == Attend::kPaged)
          if (holes && pages.held(w.first + key0 + 8 * (part & 2)) < 0)
#pragma unroll
            for (int i = 4 * part; i < 4 * part + 4; ++i) s[i] = -INFINITY;
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
    if constexpr (A == Attend::kPaged && R == 0) ranges(j);
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
      if constexpr (A == Attend::kPaged) {
        if constexpr (I == MFMAS / 2) load_range(2 * R, koff, R * C::TILE);
        if constexpr (I == MFMAS / 2 + 1) load_range(8 + 2 * R, voff, VOFF + ((R + 2) & 3) * C::TILE);
      } else {
        if constexpr (I == MFMAS / 2) load_k(j + 4, R);
        if constexpr (I == MFMAS / 2 + 1) load_v(j + 2, (R + 2) & 3);
      }
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
    const int full = lim0 / C::KT;
    int j = 0;
    for (; j + 4 <= full; j += 4) {
      step.template operator()<false, 0>(j);
      step.template operator()<false, 1>(j + 1);
      step.template operator()<false, 2>(j + 2);
      step.template operator()<false, 3>(j + 3);
    }
    do {   // at most four steps are left, but for the mask's
      if (j < n) step.template operator()<true, 0>(j);
      if (j + 1 < n) step.template operator()<true, 1>(j + 1);
      if (j + 2 < n) step.template operator()<true, 2>(j + 2);
      if (j + 3 < n) step.template operator()<true, 3>(j + 3);
      j += 4;
    } while (A != Attend::kDense && j < n);
    wait_vm<0>();
    // products of the last 32 keys
    const int last = (n - 1) & 3;
    const bool odd = last & 1;
    const u32x4 w0 = odd ? pv[1][0] : pv[0][0], w1 = odd ? pv[1][1] : pv[0][1];
#pragma unroll
    for (int i = 0; i < DK; ++i)
      o[i % DT] = mfma32<F16>(i < 2 ? va[i] : read_v(last, i), i / DT == 0 ? w0 : w1, o[i % DT]);
  }

  const AttnParams& pe = A == Attend::kDense ? p : params_again();
  if constexpr (A != Attend::kDense)
    if (lim0 < len && any_not_finite(o)) see_again<F16, C, A, 1>(o, qv, pe, w, origin, m, l, lim, lim0, 0);
  if (row >= rows) return;
  l = other_sum(l);
  store_row<F16, C>(pe, o, m, l, w, wave * 32 + l32, tok, hq, h);
}

// Joins the parts of the cut tiles' rows, in order: one thread per 4 values,
// blockIdx.y the cut tile.
template <bool F16, Attend A>
__global__ __launch_bounds__(256) void attention_join_kernel(const AttnParams p, int tile_rows) {
  const int per = p.D / 4, nth = blockIdx.y, id = p.whole + nth;
  int pair = id % p.pairs, tile = id / p.pairs, parts = p.parts;
  if constexpr (A == Attend::kPaged) tile = p.per_seq / p.kv_heads - 1 - tile;
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

}  // namespace w4a4
