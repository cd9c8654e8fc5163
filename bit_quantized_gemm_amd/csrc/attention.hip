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
// K and V go to LDS by direct-to-LDS buffer loads, two stages of KT keys. The
// descriptors end with the sequence's last key, so keys past kv_lens and the
// padding of head sizes to DP read as zeros, whatever memory holds there.
// 16-byte chunks are XOR-swizzled by row (K: chunk ^ row, for reads of 32 rows
// at one chunk; V: chunk ^ 2 row, for transposed reads of 8 rows at two).
//
// Rows of a (sequence, key head) are (token, query head of the group) pairs, so
// heads that share keys share a tile. Few rows: the waves of a workgroup take
// different keys for the same 32 rows and join in LDS, and the keys are split
// over workgroups whose parts a second launch joins, in order.
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

namespace w4a4 {

struct AttnParams {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  float* lse;
  const int32_t* kv_lens;
  float* part_o;       // splits > 1: [split][pair][row][D] sums, then
  float* part_ms;      //             [split][pair][row][2] maximum (log2 units) and sum
  int64_t qs[3], ks[3], vs[3], os[3];   // batch, token, head
  int q_len, kv_len, kv_heads, D, group;   // group: query heads of a key head
  int rows;            // q_len * group
  int tiles;           // row tiles of a (sequence, key head) pair
  int pairs;           // batch * kv_heads
  int splits;
  float c;             // scale * log2(e)
};

// WQ waves over query rows (32 each), WK waves over the keys of a stage; DP:
// head size padded to 64, 96 or 128.
template <int DP_, int WQ_, int WK_, int KT_>
struct AttnCfg {
  static constexpr int DP = DP_, WQ = WQ_, WK = WK_, KT = KT_;
  static constexpr int THREADS = WQ * WK * kWave;
  static constexpr int ROWS = WQ * 32;
  static constexpr int ROWB = DP > 64 ? 256 : 128;         // bytes of a key's row in LDS
  static constexpr int CH = ROWB / 16;                     // 16-byte chunks of a row
  static constexpr int TILE = KT * ROWB;                   // K or V of a stage
  static constexpr int RPR = THREADS * 16 / ROWB;          // rows a round of loads covers
  static constexpr int ROUNDS = KT / RPR;
  static constexpr int NKT = KT / (32 * WK);               // 32-key tiles of a wave's share
  static constexpr int LDS = 4 * TILE;
  static constexpr int MERGE = WK > 1 ? WK * 32 * (DP + 4) * 4 : 0;   // join of the waves' parts
  static_assert(KT % RPR == 0 && ROUNDS >= 1 && NKT >= 1, "whole rounds and key tiles");
  static_assert(MERGE <= LDS && LDS <= kLdsLimit, "LDS budget");
};

// Position of chunk c of row r.
template <class C>
__device__ __forceinline__ int k_chunk(int r, int c) { return c ^ (C::CH == 16 ? r & 15 : (r >> 1) & 7); }
template <class C>
__device__ __forceinline__ int v_chunk(int r, int c) { return c ^ (C::CH == 16 ? (r & 7) << 1 : ((r >> 1) & 3) << 1); }

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Transposed read: the lanes of a group of 16 pass the addresses of 4 rows x 4
// runs of 4 values; lane i gets column i of the 4 rows.
__device__ __forceinline__ u32x2 read_transposed(const uint8_t* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (__attribute__((address_space(3))) s16x4*)p));
}

// max(v, v of lane ^ 32); likewise the sum
__device__ __forceinline__ float other_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return fmaxf(__builtin_bit_cast(float, uint32_t(r[0])), __builtin_bit_cast(float, uint32_t(r[1])));
}
__device__ __forceinline__ float other_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, v), __builtin_bit_cast(uint32_t, v), false, false);
  return __builtin_bit_cast(float, uint32_t(r[0])) + __builtin_bit_cast(float, uint32_t(r[1]));
}

template <bool F16, class C, bool SPLIT>
__global__ __launch_bounds__(C::THREADS) void attention_kernel(const AttnParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::LDS];
  constexpr int DK = C::DP / 16, DT = C::DP / 32;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wq = wave % C::WQ, wk = wave / C::WQ;
  const int l32 = lane & 31, h = lane >> 5;

  const int pair = blockIdx.x % p.pairs;
  const int tile = blockIdx.x / p.pairs % p.tiles;
  const int split = SPLIT ? blockIdx.x / p.pairs / p.tiles : 0;
  const int b = pair / p.kv_heads, kvh = pair - b * p.kv_heads;
  const int D = p.D;
  int len = p.kv_len;
  if (p.kv_lens) len = min(max(p.kv_lens[b], 0), p.kv_len);
  len = __builtin_amdgcn_readfirstlane(len);
  const int nt = (len + C::KT - 1) / C::KT;
  const int t0 = SPLIT ? int(int64_t(nt) * split / p.splits) : 0;
  const int t1 = SPLIT ? int(int64_t(nt) * (split + 1) / p.splits) : nt;

  // this lane's query row
  const int row = tile * C::ROWS + wq * 32 + l32;
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

  // stage loads: round u covers rows u RPR .. of the stage; lane -> (row,
  // chunk position); chunks past D are out of every range
  const int dr = tid / C::CH, dp = tid % C::CH;
  const int kc = k_chunk<C>(dr, dp), vc = v_chunk<C>(dr, dp);
  static_assert(C::RPR % 16 == 0, "the swizzles repeat every 16 rows");
  const uint32_t kst = uint32_t(p.ks[1]) * 2u, vst = uint32_t(p.vs[1]) * 2u;   // token strides in bytes
  const bool klive = kc * 8 < D, vlive = vc * 8 < D;
  const uint32_t koff = klive ? uint32_t(dr) * kst + uint32_t(kc) * 16u : 0xFFFFFFF0u, kstep = klive ? C::RPR * kst : 0u;
  const uint32_t voff = vlive ? uint32_t(dr) * vst + uint32_t(vc) * 16u : 0xFFFFFFF0u, vstep = vlive ? C::RPR * vst : 0u;
  const uint8_t* kb = reinterpret_cast<const uint8_t*>(p.k + int64_t(b) * p.ks[0] + int64_t(kvh) * p.ks[2]);
  const uint8_t* vb = reinterpret_cast<const uint8_t*>(p.v + int64_t(b) * p.vs[0] + int64_t(kvh) * p.vs[2]);
  auto load_stage = [&](int t) __attribute__((always_inline)) {
    uint8_t* dst = smem + (t & 1) * 2 * C::TILE + wave * 1024;
    // (rows - 1) strides and one row: below 2^31, strides are below 2^24 bytes
    const int rows = min(len - t * C::KT, C::KT);
    const __amdgpu_buffer_rsrc_t kr = row_rsrc(kb + int64_t(t * C::KT) * kst, uint32_t(rows - 1) * kst + uint32_t(D) * 2u);
    const __amdgpu_buffer_rsrc_t vr = row_rsrc(vb + int64_t(t * C::KT) * vst, uint32_t(rows - 1) * vst + uint32_t(D) * 2u);
#pragma unroll
    for (int u = 0; u < C::ROUNDS; ++u) {
      dma_rows(kr, koff + u * kstep, dst + u * C::RPR * C::ROWB);
      dma_rows(vr, voff + u * vstep, dst + u * C::RPR * C::ROWB + C::TILE);
    }
  };

  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;   // maximum in log2 units; this lane's part of the sum

  // addresses of this lane's reads inside a stage
  const int krow = wk * 32 * C::NKT + l32;
  const int vr = (lane & 15) >> 2;                       // row of the four
  const int vcol = 4 * ((lane >> 4) & 1) + (lane & 3);   // run of 4 values among the 32 of a d tile

  if (t0 < t1) load_stage(t0);
  for (int t = t0; t < t1; ++t) {
    wait_vm_lgkm0<0>();
    __syncthreads();
    if (t + 1 < t1) load_stage(t + 1);
    const uint8_t* st = smem + (t & 1) * 2 * C::TILE;

    f32x16 sc[C::NKT];
#pragma unroll
    for (int j = 0; j < C::NKT; ++j) {
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[j][i] = 0.f;
#pragma unroll
      for (int s = 0; s < DK; ++s) {
        const int r = krow + 32 * j;
        const u32x4 a = *reinterpret_cast<const u32x4*>(st + r * C::ROWB + k_chunk<C>(r, 2 * s + h) * 16);
        sc[j] = mfma32<F16>(a, qv[s], sc[j]);
      }
    }
    if ((t + 1) * C::KT > len) {   // the sequence ends in this stage
#pragma unroll
      for (int j = 0; j < C::NKT; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = t * C::KT + wk * 32 * C::NKT + 32 * j + 8 * (i >> 2) + 4 * h + (i & 3);
          if (key >= len) sc[j][i] = -INFINITY;
        }
    }
    float top = sc[0][0];
#pragma unroll
    for (int j = 0; j < C::NKT; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, sc[j][i]);
    top = other_max(top) * p.c;
    const float mn = fmaxf(m, top);
    const float ms = mn == -INFINITY ? 0.f : mn;   // no key yet, or none with weight
    const float alpha = __builtin_amdgcn_exp2f(m - ms);
    m = mn;
    l *= alpha;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] *= alpha;
    u32x4 pv[2 * C::NKT];
#pragma unroll
    for (int j = 0; j < C::NKT; ++j)
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[j][i], p.c, -ms));
        const float e1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[j][i + 1], p.c, -ms));
        l += e0 + e1;
        pv[2 * j + (i >> 3)][(i >> 1) & 3] = narrow2<F16>(e0, e1);
      }
#pragma unroll
    for (int j = 0; j < 2 * C::NKT; ++j)
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const int r0 = wk * 32 * C::NKT + 16 * j + 4 * h + vr;
        const int col = 8 * d + vcol;   // run of 4 values in the row
        const u32x2 lo = read_transposed(st + C::TILE + r0 * C::ROWB + v_chunk<C>(r0, col >> 1) * 16 + (col & 1) * 8);
        const u32x2 hi = read_transposed(st + C::TILE + (r0 + 8) * C::ROWB + v_chunk<C>(r0 + 8, col >> 1) * 16 + (col & 1) * 8);
        o[d] = mfma32<F16>(u32x4{lo.x, lo.y, hi.x, hi.y}, pv[j], o[d]);
      }
  }
  l = other_sum(l);

  if constexpr (C::WK > 1) {
    // join the waves' keys: each writes its sums, maximum and sum; wave 0 adds
    // them in order
    static_assert(C::WQ == 1, "waves over keys share one row tile");
    float* mg = reinterpret_cast<float*>(smem);
    constexpr int S = C::DP + 4;
    __syncthreads();
    float* mine = mg + (wk * 32 + l32) * S;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<f32x4*>(mine + 32 * d + 2 * i + 4 * h) = f32x4{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
    if (h == 0) {
      mine[C::DP] = m;
      mine[C::DP + 1] = l;
    }
    __syncthreads();
    if (wk != 0) return;
    float mm = m;
#pragma unroll
    for (int w = 1; w < C::WK; ++w) mm = fmaxf(mm, mg[(w * 32 + l32) * S + C::DP]);
    const float ms = mm == -INFINITY ? 0.f : mm;
    const float f0 = __builtin_amdgcn_exp2f(m - ms);
    l *= f0;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] *= f0;
#pragma unroll
    for (int w = 1; w < C::WK; ++w) {
      const float* other = mg + (w * 32 + l32) * S;
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
    m = mm;
  }

  if (row >= p.rows) return;
  if constexpr (SPLIT) {
    const int64_t at = (int64_t(split) * p.pairs + pair) * p.rows + row;
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
  } else {
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;   // a NaN sum stays one
    uint16_t* out = p.out + int64_t(b) * p.os[0] + int64_t(tok) * p.os[1] + int64_t(hq) * p.os[2];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const int e = 32 * d + 2 * i + 4 * h;
        if (e < D)
          *reinterpret_cast<u32x2*>(out + e) = u32x2{narrow2<F16>(o[d][i] * inv, o[d][i + 1] * inv),
                                                     narrow2<F16>(o[d][i + 2] * inv, o[d][i + 3] * inv)};
      }
    if (p.lse && h == 0)
      p.lse[(int64_t(b) * p.kv_heads * p.group + hq) * p.q_len + tok] = l == 0.f ? -INFINITY : (m + __builtin_log2f(l)) * 0.6931471805599453f;
  }
}

// Joins the splits' parts of a row, in split order: one thread per 4 values.
template <bool F16>
__global__ __launch_bounds__(256) void attention_join_kernel(const AttnParams p) {
  const int per = p.D / 4;
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t all = int64_t(p.pairs) * p.rows;
  const int64_t at = i / per;
  if (at >= all) return;
  const int e = int(i - at * per) * 4;
  float mm = -INFINITY;
  for (int s = 0; s < p.splits; ++s) mm = fmaxf(mm, p.part_ms[(s * all + at) * 2]);
  const float ms = mm == -INFINITY ? 0.f : mm;
  float l = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < p.splits; ++s) {
    const float f = __builtin_amdgcn_exp2f(p.part_ms[(s * all + at) * 2] - ms);
    l += p.part_ms[(s * all + at) * 2 + 1] * f;
    o += *reinterpret_cast<const f32x4*>(p.part_o + (s * all + at) * p.D + e) * f;
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  const int pair = int(at / p.rows), row = int(at - int64_t(pair) * p.rows);
  const int b = pair / p.kv_heads, tok = row / p.group, hq = (pair - b * p.kv_heads) * p.group + row % p.group;
  uint16_t* out = p.out + int64_t(b) * p.os[0] + int64_t(tok) * p.os[1] + int64_t(hq) * p.os[2];
  *reinterpret_cast<u32x2*>(out + e) = u32x2{narrow2<F16>(o.x * inv, o.y * inv), narrow2<F16>(o.z * inv, o.w * inv)};
  if (p.lse && e == 0)
    p.lse[(int64_t(b) * p.kv_heads * p.group + hq) * p.q_len + tok] = l == 0.f ? -INFINITY : (mm + __builtin_log2f(l)) * 0.6931471805599453f;
}

// ------------------------------------------------------------------ host side

struct AttnPlan {
  int shape;     // 0: many rows (4 waves of 32 rows); 1: few (4 waves over the keys)
  int rows, tiles, pairs, splits, rows_all;
  int64_t o_bytes, bytes;
};

static bool attn_sizes_ok(const cross_attention_t* a) {
  if (!a || a->batch < 0 || a->q_len < 0 || a->kv_len < 0 || a->q_heads < 0 || a->kv_heads < 1) return false;
  if (a->q_heads % a->kv_heads != 0) return false;
  if (a->head_dim < 8 || a->head_dim > CROSS_ATTENTION_MAX_HEAD_DIM || a->head_dim % 8 != 0) return false;
  const int64_t lim = int64_t(1) << 31;
  return int64_t(a->q_len) * a->q_heads < lim && int64_t(a->batch) * a->kv_heads < lim / 256 &&
         int64_t(a->batch) * a->q_len * a->q_heads < lim;
}

static AttnPlan attn_plan(const cross_attention_t* a) {
  AttnPlan pl{};
  const int group = a->q_heads / a->kv_heads;
  pl.rows_all = a->q_len * group;
  pl.pairs = a->batch * a->kv_heads;
  pl.shape = pl.rows_all <= 32 ? 1 : 0;
  pl.rows = pl.shape == 1 ? 32 : 128;
  pl.tiles = (pl.rows_all + pl.rows - 1) / pl.rows;
  const int kt = pl.shape == 1 ? 128 : 64;
  const int64_t wgs = int64_t(pl.tiles) * pl.pairs;
  const int nt = (a->kv_len + kt - 1) / kt;
  int64_t s = wgs > 0 ? std::min<int64_t>(2 * kNumCUs / wgs, nt / 2) : 1;
  pl.splits = int(std::max<int64_t>(1, std::min<int64_t>(s, 64)));
  if (pl.splits > 1) {
    const int64_t n = int64_t(pl.splits) * pl.pairs * pl.rows_all;
    pl.o_bytes = n * a->head_dim * 4;
    pl.bytes = pl.o_bytes + n * 8;
  }
  return pl;
}

template <bool F16, bool SPLIT>
static const void* attention_of(int shape, int D) {
  if (shape == 1)
    return D <= 64 ? reinterpret_cast<const void*>(attention_kernel<F16, AttnCfg<64, 1, 4, 128>, SPLIT>)
         : D <= 96 ? reinterpret_cast<const void*>(attention_kernel<F16, AttnCfg<96, 1, 4, 128>, SPLIT>)
                   : reinterpret_cast<const void*>(attention_kernel<F16, AttnCfg<128, 1, 4, 128>, SPLIT>);
  return D <= 64 ? reinterpret_cast<const void*>(attention_kernel<F16, AttnCfg<64, 4, 1, 64>, SPLIT>)
       : D <= 96 ? reinterpret_cast<const void*>(attention_kernel<F16, AttnCfg<96, 4, 1, 64>, SPLIT>)
                 : reinterpret_cast<const void*>(attention_kernel<F16, AttnCfg<128, 4, 1, 64>, SPLIT>);
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
  if (a->kv_len <= 1) p.ks[1] = p.vs[1] = 0;   // the stride of a single key is not used
  p.q_len = a->q_len;
  p.kv_len = a->kv_len;
  p.kv_heads = a->kv_heads;
  p.D = D;
  p.group = a->q_heads / a->kv_heads;
  p.rows = pl.rows_all;
  p.tiles = pl.tiles;
  p.pairs = pl.pairs;
  p.splits = pl.splits;
  p.c = a->scale * 1.4426950408889634f;
  void* args[] = {&p};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const bool split = pl.splits > 1;
  const void* k = a->f16 ? (split ? attention_of<true, true>(pl.shape, D) : attention_of<true, false>(pl.shape, D))
                         : (split ? attention_of<false, true>(pl.shape, D) : attention_of<false, false>(pl.shape, D));
  const int64_t grid = int64_t(pl.pairs) * pl.tiles * pl.splits;
  if (grid >= (int64_t(1) << 31)) return GEMM_W4A4_EINVAL;
  hipError_t e = hipLaunchKernel(k, dim3(unsigned(grid)), dim3(256), args, 0, st);
  if (e == hipSuccess && split) {
    const int64_t n = int64_t(pl.pairs) * pl.rows_all * (D / 4);
    e = hipLaunchKernel(a->f16 ? reinterpret_cast<const void*>(attention_join_kernel<true>)
                               : reinterpret_cast<const void*>(attention_join_kernel<false>),
                        dim3(unsigned((n + 255) / 256)), dim3(256), args, 0, st);
  }
  return e == hipSuccess ? GEMM_W4A4_OK : GEMM_W4A4_ELAUNCH;
}

}  // namespace w4a4

extern "C" int cross_attention(const cross_attention_t* args, void* stream) { return w4a4::attention_run(args, stream); }

extern "C" int64_t cross_attention_workspace(const cross_attention_t* args) {
  return w4a4::attn_sizes_ok(args) ? w4a4::attn_plan(args).bytes : GEMM_W4A4_EINVAL;
}
