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
#include "w4a4_attention.hpp"
#include "w4a4_host.hpp"
#include "w4a4_strided.hpp"

namespace w4a4 {

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
    return D <= 64 ? reinterpret_cast<const void*>(attention_few_kernel<F16, FewAttn<64>, Attend::kDense>)
         : D <= 96 ? reinterpret_cast<const void*>(attention_few_kernel<F16, FewAttn<96>, Attend::kDense>)
                   : reinterpret_cast<const void*>(attention_few_kernel<F16, FewAttn<128>, Attend::kDense>);
  return D <= 64 ? reinterpret_cast<const void*>(attention_wide_kernel<F16, WideAttn<64>, Attend::kDense>)
       : D <= 96 ? reinterpret_cast<const void*>(attention_wide_kernel<F16, WideAttn<96>, Attend::kDense>)
                 : reinterpret_cast<const void*>(attention_wide_kernel<F16, WideAttn<128>, Attend::kDense>);
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
    e = hipLaunchKernel(a->f16 ? reinterpret_cast<const void*>(attention_join_kernel<true, Attend::kDense>)
                               : reinterpret_cast<const void*>(attention_join_kernel<false, Attend::kDense>),
                        dim3(unsigned((rows * (D / 4) + 255) / 256), unsigned(pl.cut)), dim3(256), args, 0, st);
  }
  return e == hipSuccess ? GEMM_W4A4_OK : GEMM_W4A4_ELAUNCH;
}

}  // namespace w4a4

extern "C" int cross_attention(const cross_attention_t* args, void* stream) { return w4a4::attention_run(args, stream); }

extern "C" int64_t cross_attention_workspace(const cross_attention_t* args) {
  return w4a4::attn_sizes_ok(args) ? w4a4::attn_plan(args).bytes : GEMM_W4A4_EINVAL;
}
