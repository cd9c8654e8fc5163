// packed_attention.hip — attention within sequences of different lengths packed one
// after the other, causal or not (packed_attention in gemm_w4a4.h): the many-row kernel of
// w4a4_attention.hpp on 128-row tiles that end with their sequence.
//
// With the mask a tile's keys end with its last row's, so its work grows with its place in
// the sequence. Workgroups therefore take the tiles of all sequences by that place, the
// last ones first (packed_tile), and the key heads of a tile beside each other.
#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_w4a4.h"
#include "w4a4_attention.hpp"
#include "w4a4_host.hpp"
#include "w4a4_strided.hpp"

namespace w4a4 {

template <bool F16>
static const void* packed_of(bool few, int D) {
  if (few)
    return D <= 64 ? reinterpret_cast<const void*>(attention_few_kernel<F16, FewAttn<64>, Attend::kPacked>)
         : D <= 96 ? reinterpret_cast<const void*>(attention_few_kernel<F16, FewAttn<96>, Attend::kPacked>)
                   : reinterpret_cast<const void*>(attention_few_kernel<F16, FewAttn<128>, Attend::kPacked>);
  return D <= 64 ? reinterpret_cast<const void*>(attention_wide_kernel<F16, WideAttn<64>, Attend::kPacked>)
       : D <= 96 ? reinterpret_cast<const void*>(attention_wide_kernel<F16, WideAttn<96>, Attend::kPacked>)
                 : reinterpret_cast<const void*>(attention_wide_kernel<F16, WideAttn<128>, Attend::kPacked>);
}

static int packed_run(const packed_attention_t* a, void* stream) {
  if (!a || a->tokens < 0 || a->seqs < 0 || a->seqs > PACKED_ATTENTION_MAX_SEQS || a->q_heads < 0 || a->kv_heads < 1) return GEMM_W4A4_EINVAL;
  if (a->q_heads % a->kv_heads != 0 || (a->f16 | 1) != 1 || (a->causal | 1) != 1) return GEMM_W4A4_EINVAL;
  const int D = a->head_dim;
  if (D < 8 || D > CROSS_ATTENTION_MAX_HEAD_DIM || D % 8 != 0) return GEMM_W4A4_EINVAL;
  if (!(a->scale > 0.f && a->scale <= 1e30f)) return GEMM_W4A4_EINVAL;
  const int64_t lim = int64_t(1) << 31;
  if (int64_t(a->tokens) * a->q_heads > lim - CROSS_ATTENTION_PAST_END || a->kv_heads >= 1 << 20) return GEMM_W4A4_EINVAL;
  const int qsz[3] = {a->tokens, a->q_heads, 1}, ksz[3] = {a->tokens, a->kv_heads, 1};
  const auto three = [](const int64_t (&s)[2], int64_t (&to)[3]) { to[0] = s[0], to[1] = s[1], to[2] = 0; };
  int64_t qs[3], ks[3], vs[3], os[3];
  three(a->q_stride, qs);
  three(a->k_stride, ks);
  three(a->v_stride, vs);
  three(a->out_stride, os);
  const int64_t qe = strided_extent(qsz, qs, D), ke = strided_extent(ksz, ks, D), ve = strided_extent(ksz, vs, D), oe = strided_extent(qsz, os, D);
  if (qe < 0 || ke < 0 || ve < 0 || oe < 0 || !strides_apart(qsz, os, D)) return GEMM_W4A4_EINVAL;
  for (int i = 0; i < 2; ++i) {
    if (qsz[i] > 1 && ((qs[i] | os[i]) & 7)) return GEMM_W4A4_EINVAL;
    if (ksz[i] > 1 && ((ks[i] | vs[i]) & 7)) return GEMM_W4A4_EINVAL;
  }
  // (v: rows that overlap in memory would bring in what lies behind a tile's last key)
  if (a->tokens > 1 && (ks[0] >= (int64_t(1) << 23) || vs[0] >= (int64_t(1) << 23) || vs[0] < D)) return GEMM_W4A4_EINVAL;
  if (a->tokens == 0 || a->seqs == 0 || a->q_heads == 0) return GEMM_W4A4_OK;
  if (!a->q || !a->k || !a->v || !a->out || !a->starts) return GEMM_W4A4_EINVAL;
  if ((uintptr_t(a->q) | uintptr_t(a->k) | uintptr_t(a->v) | uintptr_t(a->out)) & 15u) return GEMM_W4A4_EALIGN;
  if ((uintptr_t(a->lse) | uintptr_t(a->starts)) & 3u) return GEMM_W4A4_EALIGN;
  const struct { const void* p; size_t n; } outs[] = {{a->out, size_t(oe) * 2}, {a->lse, size_t(a->q_heads) * a->tokens * 4}},
      ins[] = {{a->q, size_t(qe) * 2}, {a->k, size_t(ke) * 2}, {a->v, size_t(ve) * 2}, {a->starts, (size_t(a->seqs) + 1) * 4}};
  for (const auto& o : outs)
    for (const auto& i : ins)
      if (overlaps(o.p, o.n, i.p, i.n)) return GEMM_W4A4_EOVERLAP;
  if (overlaps(outs[0].p, outs[0].n, outs[1].p, outs[1].n)) return GEMM_W4A4_EOVERLAP;
  const int group = a->q_heads / a->kv_heads;
  // Few tiles leave compute units idle and wait out their keys one step after the other: there
  // 32-row tiles, whose waves share the keys. By the 128-row tiles to expect, a sequence's last
  // one counted half (both measured, us, 128-row tiles against 32-row ones; 24 heads on 8 of 128
  // where no others are named). Fewer than 180: one prompt of 512 14.8 and 11.7, of 2048 with 8 heads of 64 32.1 and
  // 17.5, 4096 with 4 heads 69.1 and 40.9, 532 + 250 + 117 + 102 with 16 of 72 13.0 and 12.3. More:
  // one of 1024 22.8 and 24.4, eight of 256 15.1 and 26.5, 32 of 64 10.9 and 23.2. (One long prompt of few
  // heads gains from 32-row tiles past it too: 8192 with 8 heads of 64 130 and 110.)
  constexpr int kWide = WideAttn<128>::ROWS, kFew = FewAttn<128>::ROWS, kFewTiles = 180;
  static_assert(WideAttn<64>::ROWS == kWide && WideAttn<96>::ROWS == kWide && FewAttn<64>::ROWS == kFew && FewAttn<96>::ROWS == kFew, "one tile height");
  const bool few = int64_t(a->tokens) * a->q_heads + int64_t(std::min(a->seqs, a->tokens)) * a->kv_heads * (kWide / 2) < int64_t(kFewTiles) * kWide;
  // the most tiles that sequences of these tokens can have; workgroups past the last leave
  const int64_t tiles = int64_t(a->tokens) * group / (few ? kFew : kWide) + std::min(a->seqs, a->tokens);
  if (tiles * a->kv_heads >= int64_t(1) << 24) return GEMM_W4A4_EINVAL;   // (a launch holds fewer than 2^32 threads)
  const int dev_rc = check_device();
  if (dev_rc != GEMM_W4A4_OK) return dev_rc;

  AttnParams p{};
  p.q = static_cast<const uint16_t*>(a->q);
  p.k = static_cast<const uint16_t*>(a->k);
  p.v = static_cast<const uint16_t*>(a->v);
  p.out = static_cast<uint16_t*>(a->out);
  p.lse = a->lse;
  for (int i = 0; i < 2; ++i) {
    p.qs[i + 1] = qs[i];
    p.ks[i + 1] = ks[i];
    p.vs[i + 1] = vs[i];
    p.os[i + 1] = os[i];
  }
  if (a->tokens == 1) p.ks[1] = p.vs[1] = D;   // the stride of a single key is not the caller's to keep
  p.q_len = p.kv_len = a->tokens;
  p.kv_heads = a->kv_heads;
  p.D = D;
  p.group = group;
  p.c = a->scale * 1.4426950408889634f;
  p.starts = a->starts;
  p.seqs = a->seqs;
  p.causal = a->causal;
  void* args[] = {&p};
  const hipError_t e = hipLaunchKernel(a->f16 ? packed_of<true>(few, D) : packed_of<false>(few, D), dim3(unsigned(tiles * a->kv_heads)), dim3(256),
                                       args, 0, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GEMM_W4A4_OK : GEMM_W4A4_ELAUNCH;
}

}  // namespace w4a4

extern "C" int packed_attention(const packed_attention_t* args, void* stream) { return w4a4::packed_run(args, stream); }
