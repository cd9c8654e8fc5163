// paged_attention.hip — attention of each sequence's newest tokens over a paged
// cache (paged_attention in gemm_w4a4.h): the kernels of w4a4_attention.hpp,
// whose loads of 16 keys find their page in the table, and their join.
//
// Few new tokens are bound by reading the cache, pieces of prompts by the matrix cores (2048 tokens
// of 24 heads over 8000 keys: 204 to 221 us from card to card, 794 to 861 TFLOP/s of the unmasked scores). The keys of tiles that fill no round of the compute units
// are cut into parts, since sequences' lengths are known only to the device; a
// second launch joins them in order.
#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_w4a4.h"
#include "w4a4_attention.hpp"
#include "w4a4_host.hpp"
#include "w4a4_strided.hpp"

namespace w4a4 {

struct PagedPlan {
  bool few;     // 32-row tiles, waves over the keys
  int rows;     // rows of a tile
  int tiles, rows_all;
  int64_t whole;
  int cut, parts;
  bool even;
  int64_t o_bytes, bytes;
};

static bool paged_sizes_ok(const paged_attention_t* a) {
  if (!a || a->batch < 0 || a->q_len < 0 || a->q_heads < 0 || a->kv_heads < 1 || a->q_heads % a->kv_heads != 0) return false;
  if (a->head_dim < 8 || a->head_dim > CROSS_ATTENTION_MAX_HEAD_DIM || a->head_dim % 8 != 0) return false;
  if (a->pages < 0 || a->table_width < 0 || a->page_size < PAGED_ATTENTION_PAGE_MULTIPLE || a->page_size % PAGED_ATTENTION_PAGE_MULTIPLE != 0)
    return false;
  // rows and keys are counted in int, with what is asked for ahead
  const int64_t lim = int64_t(1) << 31, most = lim - CROSS_ATTENTION_PAST_END;
  return int64_t(a->q_len) * a->q_heads <= most && int64_t(a->table_width) * a->page_size <= most / 2 && a->q_len <= most / 2 &&
         int64_t(a->batch) * a->kv_heads < lim / 256 && int64_t(a->batch) * a->q_len * a->q_heads < lim;
}

// Which tiles are cut, as for cross_attention, into parts of at least a step of all waves
// (kMinPart keys; three tokens over 1001 keys: 256 12.9 us, 128 11.3, 64 10.8; eight
// sequences of 1000 16.4, 15.3 and 13.5, of 200 10.3, 11.0 and 11.6). Up to kShort
// keys each sequence's own are cut into as many parts; past that parts have even length over the
// sequences, which takes the device 2 us to work out (one token, us, even parts against own: eight sequences of
// 1000 to 650 15.6 and 14.1, four of 3000 to 100 14.9 and 14.3; one of 300 in a table of 8192, where most of its own
// 64 parts are empty, 13.9 and 16.1).
static PagedPlan paged_plan(const paged_attention_t* a) {
  constexpr int kShort = 4096;
  // 32-row tiles read the keys again for every 32 rows, but split them over their waves (us, 32-row
  // tiles against 128-row ones, 24 heads on 8 where no others are named): 64 rows of 2 sequences of 4000, 8 heads
  // of 64 14.9 and 15.9, 48 rows of 32 of 1000 30.3 and 28.2; 66 rows of 8 of 1000 22.4 and 20.0, 120 of
  // 32 58 and 30, 1536 over 4096 keys 69 and 45, over 512 19.0 and 21.8, 6144 over 8000 476 and 204.
  constexpr int kFewRows = 64;
  PagedPlan pl{};
  pl.rows_all = a->q_len * (a->q_heads / a->kv_heads);
  pl.few = pl.rows_all <= kFewRows;
  pl.rows = pl.few ? FewAttn<128>::ROWS : WideAttn<128>::ROWS;
  const int kMinPart = pl.few ? 128 : 256;
  pl.tiles = (pl.rows_all + pl.rows - 1) / pl.rows;
  pl.whole = int64_t(pl.tiles) * a->batch * a->kv_heads;
  pl.parts = 1;
  const int left = int(pl.whole % kNumCUs);
  // A prompt's own keys: the tiles differ in length by the mask, the short ones fill the last round, and parts
  // of them only cost the join (us, cut and not: 2048 tokens over as many 59 and 51, 1600 47 and 40, 2048 of
  // 24 key heads over 4096 110 and 107; but 2048 over 8000 204 and 210, 1408 162 and 192, 1700 over 6000 139 and 150).
  // By the table's width, since lengths are on the device: in a table of three times its keys a prompt is cut.
  const bool own_keys = !pl.few && pl.whole >= kNumCUs && int64_t(a->table_width) * a->page_size < int64_t(a->q_len) * 3;
  if (left > 0 && !own_keys) {
    const int slots = pl.whole < kNumCUs ? 2 * kNumCUs : kNumCUs;
    const int parts = std::min(slots / left, a->table_width * a->page_size / kMinPart);
    if (parts > 1) {
      pl.parts = parts;
      pl.cut = left;
      pl.whole -= left;
      pl.even = pl.whole == 0 && a->table_width * a->page_size > kShort;
      const int64_t n = int64_t(left) * parts * pl.rows;
      pl.o_bytes = n * a->head_dim * 4;
      pl.bytes = pl.o_bytes + n * 8;
    }
  }
  return pl;
}

template <bool F16>
static const void* paged_of(bool few, int D) {
  if (!few)
    return D <= 64 ? reinterpret_cast<const void*>(attention_wide_kernel<F16, WideAttn<64>, Attend::kPaged>)
         : D <= 96 ? reinterpret_cast<const void*>(attention_wide_kernel<F16, WideAttn<96>, Attend::kPaged>)
                   : reinterpret_cast<const void*>(attention_wide_kernel<F16, WideAttn<128>, Attend::kPaged>);
  return D <= 64 ? reinterpret_cast<const void*>(attention_few_kernel<F16, FewAttn<64>, Attend::kPaged>)
       : D <= 96 ? reinterpret_cast<const void*>(attention_few_kernel<F16, FewAttn<96>, Attend::kPaged>)
                 : reinterpret_cast<const void*>(attention_few_kernel<F16, FewAttn<128>, Attend::kPaged>);
}

static int paged_run(const paged_attention_t* a, void* stream) {
  if (!paged_sizes_ok(a) || (a->f16 | 1) != 1 || !(a->scale > 0.f && a->scale <= 1e30f)) return GEMM_W4A4_EINVAL;
  const int D = a->head_dim;
  const int qsz[3] = {a->batch, a->q_len, a->q_heads}, csz[3] = {a->pages, a->page_size, a->kv_heads}, tsz[3] = {a->batch, 1, 1};
  const int64_t tst[3] = {a->table_stride, 0, 0};
  const int64_t qe = strided_extent(qsz, a->q_stride, D), ke = strided_extent(csz, a->k_stride, D), ve = strided_extent(csz, a->v_stride, D),
                oe = strided_extent(qsz, a->out_stride, D), te = strided_extent(tsz, tst, a->table_width);
  if (qe < 0 || ke < 0 || ve < 0 || oe < 0 || te < 0 || !strides_apart(qsz, a->out_stride, D)) return GEMM_W4A4_EINVAL;
  for (int i = 0; i < 3; ++i) {
    if (qsz[i] > 1 && ((a->q_stride[i] | a->out_stride[i]) & 7)) return GEMM_W4A4_EINVAL;
    if (csz[i] > 1 && ((a->k_stride[i] | a->v_stride[i]) & 7)) return GEMM_W4A4_EINVAL;
  }
  // (tokens of v that overlap in memory would bring in what lies behind the last key)
  if (a->k_stride[1] >= (int64_t(1) << 23) || a->v_stride[1] >= (int64_t(1) << 23) || a->v_stride[1] < D) return GEMM_W4A4_EINVAL;
  if (a->batch == 0 || a->q_len == 0 || a->q_heads == 0) return GEMM_W4A4_OK;
  const bool keys = a->pages > 0 && a->table_width > 0;
  if (!a->q || !a->out || !a->lens || (keys && (!a->k_cache || !a->v_cache || !a->table))) return GEMM_W4A4_EINVAL;
  if ((uintptr_t(a->q) | uintptr_t(a->out) | (keys ? uintptr_t(a->k_cache) | uintptr_t(a->v_cache) : 0u)) & 15u) return GEMM_W4A4_EALIGN;
  if ((uintptr_t(a->lse) | uintptr_t(a->lens) | (keys ? uintptr_t(a->table) : 0u)) & 3u) return GEMM_W4A4_EALIGN;
  const PagedPlan pl = paged_plan(a);
  // (a launch holds fewer than 2^32 threads; by the smaller tiles, so that what is refused does not go by the plan)
  constexpr int kRows = FewAttn<128>::ROWS;
  if ((int64_t(pl.rows_all) + kRows - 1) / kRows * a->batch * a->kv_heads >= int64_t(1) << 24) return GEMM_W4A4_EINVAL;
  if (pl.bytes > 0) {
    if (!a->workspace || a->workspace_bytes < pl.bytes) return GEMM_W4A4_ESCRATCH;
    if (uintptr_t(a->workspace) & 15u) return GEMM_W4A4_EALIGN;
  }
  const struct { const void* p; size_t n; } outs[] = {
      {a->out, size_t(oe) * 2}, {a->lse, size_t(a->batch) * size_t(a->q_heads) * size_t(a->q_len) * 4},
      {pl.bytes > 0 ? a->workspace : nullptr, size_t(pl.bytes)}};
  const struct { const void* p; size_t n; } ins[] = {
      {a->q, size_t(qe) * 2}, {keys ? a->k_cache : nullptr, size_t(ke) * 2}, {keys ? a->v_cache : nullptr, size_t(ve) * 2},
      {keys ? a->table : nullptr, size_t(te) * 4}, {a->lens, size_t(a->batch) * 4}};
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
  p.k = static_cast<const uint16_t*>(a->k_cache);
  p.v = static_cast<const uint16_t*>(a->v_cache);
  p.out = static_cast<uint16_t*>(a->out);
  p.lse = a->lse;
  p.kv_lens = a->lens;
  p.part_o = static_cast<float*>(a->workspace);
  p.part_ms = pl.bytes > 0 ? p.part_o + pl.o_bytes / 4 : nullptr;
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = a->q_stride[i];
    p.ks[i] = a->k_stride[i];
    p.vs[i] = a->v_stride[i];
    p.os[i] = a->out_stride[i];
  }
  p.table = a->table;
  p.table_stride = a->batch > 1 ? a->table_stride : 0;
  p.pages = a->pages;
  p.page_size = a->page_size;
  p.page_index = page_index(a->page_size);
  p.q_len = a->q_len;
  p.kv_len = keys ? a->table_width * a->page_size : 0;
  p.kv_heads = a->kv_heads;
  p.D = D;
  p.group = a->q_heads / a->kv_heads;
  p.rows = pl.rows_all;
  p.pairs = a->batch * a->kv_heads;
  p.whole = int(std::min<int64_t>(pl.whole, INT32_MAX));
  p.cut = pl.cut;
  p.parts = pl.parts;
  p.batch = a->batch;
  p.per_seq = pl.tiles * a->kv_heads;
  p.even = pl.even;
  p.c = a->scale * 1.4426950408889634f;
  int tile_rows = pl.rows;
  void* args[] = {&p, &tile_rows};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t grid = pl.whole + int64_t(pl.cut) * pl.parts;
  hipError_t e = hipLaunchKernel(a->f16 ? paged_of<true>(pl.few, D) : paged_of<false>(pl.few, D), dim3(unsigned(grid)), dim3(256), args, 0, st);
  if (e == hipSuccess && pl.cut > 0) {
    const int rows = std::min(tile_rows, pl.rows_all);
    e = hipLaunchKernel(a->f16 ? reinterpret_cast<const void*>(attention_join_kernel<true, Attend::kPaged>)
                               : reinterpret_cast<const void*>(attention_join_kernel<false, Attend::kPaged>),
                        dim3(unsigned((rows * (D / 4) + 255) / 256), unsigned(pl.cut)), dim3(256), args, 0, st);
  }
  return e == hipSuccess ? GEMM_W4A4_OK : GEMM_W4A4_ELAUNCH;
}

}  // namespace w4a4

extern "C" int paged_attention(const paged_attention_t* args, void* stream) { return w4a4::paged_run(args, stream); }

extern "C" int64_t paged_attention_workspace(const paged_attention_t* args) {
  return w4a4::paged_sizes_ok(args) ? w4a4::paged_plan(args).bytes : GEMM_W4A4_EINVAL;
}
