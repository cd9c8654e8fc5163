// cache_append.hip — keys and values of new tokens into a paged cache
// (cache_append in gemm_w4a4.h): a scatter of whole rows, bound by memory at
// many tokens and by the launch at few.
//
// A thread copies one 16-byte run of kAppendTokens tokens, their slots and then
// their loads in flight together.
#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include "gemm_w4a4.h"
#include "w4a4_common.hpp"
#include "w4a4_host.hpp"
#include "w4a4_strided.hpp"

namespace w4a4 {

struct AppendParams {
  const uint16_t *k, *v;
  uint16_t *k_cache, *v_cache;
  const int64_t* slots;
  int64_t ks[2], vs[2];     // token, head
  int64_t kcs[3], vcs[3];   // page, token, head
  int tokens, page_size, slot_count;
  int runs, head_runs;      // 16-byte runs of a token's keys, of a head
};

constexpr int kAppendTokens = 2;

__global__ __launch_bounds__(256) void cache_append_kernel(const AppendParams p) {
  const int u = blockIdx.x * 256 + threadIdx.x;   // run of the token's keys, then of its values
  if (u >= 2 * p.runs) return;
  const bool val = u >= p.runs;
  const int w = val ? u - p.runs : u, head = w / p.head_runs, c = (w - head * p.head_runs) * 8;
  const uint16_t* from = val ? p.v + head * p.vs[1] + c : p.k + head * p.ks[1] + c;
  uint16_t* to = val ? p.v_cache + head * p.vcs[2] + c : p.k_cache + head * p.kcs[2] + c;
  const int64_t step = val ? p.vs[0] : p.ks[0];
  const int64_t page_step = val ? p.vcs[0] : p.kcs[0], token_step = val ? p.vcs[1] : p.kcs[1];
  for (int t0 = blockIdx.y * kAppendTokens; t0 < p.tokens; t0 += gridDim.y * kAppendTokens) {
    int64_t slot[kAppendTokens];
    u32x4 d[kAppendTokens];
#pragma unroll
    for (int i = 0; i < kAppendTokens; ++i) slot[i] = p.slots[min(t0 + i, p.tokens - 1)];
#pragma unroll
    for (int i = 0; i < kAppendTokens; ++i) {
      if (t0 + i >= p.tokens || slot[i] < 0 || slot[i] >= p.slot_count) slot[i] = -1;   // nothing to write
      else d[i] = *reinterpret_cast<const u32x4*>(from + (t0 + i) * step);
    }
#pragma unroll
    for (int i = 0; i < kAppendTokens; ++i)
      if (slot[i] >= 0) {
        const int page = int(slot[i]) / p.page_size, at = int(slot[i]) - page * p.page_size;
        *reinterpret_cast<u32x4*>(to + page * page_step + at * token_step) = d[i];
      }
  }
}

static int cache_append_run(const cache_append_t* a, void* stream) {
  if (!a || a->tokens < 0 || a->tokens > 1 << 30 || a->heads < 1 || a->pages < 0 || a->page_size < 1) return GEMM_W4A4_EINVAL;
  const int D = a->head_dim;
  if (D < 8 || D > CROSS_ATTENTION_MAX_HEAD_DIM || D % 8 != 0) return GEMM_W4A4_EINVAL;
  if (int64_t(a->pages) * a->page_size >= (int64_t(1) << 31) || a->heads >= 1 << 20) return GEMM_W4A4_EINVAL;
  const int nsz[3] = {a->tokens, a->heads, 1}, csz[3] = {a->pages, a->page_size, a->heads};
  const int64_t kst[3] = {a->k_stride[0], a->k_stride[1], 0}, vst[3] = {a->v_stride[0], a->v_stride[1], 0};
  const int64_t ke = strided_extent(nsz, kst, D), ve = strided_extent(nsz, vst, D),
                kce = strided_extent(csz, a->k_cache_stride, D), vce = strided_extent(csz, a->v_cache_stride, D);
  if (ke < 0 || ve < 0 || kce < 0 || vce < 0) return GEMM_W4A4_EINVAL;
  if (!strides_apart(csz, a->k_cache_stride, D) || !strides_apart(csz, a->v_cache_stride, D)) return GEMM_W4A4_EINVAL;
  for (int i = 0; i < 3; ++i) {
    if (i < 2 && nsz[i] > 1 && ((kst[i] | vst[i]) & 7)) return GEMM_W4A4_EINVAL;
    if (csz[i] > 1 && ((a->k_cache_stride[i] | a->v_cache_stride[i]) & 7)) return GEMM_W4A4_EINVAL;
  }
  if (a->tokens == 0 || a->pages == 0) return GEMM_W4A4_OK;
  if (!a->k || !a->v || !a->k_cache || !a->v_cache || !a->slots) return GEMM_W4A4_EINVAL;
  if ((uintptr_t(a->k) | uintptr_t(a->v) | uintptr_t(a->k_cache) | uintptr_t(a->v_cache)) & 15u) return GEMM_W4A4_EALIGN;
  if (uintptr_t(a->slots) & 7u) return GEMM_W4A4_EALIGN;
  const struct { const void* p; size_t n; } outs[] = {{a->k_cache, size_t(kce) * 2}, {a->v_cache, size_t(vce) * 2}},
      ins[] = {{a->k, size_t(ke) * 2}, {a->v, size_t(ve) * 2}, {a->slots, size_t(a->tokens) * 8}};
  for (const auto& o : outs)
    for (const auto& i : ins)
      if (overlaps(o.p, o.n, i.p, i.n)) return GEMM_W4A4_EOVERLAP;
  // Keys and values may lie in one buffer, a page or a token of the one beside that of
  // the other: extents that cross are fine where the strides are the same and the two
  // caches, as one more dimension, stay apart.
  if (overlaps(a->k_cache, size_t(kce) * 2, a->v_cache, size_t(vce) * 2)) {
    const uintptr_t k = uintptr_t(a->k_cache), v = uintptr_t(a->v_cache);
    const int size[4] = {csz[0], csz[1], csz[2], 2};
    const int64_t st[4] = {a->k_cache_stride[0], a->k_cache_stride[1], a->k_cache_stride[2], int64_t((k < v ? v - k : k - v) / 2)};
    for (int i = 0; i < 3; ++i)
      if (csz[i] > 1 && a->k_cache_stride[i] != a->v_cache_stride[i]) return GEMM_W4A4_EOVERLAP;
    if (!strides_apart(size, st, D)) return GEMM_W4A4_EOVERLAP;
  }
  const int dev_rc = check_device();
  if (dev_rc != GEMM_W4A4_OK) return dev_rc;
  AppendParams p{};
  p.k = static_cast<const uint16_t*>(a->k);
  p.v = static_cast<const uint16_t*>(a->v);
  p.k_cache = static_cast<uint16_t*>(a->k_cache);
  p.v_cache = static_cast<uint16_t*>(a->v_cache);
  p.slots = a->slots;
  for (int i = 0; i < 3; ++i) {
    if (i < 2) p.ks[i] = kst[i], p.vs[i] = vst[i];
    p.kcs[i] = a->k_cache_stride[i];
    p.vcs[i] = a->v_cache_stride[i];
  }
  p.tokens = a->tokens;
  p.page_size = a->page_size;
  p.slot_count = a->pages * a->page_size;
  p.head_runs = D / 8;
  p.runs = a->heads * p.head_runs;
  const int64_t groups = (int64_t(a->tokens) + kAppendTokens - 1) / kAppendTokens;
  void* args[] = {&p};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(cache_append_kernel),
                                       dim3(unsigned((2 * p.runs + 255) / 256), unsigned(std::min<int64_t>(groups, 65535))), dim3(256),
                                       args, 0, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GEMM_W4A4_OK : GEMM_W4A4_ELAUNCH;
}

}  // namespace w4a4

extern "C" int cache_append(const cache_append_t* args, void* stream) { return w4a4::cache_append_run(args, stream); }
