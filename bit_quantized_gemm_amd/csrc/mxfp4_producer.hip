// mxfp4_producer.hip — 16-bit activations x [M, K] to the MXFP4 operand of
// gemm_mxfp4 (E2M1 codes [M, K/2], one UE8M0 scale per 32 k at [K/32, M]) and
// lora_act_in [M, R] = x @ lora_down^T (quantize_mxfp4_act in gemm_w4a4.h).
//
// Bound by memory: 2 bytes read and 17/32 written an element. x is read once,
// in the layout of the LoRA product's A operand: lane (r, g) of a wave holds row
// r, k = 32 i + 8 g .. + 7 for the four blocks i of a 128-wide span, so that
// four lanes read 64 neighbouring bytes (one whole block a lane, 64 bytes
// apart, cost four times the cache cycles). 4096 x 3072, R = 32: 11.3 us, 2.85
// TB/s; 1001 x 12288, R = 128: 16.0 us, 2.2 TB/s. Past the launches, each of the
// loads, the quantisation, the products and the stores adds its part of a span's
// chain: no one of them alone bounds it. A block's largest magnitude meets over its four lanes by lane swaps, and so
// do its codes, which leave as 16 bytes a lane.
//
// The scale of a block is a power of two read off the exponent of its largest
// magnitude, and gfx950's FP4 conversion divides by a power of two and rounds
// to nearest even, saturating at 6, exactly, subnormal inputs and the smallest
// scale (2^-127) included (checked against the definition over every 16-bit
// pattern at scale bytes 0 .. 252): two values an instruction.
//
// Few ranks or rows: the waves of a workgroup share its 16 rows and take the
// spans of K in turn; their partial LoRA sums meet in LDS. Else 16 rows a wave,
// and lora_down shared in LDS. When the row blocks do not fill the chip, K is
// split over workgroups too; the slices' float32 sums go to the caller's
// workspace and a second launch adds them in slice order.
#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_w4a4.h"
#include "w4a4_buffer.hpp"
#include "w4a4_common.hpp"
#include "w4a4_half.hpp"
#include "w4a4_host.hpp"

namespace w4a4 {

struct MxProdParams {
  const uint16_t* x;
  const uint16_t* lora_down;
  uint8_t* act;
  uint8_t* ascales;
  uint16_t* lora_act_in;
  float* part;          // ks > 1 and R > 0: [slice][M][R] float32 sums
  int M, K, R;
  int ks, sps;          // K slices, spans per slice
  int groups;           // workgroups that share rows and slice, some rank tiles each
};

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// max over the lanes l, l ^ 16, l ^ 32, l ^ 48, of both halves of a dword
__device__ __forceinline__ u16x2 max_of_four(u16x2 v) {
  const uint32_t a = __builtin_bit_cast(uint32_t, v);
  const auto s = __builtin_amdgcn_permlane32_swap(a, a, false, false);
  const u16x2 m = __builtin_elementwise_max(__builtin_bit_cast(u16x2, uint32_t(s[0])), __builtin_bit_cast(u16x2, uint32_t(s[1])));
  const uint32_t b = __builtin_bit_cast(uint32_t, m);
  const auto t = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  return __builtin_elementwise_max(__builtin_bit_cast(u16x2, uint32_t(t[0])), __builtin_bit_cast(u16x2, uint32_t(t[1])));
}

// 8 values (low half = even k) divided by a power of two -> 8 codes. (The
// dwords are copied out first: this compiler's bit-cast of a vector element
// reads the vector's first one.)
template <bool F16>
__device__ __forceinline__ uint32_t codes_of(const u32x4& d, float scale) {
  uint32_t w = 0u;
  const uint32_t d0 = d.x, d1 = d.y, d2 = d.z, d3 = d.w;
  if constexpr (F16) {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(f16x2, d0), scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(f16x2, d1), scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(f16x2, d2), scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w, __builtin_bit_cast(f16x2, d3), scale, 3);
  } else {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, d0), scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, d1), scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, d2), scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, d3), scale, 3);
  }
  return w;
}

// The four blocks of a span, d[i] this lane's 8 values of block i -> the
// scale byte and the 16 bytes of codes of block g. Magnitudes order like their
// bit patterns, NaN above infinity above every finite value.
template <bool F16>
__device__ __forceinline__ uint32_t quantize_span(const u32x4 (&d)[4], int g, u32x4& codes) {
  u16x2 pairs[2];   // maxima of blocks 0 and 1, 2 and 3
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u16x2 m = __builtin_bit_cast(u16x2, d[i].x & 0x7FFF7FFFu);
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, d[i].y & 0x7FFF7FFFu));
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, d[i].z & 0x7FFF7FFFu));
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, d[i].w & 0x7FFF7FFFu));
    pairs[i >> 1][i & 1] = m[0] > m[1] ? m[0] : m[1];
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) pairs[i] = max_of_four(pairs[i]);
  uint32_t c[4], byte[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t top = pairs[i >> 1][i & 1];
    const bool finite = top < (F16 ? 0x7C00u : 0x7F80u);
    // biased float32 exponent of the largest magnitude (a binary16 subnormal
    // is a normal float32; a bfloat16 one has exponent 0, which the max covers)
    const uint32_t e = __builtin_bit_cast(uint32_t, widen<F16>(uint16_t(finite ? top : 0u))) >> 23;
    const uint32_t b = uint32_t(max(int(e) - 2, 0));
    const float scale = __builtin_bit_cast(float, b == 0 ? 0x00400000u : b << 23);   // 2^(b - 127)
    const uint32_t w = codes_of<F16>(d[i], scale);
    c[i] = finite ? w : 0u;
    byte[i] = finite ? b : 0xFFu;
  }
  // lane g's c[i] is bytes 4 g .. + 3 of block i; afterwards word s of lane g is
  // lane s's of block g
  const auto a = __builtin_amdgcn_permlane32_swap(c[0], c[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(c[1], c[3], false, false);
  const auto lo = __builtin_amdgcn_permlane16_swap(uint32_t(a[0]), uint32_t(b[0]), false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(uint32_t(a[1]), uint32_t(b[1]), false, false);
  codes = u32x4{uint32_t(lo[0]), uint32_t(lo[1]), uint32_t(hi[0]), uint32_t(hi[1])};
  const uint32_t b01 = g & 1 ? byte[1] : byte[0], b23 = g & 1 ? byte[3] : byte[2];
  return g & 2 ? b23 : b01;
}

constexpr int kMxProdWaves = 8;

// A workgroup a 16 rows, or one for each of `groups` rank tiles of them, of
// which the first writes the codes. LORA: 0 < R.
template <bool F16, bool LORA>
__global__ __launch_bounds__(kMxProdWaves * kWave) void mx_producer_kernel(const MxProdParams p) {
  constexpr int W = kMxProdWaves;
  __shared__ f32x4 red[LORA ? W * kWave : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int M = p.M, K = p.K, R = p.R;
  const int q0 = blockIdx.x % p.groups, blk = blockIdx.x / p.groups;
  const int rb = blk / p.ks, z = blk - rb * p.ks;
  const int m0 = rb * 16;
  const int nsp = (K + 127) / 128;
  const int s_end = min(nsp, (z + 1) * p.sps);
  const int row = min(m0 + r, M - 1);   // rows past M repeat the last and are not stored
  const bool live = m0 + r < M;
  const int rank = 16 * q0 + r;         // ranks past R repeat the last; their sums are not stored
  const uint16_t* xr = p.x + size_t(row) * size_t(K) + 8 * g;
  const uint16_t* lr = LORA ? p.lora_down + size_t(min(rank, R - 1)) * size_t(K) + 8 * g : nullptr;
  f32x4 acc{0.f, 0.f, 0.f, 0.f};

  // A span's x and lora_down operands are asked for one span ahead. TAIL: the
  // span that K ends in; its blocks past K (K % 32 == 0: in or out whole) read
  // as zeros.
  u32x4 x[2][4], b[2][4];
  auto load = [&]<bool TAIL>(const uint16_t* from, int k) __attribute__((always_inline)) {
    return !TAIL || k < K ? *reinterpret_cast<const u32x4*>(from + k) : u32x4{0u, 0u, 0u, 0u};
  };
  auto ask = [&]<bool TAIL>(int q, int s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[q][i] = load.template operator()<TAIL>(xr, s * 128 + 32 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if constexpr (LORA) b[q][i] = load.template operator()<TAIL>(lr, s * 128 + 32 * i);
  };
  auto work = [&]<bool TAIL>(int q, int s) __attribute__((always_inline)) {
    const int k = s * 128 + 32 * g;
    u32x4 codes;
    const uint32_t byte = quantize_span<F16>(x[q], g, codes);
    if (live && q0 == 0 && (!TAIL || k < K)) {
      *reinterpret_cast<u32x4*>(p.act + size_t(row) * size_t(K / 2) + k / 2) = codes;
      p.ascales[size_t(k / 32) * size_t(M) + row] = uint8_t(byte);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if constexpr (LORA) acc = mfma16<F16>(x[q][i], b[q][i], acc);
  };
  const int e = min(s_end, K / 128);   // past the whole spans
  int s = z * p.sps + wave;
  if (s < e) ask.template operator()<false>(0, s);
  for (; s < e; s += 2 * W) {
    if (s + W < e) ask.template operator()<false>(1, s + W);
    work.template operator()<false>(0, s);
    if (s + 2 * W < e) ask.template operator()<false>(0, s + 2 * W);
    if (s + W < e) work.template operator()<false>(1, s + W);
  }
  if (e < s_end && (e - z * p.sps) % W == wave) {   // the span that K ends in
    ask.template operator()<true>(0, e);
    work.template operator()<true>(0, e);
  }

  if constexpr (LORA) {
    red[wave * kWave + lane] = acc;
    __syncthreads();
    if (wave != 0) return;
    f32x4 sum = red[lane];
#pragma unroll
    for (int w = 1; w < W; ++w) sum += red[w * kWave + lane];
    if (rank >= R) return;
    // lane (c, g) holds rows 4g .. 4g+3 of rank c of the tile
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = m0 + 4 * g + i;
      if (m >= M) continue;
      if (p.ks > 1)
        p.part[(size_t(z) * size_t(M) + m) * size_t(R) + rank] = sum[i];
      else
        p.lora_act_in[size_t(m) * size_t(R) + rank] = narrow<F16>(sum[i]);
    }
  }
}

// Read per 16 rows, lora_down outweighs x by R / 16 (and both come out of the
// same cache), so for many ranks, or many rows, a workgroup takes 16 W rows, 16 a
// wave, and its waves share each span's lora_down tile in LDS. Both it and the
// waves' own x come by direct-to-LDS loads two spans ahead, lora_down in a ring
// of three, x in one of two (a wave has read its x before it asks for more).
// The chunks of a row are XOR-swizzled by row: no read meets a bank twice. 32
// rows a wave would halve the reads of lora_down from LDS, but its fewer waves
// cost more (4096 x 12288, R = 128: 40.4 us against 35.5).
template <int RT_, int W_>
struct MxShared {
  static constexpr int RT = RT_, W = W_, ROWS = 16 * W, RING = 3;
  static constexpr int TILE = RT * 16 * 256;          // a span of lora_down
  static constexpr int LOADS = RT * 4 / W;            // a wave's loads of it, 4 ranks each
  static constexpr int XTILE = 16 * 256;              // a span of a wave's x, 4 loads
  static constexpr int XOFF = RING * TILE;
  static constexpr int LDS = XOFF + W * 2 * XTILE;
  // What a wave has asked for after the loads of the span that is needed: the
  // loads of the next span, and past the first span two stores of codes, or four.
  static constexpr int YOUNGER = LOADS + 4;
  static_assert(RT * 4 % W == 0 && LDS <= kLdsLimit && YOUNGER + 2 < 64, "LDS and wait counter");
};

template <bool F16, class C>
__global__ __launch_bounds__(C::W * kWave) void mx_producer_shared_kernel(const MxProdParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::LDS];
  constexpr int RT = C::RT;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int M = p.M, K = p.K, R = p.R;
  const int blocks = gridDim.x / p.groups;   // the groups of a block often meet on one XCD
  const int q0 = blockIdx.x / blocks, blk = blockIdx.x - q0 * blocks;
  const int rb = blk / p.ks, z = blk - rb * p.ks;
  const int mw = rb * C::ROWS + 16 * wave;
  const int nsp = (K + 127) / 128;
  const int s_beg = z * p.sps, s_end = min(nsp, s_beg + p.sps);
  const uint32_t row_bytes = uint32_t(K) * 2u, l_bytes = uint32_t(R) * row_bytes, x_bytes = uint32_t(M) * row_bytes;
  // this lane's place in a load: row 4 u + lane / 16 of the tile, chunk position
  // lane % 16. Rows past M repeat the last and are not stored; ranks past R are
  // past the tensor (zeros).
  uint32_t loff[C::LOADS], xoff[4];
  int xk[4], lk[C::LOADS];   // first k of the lane's chunk in the span
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    xk[u] = 8 * (r ^ (4 * u + g));
    xoff[u] = uint32_t(min(mw + 4 * u + g, M - 1)) * row_bytes + uint32_t(xk[u]) * 2u;
  }
#pragma unroll
  for (int u = 0; u < C::LOADS; ++u) {
    const int rank = q0 * RT * 16 + (wave * C::LOADS + u) * 4 + g;
    lk[u] = 8 * (r ^ (rank & 15));
    loff[u] = uint32_t(rank) * row_bytes + uint32_t(lk[u]) * 2u;
  }
  const uint32_t lds_l = lds_address(smem) + wave * C::LOADS * 1024;
  const uint32_t lds_x = lds_address(smem) + C::XOFF + wave * 2 * C::XTILE;
  // What lies past K, and whole spans past the slice, read as zeros: offsets
  // out of every range.
  auto ask_x = [&](int s, int place) __attribute__((always_inline)) {
    const bool in = s < s_end;
    const uint32_t at = in ? uint32_t(s) * 256u : 0u;
    const u32x4 d = range_desc(reinterpret_cast<const uint8_t*>(p.x) + at, in ? x_bytes - at : 0u);
#pragma unroll
    for (int u = 0; u < 4; ++u) load_to_lds(d, s * 128 + xk[u] < K ? xoff[u] : 0xFFFFFFF0u, lds_x + place * C::XTILE + u * 1024);
  };
  auto ask_l = [&](int s, int place) __attribute__((always_inline)) {
    const bool in = s < s_end;
    const uint32_t at = in ? uint32_t(s) * 256u : 0u;
    const u32x4 d = range_desc(reinterpret_cast<const uint8_t*>(p.lora_down) + at, in ? l_bytes - at : 0u);
#pragma unroll
    for (int u = 0; u < C::LOADS; ++u) load_to_lds(d, s * 128 + lk[u] < K ? loff[u] : 0xFFFFFFF0u, lds_l + place * C::TILE + u * 1024);
  };
  f32x4 acc[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const bool live = mw + r < M;
  const int row = min(mw + r, M - 1);
  const uint32_t act_row = uint32_t(row) * (uint32_t(K) / 2u);
  const auto act = __builtin_amdgcn_make_buffer_rsrc(p.act, 0, int(uint32_t(M) * (uint32_t(K) / 2u)), 0x00020000);
  const auto ascales = __builtin_amdgcn_make_buffer_rsrc(p.ascales, 0, int(uint32_t(K / 32) * uint32_t(M)), 0x00020000);

  ask_x(s_beg, 0);
  ask_l(s_beg, 0);
  ask_x(s_beg + 1, 1);
  ask_l(s_beg + 1, 1);
  int place = 0;   // of the span in the ring of three
  for (int s = s_beg; s < s_end; ++s) {
    if (s == s_beg || q0 > 0) wait_vm_lgkm0<C::YOUNGER>();   // this wave's loads of the span
    else wait_vm_lgkm0<C::YOUNGER + 2>();
    wg_barrier();                  // everyone's, and everyone past the span before
    const int xp = (s - s_beg) & 1;
    u32x4 x[4], codes;
    const uint8_t* xt = smem + C::XOFF + (wave * 2 + xp) * C::XTILE + r * 256;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const u32x4*>(xt + (((4 * i + g) ^ r) << 4));
    __builtin_amdgcn_sched_barrier(0);
    wait_vm_lgkm0<63>();           // x is read
    ask_x(s + 2, xp);
    ask_l(s + 2, place == 0 ? 2 : place - 1);
    // the products' operands of step i + 1 are read before step i's products: one
    // wave a SIMD has nothing else to hide the reads behind
    const uint8_t* t = smem + place * C::TILE + r * 256;
    u32x4 b[2][RT];
    auto read_b = [&](int i) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < RT; ++j) b[i & 1][j] = *reinterpret_cast<const u32x4*>(t + j * 4096 + (((4 * i + g) ^ r) << 4));
      __builtin_amdgcn_sched_barrier(0);
    };
    read_b(0);
    if (q0 == 0) {
      const uint32_t byte = quantize_span<F16>(x, g, codes);
      const int k = s * 128 + 32 * g;
      // (no branch a lane: every wave issues both stores, which the waits count)
      const bool keep = live && k < K;
      __builtin_amdgcn_raw_buffer_store_b128(codes, act, keep ? act_row + uint32_t(k) / 2u : 0xFFFFFFF0u, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b8(uint8_t(byte), ascales, keep ? uint32_t(k / 32) * uint32_t(M) + uint32_t(row) : 0xFFFFFFF0u, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < 3) read_b(i + 1);
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[j] = mfma16<F16>(x[i], b[i & 1][j], acc[j]);
      __builtin_amdgcn_sched_barrier(0);
    }
    place = place == 2 ? 0 : place + 1;
  }
  wait_vm<0>();

  // lane (c, g) of tile j holds rows 4g .. 4g+3 of rank 16 j + c; the descriptor
  // drops what lies past M or R
  const bool cut = p.ks > 1;
  const uint32_t n = uint32_t(M) * uint32_t(R);
  const auto sums = cut ? __builtin_amdgcn_make_buffer_rsrc(p.part + size_t(z) * n, 0, int(n * 4u), 0x00020000)
                        : __builtin_amdgcn_make_buffer_rsrc(p.lora_act_in, 0, int(n * 2u), 0x00020000);
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int rank = 16 * (q0 * RT + j) + r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int m = mw + 4 * g + e;
      const bool in = m < M && rank < R;
      const uint32_t at = uint32_t(m) * uint32_t(R) + uint32_t(rank);
      const float sum = acc[j][e];
      if (cut)
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, sum), sums, in ? at * 4u : 0xFFFFFFF0u, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b16(narrow<F16>(sum), sums, in ? at * 2u : 0xFFFFFFF0u, 0, 0);
    }
  }
}

// lora_act_in = the slices' sums added in slice order.
template <bool F16>
__global__ __launch_bounds__(256) void mx_producer_join_kernel(const MxProdParams p) {
  const size_t n = size_t(p.M) * size_t(p.R), i = size_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  float t = 0.f;
  int z = 0;
  for (; z + 8 <= p.ks; z += 8) {   // eight slices' sums in flight
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = p.part[size_t(z + u) * n + i];
#pragma unroll
    for (int u = 0; u < 8; ++u) t += v[u];
  }
  for (; z < p.ks; ++z) t += p.part[size_t(z) * n + i];
  p.lora_act_in[i] = narrow<F16>(t);
}

// ------------------------------------------------------------------ host side

static int mx_cus() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return kNumCUs;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n <= 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) return kNumCUs;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

struct MxProdPlan {
  int shared;    // waves of the kernel that shares lora_down; 0: the other
  int threads;
  int rbs;       // row blocks
  int ks, sps;   // K slices, spans of a slice
  int tiles;     // rank tiles of a workgroup (0 or 1; shared: 2, 4, 8)
  int groups;    // workgroups that share the rank tiles of rows and slice
  int64_t bytes;
};

// Which kernel, measured (us, with the join where there is one): unshared
// against shared of 4 waves: 4096x3072 R=32 11.9 and 10.3, R=16 9.2 and 10.1,
// 2048x12288 R=32 23.7 and 15.9, 256x3072 R=32 7.3 and 5.2, 3000x3072 R=8 7.7 and
// 9.3, 256x12288 R=16 (both in slices) 8.5 and 6.8: shared for more than 16
// ranks, and for fewer where x is large or the other would need slices too.
// 8 waves of shared against 4: 4096x12288 R=128 38.4 and 43.5, 3000x6144 R=96
// 18.7 and 19.8, 4096x3072 R=128 18.1 and 16.6: 8 for more than 64 ranks of a
// large x.
static MxProdPlan mx_prod_plan(int M, int K, int R) {
  MxProdPlan pl;
  const int64_t size = int64_t(M) * K;
  const int nsp = (K + 127) / 128;
  const bool sliced = nsp / (2 * kMxProdWaves) > 1 && mx_cus() / ((M + 15) / 16) > 1;
  pl.shared = M <= 16 || R == 0 ? 0
              : R > 64 && size >= (int64_t(1) << 24) ? 8
              : R > 16 || M > 4096 || size >= (int64_t(1) << 25) || sliced ? 4 : 0;
  const int waves = pl.shared ? pl.shared : kMxProdWaves, rows = pl.shared ? 16 * waves : 16;
  pl.threads = waves * kWave;
  pl.rbs = (M + rows - 1) / rows;
  // slices that fill the chip once; of at least 2 spans a wave, or 3 of a
  // workgroup that shares them
  const int ks = std::max(1, std::min(nsp / (pl.shared ? 3 : 2 * waves), mx_cus() / pl.rbs));
  pl.sps = (nsp + ks - 1) / ks;
  pl.ks = (nsp + pl.sps - 1) / pl.sps;
  // Up to 16 rows: a workgroup for each rank tile, since one compute unit takes
  // 2.6 us to fetch a tile of 3072 k (4x3072 R=32: 8.3 us with both tiles in one
  // workgroup, 6.0 apart). Where lora_down is shared, pairs of tiles or more are
  // dealt to the compute units that are free (512x3072 R=128: 8.0 us with the 8
  // tiles in one workgroup, 5.9 in four; 64x12288 R=128 7.7 and 5.5).
  if (pl.shared) {
    pl.groups = 1;
    pl.tiles = pl.shared == 8 || R > 64 ? 8 : R > 32 ? 4 : 2;
    if (pl.shared == 4)
      for (; pl.tiles > 2 && int64_t(pl.rbs) * pl.ks * pl.groups * 2 <= mx_cus(); pl.tiles /= 2) pl.groups *= 2;
  } else {
    pl.groups = std::max(1, (R + 15) / 16);
    pl.tiles = R > 0;
  }
  pl.bytes = pl.ks > 1 && R > 0 ? int64_t(pl.ks) * M * R * 4 : 0;
  return pl;
}

static bool mx_prod_sizes_ok(int M, int K, int R) {
  if (!(M >= 1 && K >= 32 && K % 32 == 0 && R >= 0 && R <= QUANTIZE_W4A4_MAX_R)) return false;
  const int64_t lim = int64_t(1) << 31;
  return int64_t(M) * K * 2 < lim && int64_t(R) * K * 2 < lim && int64_t(M) * R * 2 < lim;
}

template <bool F16>
static const void* mx_producer_of(const MxProdPlan& pl) {
  if (pl.shared == 8) return reinterpret_cast<const void*>(mx_producer_shared_kernel<F16, MxShared<8, 8>>);
  if (pl.shared)
    return pl.tiles == 2 ? reinterpret_cast<const void*>(mx_producer_shared_kernel<F16, MxShared<2, 4>>)
         : pl.tiles == 4 ? reinterpret_cast<const void*>(mx_producer_shared_kernel<F16, MxShared<4, 4>>)
                         : reinterpret_cast<const void*>(mx_producer_shared_kernel<F16, MxShared<8, 4>>);
  return pl.tiles ? reinterpret_cast<const void*>(mx_producer_kernel<F16, true>)
                  : reinterpret_cast<const void*>(mx_producer_kernel<F16, false>);
}

template <bool F16>
static int mx_quantize_run(const uint16_t* x, const uint16_t* lora_down, uint8_t* act, uint8_t* ascales,
                           uint16_t* lora_act_in, int M, int K, int R, void* workspace, int64_t workspace_bytes,
                           void* stream) {
  if (!mx_prod_sizes_ok(M, K, R)) return GEMM_W4A4_EINVAL;
  if (!x || !act || !ascales || (R > 0 && (!lora_down || !lora_act_in))) return GEMM_W4A4_EINVAL;
  if ((uintptr_t(x) | uintptr_t(act) | (R > 0 ? uintptr_t(lora_down) : 0u)) & 15u) return GEMM_W4A4_EALIGN;
  if (R > 0 && (uintptr_t(lora_act_in) & 1u)) return GEMM_W4A4_EALIGN;
  const MxProdPlan pl = mx_prod_plan(M, K, R);
  if (pl.bytes > 0) {
    if (!workspace || workspace_bytes < pl.bytes) return GEMM_W4A4_ESCRATCH;
    if (uintptr_t(workspace) & 15u) return GEMM_W4A4_EALIGN;
  }
  const size_t Ms = size_t(M), Ks = size_t(K), Rs = size_t(R);
  const struct { const void* p; size_t n; } outs[] = {
      {act, Ms * Ks / 2}, {ascales, Ks / 32 * Ms}, {lora_act_in, R > 0 ? Ms * Rs * 2 : 0},
      {pl.bytes > 0 ? workspace : nullptr, size_t(pl.bytes)}};
  const struct { const void* p; size_t n; } ins[] = {{x, Ms * Ks * 2}, {lora_down, Rs * Ks * 2}};
  for (int a = 0; a < 4; ++a) {
    for (const auto& in : ins)
      if (overlaps(outs[a].p, outs[a].n, in.p, in.n)) return GEMM_W4A4_EOVERLAP;
    for (int b = a + 1; b < 4; ++b)
      if (overlaps(outs[a].p, outs[a].n, outs[b].p, outs[b].n)) return GEMM_W4A4_EOVERLAP;
  }
  const int dev_rc = check_device();
  if (dev_rc != GEMM_W4A4_OK) return dev_rc;
  MxProdParams p{x, lora_down, act, ascales, lora_act_in, static_cast<float*>(workspace),
                 M, K, R, pl.ks, pl.sps, pl.groups};
  void* args[] = {&p};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = hipLaunchKernel(mx_producer_of<F16>(pl),
                                 dim3(unsigned(pl.rbs) * unsigned(pl.ks) * unsigned(pl.groups)),
                                 dim3(pl.threads), args, 0, st);
  if (e == hipSuccess && pl.bytes > 0)
    e = hipLaunchKernel(reinterpret_cast<const void*>(mx_producer_join_kernel<F16>),
                        dim3(unsigned((Ms * Rs + 255) / 256)), dim3(256), args, 0, st);
  return e == hipSuccess ? GEMM_W4A4_OK : GEMM_W4A4_ELAUNCH;
}

}  // namespace w4a4

extern "C" int quantize_mxfp4_act(const uint16_t* x, const uint16_t* lora_down, uint8_t* act, uint8_t* ascales,
                                  uint16_t* lora_act_in, int M, int K, int R, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
  return w4a4::mx_quantize_run<false>(x, lora_down, act, ascales, lora_act_in, M, K, R, workspace, workspace_bytes, stream);
}

extern "C" int quantize_mxfp4_act_f16(const uint16_t* x, const uint16_t* lora_down, uint8_t* act, uint8_t* ascales,
                                      uint16_t* lora_act_in, int M, int K, int R, void* workspace,
                                      int64_t workspace_bytes, void* stream) {
  return w4a4::mx_quantize_run<true>(x, lora_down, act, ascales, lora_act_in, M, K, R, workspace, workspace_bytes, stream);
}

extern "C" int64_t quantize_mxfp4_workspace(int M, int K, int R) {
  return w4a4::mx_prod_sizes_ok(M, K, R) ? w4a4::mx_prod_plan(M, K, R).bytes : GEMM_W4A4_EINVAL;
}
