// mxfp4_producer.hip — 16-bit activations x [M, K] to the MXFP4 operand of
// gemm_mxfp4 (E2M1 codes [M, K/2], one UE8M0 scale per 32 k at [K/32, M]) and
// lora_act_in [M, R] = x @ lora_down^T (quantize_mxfp4_act in gemm_w4a4.h).
//
// Bound by memory: 2 bytes read and 17/32 written an element. x is read once:
// lane (r, g) of a wave holds row r, k = 32 g .. 32 g + 31 of a 128-wide span,
// one whole scale block, so its largest magnitude needs no other lane, and the
// same registers are the A operand of the LoRA product (the order of k is free
// as long as lora_down is read in the same one).
//
// The scale of a block is a power of two read off the exponent of its largest
// magnitude, and gfx950's FP4 conversion divides by a power of two and rounds
// to nearest even, saturating at 6, exactly, subnormal inputs and the smallest
// scale (2^-127) included (checked against the definition over every 16-bit
// pattern at scale bytes 0 .. 252): two values an instruction.
//
// The waves of a workgroup share its 16 rows and take the spans of K in turn;
// their partial LoRA sums meet in LDS. When the row blocks do not fill the
// chip, K is split over workgroups too; the slices' float32 sums go to the
// caller's workspace and a second launch adds them in slice order.
#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_w4a4.h"
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
};

// 32 values (16 dwords, low half = even k) of one block -> its scale byte and
// codes. Magnitudes order like their bit patterns, NaN above infinity above
// every finite value: a packed 16-bit max.
template <bool F16>
__device__ __forceinline__ uint32_t quantize_block32(const uint32_t (&d)[16], u32x4& codes) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  u16x2 m = __builtin_bit_cast(u16x2, d[0] & 0x7FFF7FFFu);
#pragma unroll
  for (int i = 1; i < 16; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, d[i] & 0x7FFF7FFFu));
  const uint32_t top = max(uint32_t(m[0]), uint32_t(m[1]));
  const bool finite = top < (F16 ? 0x7C00u : 0x7F80u);
  // biased float32 exponent of the largest magnitude (a binary16 subnormal is
  // a normal float32; a bfloat16 one has exponent 0, which the max covers)
  const uint32_t e = __builtin_bit_cast(uint32_t, widen<F16>(uint16_t(finite ? top : 0u))) >> 23;
  const uint32_t byte = uint32_t(max(int(e) - 2, 0));
  const float scale = __builtin_bit_cast(float, byte == 0 ? 0x00400000u : byte << 23);   // 2^(byte - 127)
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if constexpr (F16) {
      const f16x2 v = __builtin_bit_cast(f16x2, d[i]);
      switch (i & 3) {   // the byte must be an immediate; folds after unrolling
        case 0: w[i >> 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w[i >> 2], v, scale, 0); break;
        case 1: w[i >> 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w[i >> 2], v, scale, 1); break;
        case 2: w[i >> 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w[i >> 2], v, scale, 2); break;
        default: w[i >> 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(w[i >> 2], v, scale, 3); break;
      }
    } else {
      const bf16x2 v = __builtin_bit_cast(bf16x2, d[i]);
      switch (i & 3) {
        case 0: w[i >> 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w[i >> 2], v, scale, 0); break;
        case 1: w[i >> 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w[i >> 2], v, scale, 1); break;
        case 2: w[i >> 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w[i >> 2], v, scale, 2); break;
        default: w[i >> 2] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w[i >> 2], v, scale, 3); break;
      }
    }
  }
  codes = finite ? u32x4{w[0], w[1], w[2], w[3]} : u32x4{0u, 0u, 0u, 0u};
  return finite ? byte : 0xFFu;
}

constexpr int kMxProdWaves = 8;
constexpr int kMxProdRows = 16;

// RT: rank tiles of 16 (0: no LoRA product).
template <bool F16, int RT>
__global__ __launch_bounds__(kMxProdWaves * kWave) void mx_producer_kernel(const MxProdParams p) {
  constexpr int W = kMxProdWaves;
  __shared__ f32x4 red[RT > 0 ? W * RT * kWave : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int M = p.M, K = p.K, R = p.R;
  const int rb = blockIdx.x / p.ks, z = blockIdx.x - rb * p.ks;
  const int m0 = rb * kMxProdRows;
  const int nsp = (K + 127) / 128;
  const int s_end = min(nsp, (z + 1) * p.sps);
  const int row = min(m0 + r, M - 1);     // rows past M repeat the last and are not stored
  const bool live_row = m0 + r < M;
  const uint16_t* xr = p.x + size_t(row) * size_t(K);
  f32x4 acc[RT > 0 ? RT : 1];
#pragma unroll
  for (int j = 0; j < RT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int s = z * p.sps + wave; s < s_end; s += W) {
    const int k0 = s * 128 + 32 * g;
    const bool live = k0 < K;              // K % 32 == 0: a block is in or out whole
    uint32_t d[16];
    u32x4 b[RT > 0 ? RT : 1][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4 v = live ? *reinterpret_cast<const u32x4*>(xr + k0 + 8 * i) : u32x4{0u, 0u, 0u, 0u};
      d[4 * i] = v.x;
      d[4 * i + 1] = v.y;
      d[4 * i + 2] = v.z;
      d[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      // ranks past R repeat the last; their sums are not stored
      const uint16_t* l = p.lora_down + size_t(min(16 * j + r, R - 1)) * size_t(K) + k0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        b[j][i] = live ? *reinterpret_cast<const u32x4*>(l + 8 * i) : u32x4{0u, 0u, 0u, 0u};
    }
    u32x4 codes;
    const uint32_t byte = quantize_block32<F16>(d, codes);
    if (live && live_row) {
      *reinterpret_cast<u32x4*>(p.act + size_t(row) * size_t(K / 2) + k0 / 2) = codes;
      p.ascales[size_t(k0 / 32) * size_t(M) + row] = uint8_t(byte);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x4 a = {d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]};
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[j] = mfma16<F16>(a, b[j][i], acc[j]);
    }
  }

  if constexpr (RT > 0) {
#pragma unroll
    for (int j = 0; j < RT; ++j) red[(wave * RT + j) * kWave + lane] = acc[j];
    __syncthreads();
    // lane (c, g) of rank tile j holds rows 4g .. 4g+3 of rank 16 j + c
    for (int j = wave; j < RT; j += W) {
      f32x4 t = red[j * kWave + lane];
#pragma unroll
      for (int w = 1; w < W; ++w) t += red[(w * RT + j) * kWave + lane];
      const int rank = 16 * j + (lane & 15);
      if (rank >= R) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int m = m0 + 4 * g + e;
        if (m >= M) continue;
        if (p.ks > 1)
          p.part[(size_t(z) * size_t(M) + m) * size_t(R) + rank] = t[e];
        else
          p.lora_act_in[size_t(m) * size_t(R) + rank] = narrow<F16>(t[e]);
      }
    }
  }
}

// lora_act_in = the slices' sums added in slice order.
template <bool F16>
__global__ __launch_bounds__(256) void mx_producer_join_kernel(const MxProdParams p) {
  const size_t n = size_t(p.M) * size_t(p.R), i = size_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  float t = p.part[i];
#pragma unroll 4
  for (int z = 1; z < p.ks; ++z) t += p.part[size_t(z) * n + i];
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
  int ks, sps;
  int64_t bytes;
};

static MxProdPlan mx_prod_plan(int M, int K, int R) {
  const int rbs = (M + kMxProdRows - 1) / kMxProdRows, nsp = (K + 127) / 128;
  const int ks = std::max(1, std::min((nsp + kMxProdWaves - 1) / kMxProdWaves, mx_cus() / rbs));
  MxProdPlan pl;
  pl.sps = (nsp + ks - 1) / ks;
  pl.ks = (nsp + pl.sps - 1) / pl.sps;
  pl.bytes = pl.ks > 1 && R > 0 ? int64_t(pl.ks) * M * R * 4 : 0;
  return pl;
}

static bool mx_prod_sizes_ok(int M, int K, int R) {
  if (!(M >= 1 && K >= 32 && K % 32 == 0 && R >= 0 && R <= QUANTIZE_W4A4_MAX_R)) return false;
  const int64_t lim = int64_t(1) << 31;
  return int64_t(M) * K * 2 < lim && int64_t(R) * K * 2 < lim && int64_t(M) * R * 2 < lim;
}

template <bool F16>
static const void* mx_producer_of(int R) {
  if (R == 0) return reinterpret_cast<const void*>(mx_producer_kernel<F16, 0>);
  if (R <= 16) return reinterpret_cast<const void*>(mx_producer_kernel<F16, 1>);
  if (R <= 32) return reinterpret_cast<const void*>(mx_producer_kernel<F16, 2>);
  if (R <= 64) return reinterpret_cast<const void*>(mx_producer_kernel<F16, 4>);
  return reinterpret_cast<const void*>(mx_producer_kernel<F16, 8>);
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
  MxProdParams p{x, lora_down, act, ascales, lora_act_in, static_cast<float*>(workspace), M, K, R, pl.ks, pl.sps};
  void* args[] = {&p};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const int rbs = (M + kMxProdRows - 1) / kMxProdRows;
  hipError_t e = hipLaunchKernel(mx_producer_of<F16>(R), dim3(unsigned(rbs) * unsigned(pl.ks)),
                                 dim3(kMxProdWaves * kWave), args, 0, st);
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
