// mxfp4_few.hip — gemm_mxfp4's operation for few rows (gemm_mxfp4_few in
// gemm_w4a4.h):
//
// y[m,n] = wcscale[n] * sum_k A[m,k] W[n,k] + bias[n] + sum_r la[m,r] lu[r,n]
//
// Bound by the weight bytes, N (K/2 + K/32): every weight is read once, from
// HBM straight into the registers that the matrix instruction takes, since no
// two waves share one. A workgroup owns 4 to 64 columns; its waves split K in
// steps of 128 and add their sums through LDS. v_mfma_scale_f32_16x16x128_f8f6f4
// with FP4 operands: lane (c, g) holds row c, k = 32 g .. 32 g + 31 as 16 bytes
// and that block's scale byte. The weights are its A operand (rows n) and the
// activations, which stay in cache, its B operand (columns m), so that a lane
// ends with 4 neighbouring columns n of one row m. Each wave adds its share
// of the LoRA ranks to its own sums, after the factor wcscale that the LoRA
// term does not take. M x K x N 1x12288x12288: 15.0 us, 5.3 TB/s; 1x3072x12288 7.0 and
// 16x12288x3072 9.4, of which the launch takes 2.8. Past 16 rows the activations
// that every workgroup reads from L2 bound it (64x12288x12288: 33 us).
#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_w4a4.h"
#include "w4a4_common.hpp"
#include "w4a4_half.hpp"
#include "w4a4_host.hpp"

namespace w4a4 {

__device__ __forceinline__ f32x4 mfma_fp4_16(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  typedef int v8i __attribute__((ext_vector_type(8)));
  const v8i av = {int(a.x), int(a.y), int(a.z), int(a.w), 0, 0, 0, 0};   // FP4 uses the low 4 dwords
  const v8i bv = {int(b.x), int(b.y), int(b.z), int(b.w), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, int(sa), 0, int(sb));
}

// MT tiles of 16 rows (M <= 16 MT), NT of 16 columns, W waves, P steps a run (of
// a row's neighbouring bytes).
template <int MT_, int NT_, int W_, int P_>
struct FewCfg {
  static constexpr int MT = MT_, NT = NT_, W = W_, P = P_, THREADS = W * kWave, COLS = 16 * NT;
  static constexpr bool AHEAD = MT > 1;
};

template <bool F16, class C>
__global__ __launch_bounds__(C::THREADS) void mx_few_kernel(const Params p, int cols) {
  constexpr int W = C::W, MT = C::MT, NT = C::NT, P = C::P;
  __shared__ f32x4 red[W * NT * MT * kWave];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int M = p.M, N = p.N, K = p.K, R = p.R;
  // Workgroup b runs on XCD b % 8; each XCD takes neighbouring columns, which share
  // the cache lines of the scales (16 columns read 16 bytes of a row of wscales:
  // 1x12288x12288 19.0 us in order, 15.0 so).
  const int xcd = blockIdx.x % 8, per = gridDim.x / 8, rem = gridDim.x % 8;
  const int n0 = (xcd * per + min(xcd, rem) + int(blockIdx.x / 8)) * cols;
  const int kb_all = K >> 5;
  const uint32_t rowbytes = uint32_t(K) >> 1;
  // rows and columns past the edge repeat the last and are not stored
  int n[NT];
  const uint8_t* w[NT];
  const uint8_t* ws[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    n[j] = min(n0 + min(16 * j + c, cols - 1), N - 1);
    w[j] = p.wgt + uint32_t(n[j]) * rowbytes + 16 * g;
    ws[j] = p.wscales + n[j];
  }
  const uint8_t* a[MT];
  const uint8_t* as[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int m = min(16 * t + c, M - 1);
    a[t] = p.act + uint32_t(m) * rowbytes + 16 * g;
    as[t] = p.ascales + m;
  }
  f32x4 acc[NT][MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[j][t] = f32x4{0.f, 0.f, 0.f, 0.f};

  // TAIL: the run that K ends in. More than 16 rows ask for a run's operands one
  // run ahead (64x12288x12288 40.2 to 33.4 us); fewer have more workgroups a
  // compute unit instead, which the registers of a run ahead would halve
  // (1x3072x12288 7.0 to 8.6).
  constexpr int D = C::AHEAD ? 2 : 1;
  u32x4 wv[D][P][NT], av[D][P][MT];
  uint32_t wsv[D][P][NT], asv[D][P][MT];
  auto ask = [&]<bool TAIL>(int q, int s0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int s = s0 + i, kb = 4 * s + g;
      const bool in = !TAIL || kb < kb_all;   // blocks past K are zeros of scale one
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        wv[q][i][j] = in ? *reinterpret_cast<const u32x4*>(w[j] + 64 * s) : u32x4{0u, 0u, 0u, 0u};
        wsv[q][i][j] = in ? ws[j][uint32_t(kb) * uint32_t(N)] : 127u;
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        av[q][i][t] = in ? *reinterpret_cast<const u32x4*>(a[t] + 64 * s) : u32x4{0u, 0u, 0u, 0u};
        asv[q][i][t] = in ? as[t][uint32_t(kb) * uint32_t(M)] : 127u;
      }
    }
  };
  auto products = [&](int q) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[j][t] = mfma_fp4_16(wv[q][i][j], av[q][i][t], acc[j][t], wsv[q][i][j], asv[q][i][t]);
  };
  const int full = (K >> 7) / P;   // whole runs
  if constexpr (C::AHEAD) {
    int s = wave;
    if (s < full) ask.template operator()<false>(0, P * s);
#pragma unroll 1
    for (; s < full; s += 2 * W) {
      if (s + W < full) ask.template operator()<false>(1, P * (s + W));
      products(0);
      if (s + 2 * W < full) ask.template operator()<false>(0, P * (s + 2 * W));
      if (s + W < full) products(1);
    }
  } else {
#pragma unroll 1
    for (int s = wave; s < full; s += W) {
      ask.template operator()<false>(0, P * s);
      products(0);
    }
  }
  if (K % (128 * P) != 0 && full % W == wave) {
    ask.template operator()<true>(0, P * full);
    products(0);
  }
  // lane (c, g) of tile (j, t): columns n0 + 16 j + 4 g + e of row 16 t + c
  float wc[NT][4];
  bool large = false;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      wc[j][e] = p.wcscale[min(n0 + 16 * j + 4 * g + e, N - 1)];
      large |= !(fabsf(wc[j][e]) < 0x1p64f);
    }
  // A factor that is infinite, NaN or so large that a wave's part of a finite sum could
  // become infinite (parts of both signs, or none, would then add up to NaN): the
  // waves' sums meet without it and without the LoRA term. The same in every wave.
  const bool apart = __builtin_amdgcn_ballot_w64(large) != 0;
  if (!apart) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][t][e] *= wc[j][e];
  }

  // ranks r0 .. r0+31: lane (c, g) supplies ranks r0 + 8g .. +7 of column n
  // (A) and of row m (B)
  for (int r0 = 32 * wave; r0 < (apart ? 0 : R); r0 += 32 * W) {
    const int rr = r0 + 8 * g;
    u32x4 uv[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      uint16_t u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = rr + i < R ? p.lora_up[uint32_t(rr + i) * uint32_t(N) + uint32_t(n[j])] : 0;
      uv[j] = u32x4{bf16_pair(u[0], u[1]), bf16_pair(u[2], u[3]), bf16_pair(u[4], u[5]), bf16_pair(u[6], u[7])};
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const uint16_t* la = p.lora_act_in + uint32_t(min(16 * t + c, M - 1)) * uint32_t(R);
      uint16_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = rr + i < R ? la[rr + i] : 0;
      const u32x4 vv = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j][t] = mfma16<F16>(uv[j], vv, acc[j][t]);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int t = 0; t < MT; ++t) red[(wave * NT * MT + j * MT + t) * kWave + lane] = acc[j][t];
  __syncthreads();
  const int end = min(n0 + cols, N);
  for (int u = wave; u < NT * MT; u += W) {
    f32x4 y = red[u * kWave + lane];
#pragma unroll
    for (int q = 1; q < W; ++q) y += red[(q * NT * MT + u) * kWave + lane];
    const int m = 16 * (u % MT) + c;
    if (m >= M) continue;
    if (apart) {
      for (int e = 0; e < 4; ++e) {
        const int col = min(n0 + 16 * (u / MT) + 4 * g + e, N - 1);
        float v = y[e] * p.wcscale[col];
        for (int r = 0; r < R; ++r)
          v += widen<F16>(p.lora_act_in[uint32_t(m) * uint32_t(R) + uint32_t(r)]) *
               widen<F16>(p.lora_up[uint32_t(r) * uint32_t(N) + uint32_t(col)]);
        y[e] = v;
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int col = n0 + 16 * (u / MT) + 4 * g + e;
      if (col < end) p.out[uint32_t(m) * uint32_t(N) + uint32_t(col)] = narrow<F16>(y[e] + p.bias[col]);
    }
  }
}

static bool few_sizes_ok(int M, int N, int K, int R) {
  if (!(M >= 1 && M <= GEMM_MXFP4_FEW_MAX_M && N >= 1 && K >= 32 && K % 32 == 0 && R >= 0 && R <= GEMM_W4A4_MAX_R))
    return false;
  const int64_t lim = int64_t(1) << 31;
  const int64_t m = M, n = N, k = K, r = R;
  return m * k / 2 < lim && n * k / 2 < lim && m * n * 2 < lim && m * r * 2 < lim && r * n * 2 < lim;
}

struct FewKernel {
  const void* fn;
  int cols, threads;
};

template <bool F16, class C>
static FewKernel few_kernel() {
  return FewKernel{reinterpret_cast<const void*>(mx_few_kernel<F16, C>), C::COLS, C::THREADS};
}

template <bool F16>
static int mx_few_run(const uint8_t* act, const uint8_t* ascales, const uint8_t* wgt, const uint8_t* wscales,
                      const float* wcscale, const float* bias, const uint16_t* lora_act_in, const uint16_t* lora_up,
                      uint16_t* out, int M, int N, int K, int R, void* stream) {
  if (!few_sizes_ok(M, N, K, R)) return GEMM_W4A4_EINVAL;
  const int rc = check_call(CallArgs{act, ascales, wgt, wscales, wcscale, bias, lora_act_in, lora_up, out, M, N, K, R, stream}, 32);
  if (rc != GEMM_W4A4_OK) return rc;
  const int dev_rc = check_device();
  if (dev_rc != GEMM_W4A4_OK) return dev_rc;
  Params p{};
  p.act = act;
  p.ascales = ascales;
  p.wgt = wgt;
  p.wscales = wscales;
  p.wcscale = wcscale;
  p.bias = bias;
  p.lora_act_in = lora_act_in;
  p.lora_up = lora_up;
  p.out = out;
  p.M = M;
  p.N = N;
  p.K = K;
  p.R = R;
  // Tiling, measured (M x K x N, us). More than 16 rows: more columns a workgroup
  // where there are many, since each reads all activations, even though just past
  // a threshold that leaves half of the compute units without one (N = 4097 and 8193:
  // 129 workgroups; N = 12288 with 64 columns: 192 of 256 units): 32 for more than 4096 columns (24x3072x6144 7.4 against 8.4 with
  // 16, 64x3072x6144 10.3 and 15.5; 40x4096x4096 10.0 and 8.4), 64 for more than
  // 8192 (64x12288x12288 40.2 against 45.8, 30x12288x12288 25.1 and 30.6); 16
  // waves for most rows and 16 columns (64x12288x3072 19.4 against 22.4 with 8).
  // Up to 16 rows many workgroups a compute unit count for more: 16 columns
  // (1x12288x12288 15.0 against 18.5 with 32), runs of 2 steps (19.1 against 20.3).
  const bool wide = N > 16 * kNumCUs, widest = N > 32 * kNumCUs;
  const FewKernel k = M <= 16 ? few_kernel<F16, FewCfg<1, 1, 8, 2>>()
                    : M <= 32 ? (widest ? few_kernel<F16, FewCfg<2, 4, 8, 1>>()
                                 : wide ? few_kernel<F16, FewCfg<2, 2, 8, 1>>()
                                        : few_kernel<F16, FewCfg<2, 1, 8, 1>>())
                    : widest  ? few_kernel<F16, FewCfg<4, 4, 8, 1>>()
                    : wide    ? few_kernel<F16, FewCfg<4, 2, 8, 1>>()
                              : few_kernel<F16, FewCfg<4, 1, 16, 1>>();
  // Up to 32 rows and 16 columns a workgroup: fewer columns where that puts every
  // compute unit to work (16x12288x3072 12 columns 9.4 against 10.2 us,
  // 32x12288x1536 6 columns 11.1 against 12.3, 1x12288x1001 4 columns 5.0 against 6.3;
  // 40x3072x2500 7.1 against 6.2, the activations being read more often).
  const int cols = k.cols > 16 || M > 32 ? k.cols : std::min(16, std::max(4, (N + kNumCUs - 1) / kNumCUs));
  void* args[] = {&p, const_cast<int*>(&cols)};
  const hipError_t e = hipLaunchKernel(k.fn, dim3((N + cols - 1) / cols), dim3(k.threads), args, 0,
                                       static_cast<hipStream_t>(stream));
  return e == hipSuccess ? GEMM_W4A4_OK : GEMM_W4A4_ELAUNCH;
}

}  // namespace w4a4

extern "C" int gemm_mxfp4_few(const uint8_t* act, const uint8_t* ascales, const uint8_t* wgt, const uint8_t* wscales,
                              const float* wcscale, const float* bias, const uint16_t* lora_act_in,
                              const uint16_t* lora_up, uint16_t* out, int M, int N, int K, int R, void* stream) {
  return w4a4::mx_few_run<false>(act, ascales, wgt, wscales, wcscale, bias, lora_act_in, lora_up, out, M, N, K, R, stream);
}

extern "C" int gemm_mxfp4_few_f16(const uint8_t* act, const uint8_t* ascales, const uint8_t* wgt,
                                  const uint8_t* wscales, const float* wcscale, const float* bias,
                                  const uint16_t* lora_act_in, const uint16_t* lora_up, uint16_t* out, int M, int N,
                                  int K, int R, void* stream) {
  return w4a4::mx_few_run<true>(act, ascales, wgt, wscales, wcscale, bias, lora_act_in, lora_up, out, M, N, K, R, stream);
}
