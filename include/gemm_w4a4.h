/*
 * gemm_w4a4.h — C ABI of the fused NVFP4 W4A4 GEMM for AMD Instinct MI355X (gfx950).
 *
 * The operation (section 2 of the SVDQuant W4A4 on Blackwell page,
 * "Blackwell 上的 SVDQuant W4A4 算子实现"):
 *
 *     y[m,n] = wcscale[n] * sum_k A[m,k] * W[n,k] + bias[n]
 *              + sum_r lora_act_in[m,r] * lora_up[r,n]
 *
 * where A and W are NVFP4: E2M1 codes (two per byte) times one FP8-E4M3 block
 * scale per 16 consecutive k (same page, section 3.1: single-level block
 * scaling, no per-tensor factor). The per-column affine is the page's
 * section 6.6 epilogue; the LoRA residual is added after the wcscale product,
 * as the section 2 formula writes it. The result is rounded to bfloat16
 * (nearest, ties to even).
 *
 * Layouts: every tensor is dense and row-major, without padding or strides.
 *   act          uint8   [M, K/2]   byte j of row m holds k = 2j (low nibble)
 *                                   and k = 2j+1 (high nibble)
 *   ascales      uint8   [K/16, M]  OCP E4M3FN bytes; scale of (m,k) is
 *                                   ascales[k/16][m]
 *   wgt          uint8   [N, K/2]   as act, one row per output column n
 *   wscales      uint8   [K/16, N]
 *   wcscale      float   [N]
 *   bias         float   [N]
 *   lora_act_in  uint16  [M, R]     bfloat16 bit patterns
 *   lora_up      uint16  [R, N]     bfloat16 bit patterns
 *   out          uint16  [M, N]     bfloat16 bit patterns (written)
 *
 * Ownership: every tensor pointer is a device pointer owned by the caller.
 * The library allocates and frees nothing, keeps no per-call state, and never
 * synchronizes: a successful call only enqueues work on `stream`.
 */
#ifndef GEMM_W4A4_H
#define GEMM_W4A4_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. Validation runs before any HIP call, so on a negative code
 * nothing has been enqueued. No C++ exception crosses this boundary. */
enum {
  GEMM_W4A4_OK = 0,
  GEMM_W4A4_EINVAL = -1,      /* bad size (M<1, N<1, K<16, K%16, R<0, R>GEMM_W4A4_MAX_R,
                                 or any tensor of 2^31 bytes or more) or a required
                                 NULL pointer */
  GEMM_W4A4_EALIGN = -2,      /* act/wgt not 16-byte aligned, wcscale/bias not 4-byte,
                                 lora/out not 2-byte aligned; other entry points: as stated
                                 with them */
  GEMM_W4A4_ELAUNCH = -3,     /* the HIP launch itself failed */
  GEMM_W4A4_EOVERLAP = -4,    /* an output overlaps an input or another output */
  GEMM_W4A4_EDEVICE = -5,     /* the current device is not gfx950 */
  GEMM_W4A4_ENOMEM = -6,      /* quantize_w4a4_act could not allocate its scratch buffer */
  GEMM_W4A4_ESCRATCH = -7     /* the call needs more scratch than quantize_w4a4_act_noalloc's
                                 fixed array (QUANTIZE_W4A4_NOALLOC_SCRATCH_BYTES), or than
                                 the workspace that the caller gave */
};

#define GEMM_W4A4_MAX_R 1024

/*
 * gemm_w4a4 — enqueue y = scaled_mma(act, wgt) * wcscale + bias + lora_act_in @ lora_up.
 *
 * act, ascales, wgt, wscales, wcscale, bias, out: required (non-NULL).
 * lora_act_in, lora_up: may be NULL only when R == 0 (no LoRA term).
 * M, N >= 1; K >= 16 with K % 16 == 0; 0 <= R <= GEMM_W4A4_MAX_R.
 * stream: a hipStream_t passed as void*; NULL selects the null stream.
 *
 * Every out[m][n] with m < M, n < N is overwritten; nothing else is written
 * and no input is modified. A plan whose tail runs its K in slices (see
 * gemm_w4a4_plan_t) first keeps the slices' float32 sums in out's first
 * rows; every element holds its result once the call's work on the stream
 * has finished. Results are deterministic: the same inputs give the same
 * bytes on every call (no atomics; slices are added in a fixed order). E4M3 NaN scale bytes
 * (0x7F, 0xFF) propagate NaN into every output their block touches.
 * Returns GEMM_W4A4_OK or one of the negative codes above.
 */
int gemm_w4a4(const uint8_t* act, const uint8_t* ascales,
              const uint8_t* wgt, const uint8_t* wscales,
              const float* wcscale, const float* bias,
              const uint16_t* lora_act_in, const uint16_t* lora_up,
              uint16_t* out, int M, int N, int K, int R, void* stream);

/*
 * gemm_w4a4_f16 — the same operation with the LoRA operands and the output in
 * IEEE binary16 instead of bfloat16 (the SVDQuant page runs its operator with
 * either 16-bit type, "c_dtype", sections 6.6 and 9.2):
 *   lora_act_in  uint16  [M, R]     binary16 bit patterns
 *   lora_up      uint16  [R, N]     binary16 bit patterns
 *   out          uint16  [M, N]     binary16 bit patterns (written), rounded to
 *                                   nearest even; magnitudes of 65520 and above
 *                                   become infinity
 * Every other argument, rule, alignment and return code is gemm_w4a4's.
 */
int gemm_w4a4_f16(const uint8_t* act, const uint8_t* ascales,
                  const uint8_t* wgt, const uint8_t* wscales,
                  const float* wcscale, const float* bias,
                  const uint16_t* lora_act_in, const uint16_t* lora_up,
                  uint16_t* out, int M, int N, int K, int R, void* stream);

/*
 * gemm_mxfp4 / gemm_mxfp4_f16 — the same operator with MXFP4 operands: E2M1
 * codes as above, but one UE8M0 scale per 32 consecutive k (value
 * 2^(b - 127), 0xFF = NaN; the DeepGEMM FP4 indexer page, "Step 0", pairs
 * E2M1 data with this block scale, applied by the matrix unit itself):
 *   ascales      uint8   [K/32, M]  UE8M0 bytes; scale of (m,k) is ascales[k/32][m]
 *   wscales      uint8   [K/32, N]
 * K >= 32 with K % 32 == 0; everything else (layouts, LoRA, affine, output
 * type bf16 or binary16, alignments, return codes) is gemm_w4a4's /
 * gemm_w4a4_f16's. No decode happens on the GPU: gfx950's scaled FP4 MFMA
 * consumes the packed bytes and the scale bytes as they are.
 */
int gemm_mxfp4(const uint8_t* act, const uint8_t* ascales,
               const uint8_t* wgt, const uint8_t* wscales,
               const float* wcscale, const float* bias,
               const uint16_t* lora_act_in, const uint16_t* lora_up,
               uint16_t* out, int M, int N, int K, int R, void* stream);
int gemm_mxfp4_f16(const uint8_t* act, const uint8_t* ascales,
                   const uint8_t* wgt, const uint8_t* wscales,
                   const float* wcscale, const float* bias,
                   const uint16_t* lora_act_in, const uint16_t* lora_up,
                   uint16_t* out, int M, int N, int K, int R, void* stream);

/*
 * Launch plan chosen by the solver for one problem size: which compiled tile
 * instance runs, and how that instance's LDS budget was solved — the ring
 * depth (stages of K in flight) and where the epilogue's first LoRA chunk and
 * per-column factors live — with the registers its code object uses. The
 * SVDQuant W4A4 on Blackwell page (section 7) shows what a miscounted buffer
 * in such a budget does: a silently shallower pipeline. Here the kernels carve
 * LDS from the same solved budget that these fields report. Pure host
 * arithmetic and table lookups (no HIP call), so it also runs without a GPU.
 */
typedef struct {
  int variant;        /* index of the compiled kernel instance */
  int block_m;        /* output rows per workgroup tile */
  int block_n;        /* output columns per workgroup tile */
  int block_k;        /* k per pipeline stage */
  int stages;         /* ring depth: LDS stages of K in flight, set by the budget solve */
  int waves_m;        /* wave grid inside a workgroup */
  int waves_n;
  int threads;        /* threads per workgroup */
  int lds_bytes;      /* LDS the instance uses: lds_ring_bytes + lds_side_bytes */
  int lds_stage_bytes;/* bytes of one ring stage (packed operands and their scales) */
  int lds_limit;      /* LDS available to one workgroup on gfx950 */
  int tiles_m;
  int tiles_n;
  int grid;           /* workgroups launched */
  int k_stages;       /* pipeline iterations over K */
  int lora_steps;     /* 16-deep LoRA MFMA steps (ceil(R/16)) */
  int occupancy;      /* workgroups of this instance per compute unit (LDS share = lds_limit / occupancy) */
  int policy;         /* budget solve: 0 deepest ring first, 1 whole side region first */
  int lora_place;     /* where the first 32 LoRA ranks and wcscale/bias wait for the epilogue:
                         0 nowhere: loaded by the epilogue and staged through the drained ring;
                         1 side region with wcscale/bias and the lora_act_in rows (lora_up in
                           registers held through the K-loop);
                         2 side region with the lora_up rows too.
                         Ranks past 32 always go through the drained ring. */
  int lds_ring_bytes; /* stages * lds_stage_bytes */
  int lds_side_bytes; /* side region beside the ring (0 when lora_place == 0) */
  int flavour;        /* kernel flavour the shape gets when every tensor is 16-byte aligned:
                         0 general, 1 fast, 2 fast with act-scale windows; -1 in variant_info */
  int vgprs;          /* vector registers a lane of that kernel (bf16 output) holds, architectural and
                         accumulation together, from its code object; -1 if unknown */
  int agprs;          /* of which accumulation registers */
  int sgprs;          /* scalar registers, same kernel */
  int regs_limit;     /* VGPR + AGPR a lane may hold at this occupancy (512 per SIMD lane, shared) */
  int k_groups;       /* waves sharing each wave tile, splitting every stage's k-steps between them
                         (threads = 64 * waves_m * waves_n * k_groups) */
  /* A split plan (the solver's choice only, tail_variant >= 0): the fields
   * above describe a first launch over the first M - tail_rows rows (whole
   * tile rows: tiles_m * block_m of them), and a second launch of instance
   * tail_variant, whose block_m divides the first one's, covers the last
   * tail_rows rows in tail_grid workgroups. Both run on the call's stream, in order, on
   * disjoint output rows. Not split: tail_variant -1, the others 0. */
  int tail_variant;
  int tail_rows;
  int tail_block_m;
  int tail_block_n;
  int tail_grid;
  /* K slices of the tail launch (1: it runs whole). Above 1, its workgroups
   * (tail_grid of them, counted with the slices) each run one slice of K and
   * write float32 sums into the first tail_splits * tail_rows * 2 rows of out,
   * rows the first launch writes later; a reduction launch adds the slices
   * into the last tail_rows rows. The three launches run on the call's stream
   * in the order slices, reduction, first launch; the call allocates nothing.
   * When the call's pointers do not allow the fast flavour the tail runs
   * whole, after the first launch. */
  int tail_splits;
} gemm_w4a4_plan_t;

/* Fill *plan for (M, N, K, R). Returns GEMM_W4A4_OK or GEMM_W4A4_EINVAL
 * (same size rules as gemm_w4a4; plan may not be NULL). */
int gemm_w4a4_plan(int M, int N, int K, int R, gemm_w4a4_plan_t* plan);

/* Number of compiled kernel instances, and the plan fields fixed by instance
 * `variant` (problem-size fields are zero). Returns GEMM_W4A4_EINVAL for an
 * unknown index. Used to check the solver against the compiled code objects. */
int gemm_w4a4_num_variants(void);
int gemm_w4a4_variant_info(int variant, gemm_w4a4_plan_t* plan);

/* The same three for the MXFP4 kernels (K % 32 == 0). */
int gemm_mxfp4_plan(int M, int N, int K, int R, gemm_w4a4_plan_t* plan);
int gemm_mxfp4_num_variants(void);
int gemm_mxfp4_variant_info(int variant, gemm_w4a4_plan_t* plan);

/* Operand formats and output types of gemm_w4a4_run / gemm_w4a4_plan_variant. */
enum { GEMM_W4A4_FMT_NVFP4 = 0, GEMM_W4A4_FMT_MXFP4 = 1 };

/*
 * gemm_w4a4_run — the same operator with every choice explicit, for callers
 * that pick the tiling per shape themselves (the solver's choice is a model;
 * this runs any compiled instance):
 *   format   GEMM_W4A4_FMT_NVFP4 (as gemm_w4a4) or GEMM_W4A4_FMT_MXFP4 (as gemm_mxfp4)
 *   out_f16  0: LoRA operands and output bfloat16; 1: binary16 (as the _f16 calls)
 *   variant  a compiled instance of that format, 0 <= variant < its
 *            num_variants, or -1 for the solver's choice
 * Every other argument, layout, rule and return code is the named entry
 * point's; an unknown format or variant returns GEMM_W4A4_EINVAL.
 */
int gemm_w4a4_run(int format, int out_f16, int variant,
                  const uint8_t* act, const uint8_t* ascales,
                  const uint8_t* wgt, const uint8_t* wscales,
                  const float* wcscale, const float* bias,
                  const uint16_t* lora_act_in, const uint16_t* lora_up,
                  uint16_t* out, int M, int N, int K, int R, void* stream);

/* The plan gemm_w4a4_run would follow for (format, variant, M, N, K, R);
 * variant -1 gives the solver's choice (the format's _plan call). */
int gemm_w4a4_plan_variant(int format, int variant, int M, int N, int K, int R,
                           gemm_w4a4_plan_t* plan);

/*
 * quantize_w4a4_act — the other half of an SVDQuant W4A4 layer (the SVDQuant
 * W4A4 on Blackwell page, section 1, calls gemm_w4a4 the compute-bound half):
 * from the bf16 activations x, the NVFP4 operand gemm_w4a4 consumes and the
 * rank-R LoRA input, in one pass over x.
 *
 *   x            uint16  [M, K]     bfloat16 bit patterns (read)
 *   lora_down    uint16  [R, K]     bfloat16 bit patterns, one rank per row (read);
 *                                   may be NULL iff R == 0
 *   act          uint8   [M, K/2]   written: two E2M1 codes per byte, low nibble = even k
 *   ascales      uint8   [K/16, M]  written: OCP E4M3FN scale of (m, k) at [k/16][m]
 *   lora_act_in  uint16  [M, R]     written: bfloat16 bits of sum_k x[m,k] * lora_down[r,k]
 *                                   (float32 accumulation, rounded to nearest even);
 *                                   may be NULL iff R == 0
 *
 * The pages fix these layouts (section 2; single-level scaling, section 3.1)
 * but not how a block's scale is chosen or its codes rounded. This library's
 * reading, per row and block of 16 consecutive k:
 *   - a block holding a NaN or an infinity gets scale byte 0x7F (NaN) and zero codes;
 *   - otherwise scale = E4M3FN nearest-even of max|x| / 6, saturating at 448;
 *   - code = sign bit of x | E2M1 magnitude of |x| / scale, nearest with ties
 *     to the even code, saturating at 6; a zero scale keeps only the sign bit.
 * Every rounding decision is exact (the same as on the real numbers).
 *
 * M >= 1; K >= 16 with K % 16 == 0; 0 <= R <= QUANTIZE_W4A4_MAX_R; every
 * tensor below 2^31 bytes. Alignment: x and lora_down 16 bytes, act 8,
 * lora_act_in 2. No output may overlap an input or another output
 * (GEMM_W4A4_EOVERLAP). Device pointers owned by the caller; the work is
 * enqueued on `stream` (one launch, or two when a 128-row instance splits K
 * with R > 0: the second adds the slices' partial sums; quantize_w4a4_act_plan
 * says which).
 *
 * Scratch: when few rows meet a long K, K is split over workgroups and
 * float32 partial sums go to a scratch buffer that the library allocates per
 * device and stream on the first call on that stream that needs it (or more
 * than it holds) and keeps until the process ends. That call allocates,
 * zeroes the buffer and synchronises the device before it enqueues anything
 * (GEMM_W4A4_ENOMEM if the allocation fails); every other call allocates and
 * synchronises nothing. Calls on different streams use different buffers, so
 * they may overlap. quantize_w4a4_act_noalloc never allocates. Other return
 * codes as for gemm_w4a4.
 */
#define QUANTIZE_W4A4_MAX_R 128
int quantize_w4a4_act(const uint16_t* x, const uint16_t* lora_down, uint8_t* act,
                      uint8_t* ascales, uint16_t* lora_act_in, int M, int K, int R,
                      void* stream);

/* The launch quantize_w4a4_act would make for (M, K, R): host only, nothing
 * enqueued. The instance follows the rank and, at R <= 32, the shape; K is
 * split over workgroups so that all row blocks' workgroups spread over the
 * compute units in one round (the device's count; 256 when no device is
 * current). */
typedef struct {
  int variant;          /* compiled producer instance */
  int wide;             /* 1: the waves of a workgroup share each span (lora_down tile in LDS) */
  int rank_tiles;       /* 16-rank tiles the instance covers (R <= 16 * rank_tiles) */
  int rows;             /* rows of x per workgroup */
  int threads;          /* threads per workgroup */
  int lds_bytes;        /* LDS per workgroup */
  int row_blocks;       /* ceil(M / rows) */
  int k_slices;         /* workgroups sharing a row block's K */
  int spans_per_slice;  /* 128-wide spans of K per slice */
  int grid;             /* workgroups of the first launch (row_blocks * k_slices) */
  int launches;         /* 2 when a wide kernel's slices are added by a second launch */
  long long scratch_bytes;  /* scratch the call needs (arrival counters + partial sums); 0 unsplit */
} quantize_w4a4_plan_t;

/* Fill *plan. Returns GEMM_W4A4_OK, or GEMM_W4A4_EINVAL for sizes
 * quantize_w4a4_act rejects or a NULL plan. */
int quantize_w4a4_act_plan(int M, int K, int R, quantize_w4a4_plan_t* plan);

/*
 * quantize_w4a4_act_noalloc — quantize_w4a4_act for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc. Same arguments, kernels and results as
 * quantize_w4a4_act; it calls no allocating routine.
 *
 * When K is split over several workgroups (few rows, long K), the kernels
 * keep float32 partial sums (and, for R <= 32, one arrival counter per 16
 * rows) in scratch memory; quantize_w4a4_act allocates that buffer on first
 * need, this entry
 * point uses a fixed device array of QUANTIZE_W4A4_NOALLOC_SCRATCH_BYTES
 * (4 KiB of counters + 16 MiB of partial sums) that each GPU holds until the
 * process ends. Both entry points split K only as far as 16 MiB of partial
 * sums allow; a call that would still need more returns GEMM_W4A4_ESCRATCH
 * with nothing enqueued. The counters are zero at load and every completed call
 * returns them to zero.
 *
 * Every call on one GPU shares that GPU's array: calls that overlap on one
 * GPU (concurrent streams, or host threads) race on it and must be ordered
 * by the caller. Return codes as for quantize_w4a4_act, plus
 * GEMM_W4A4_ESCRATCH.
 */
#define QUANTIZE_W4A4_NOALLOC_SCRATCH_BYTES (4096 + (16 << 20))
int quantize_w4a4_act_noalloc(const uint16_t* x, const uint16_t* lora_down, uint8_t* act,
                              uint8_t* ascales, uint16_t* lora_act_in, int M, int K, int R,
                              void* stream);

/*
 * quantize_mxfp4_act / quantize_mxfp4_act_f16 — the producer of gemm_mxfp4's
 * operand: 16-bit activations x to E2M1 codes and UE8M0 block scales, and the
 * rank-R LoRA input, in one pass over x. With R = 0 it also lays out weights
 * (rows n of wgt [N, K] in place of rows m).
 *
 *   x            uint16  [M, K]     bfloat16 (_f16: binary16) bit patterns (read)
 *   lora_down    uint16  [R, K]     same type, one rank per row (read); may be NULL iff R == 0
 *   act          uint8   [M, K/2]   written: two E2M1 codes per byte, low nibble = even k
 *   ascales      uint8   [K/32, M]  written: UE8M0 scale of (m, k) at [k/32][m]
 *   lora_act_in  uint16  [M, R]     written, x's type: sum_k x[m,k] * lora_down[r,k]
 *                                   (float32 accumulation, rounded to nearest even);
 *                                   may be NULL iff R == 0
 *
 * Per row and block of 32 consecutive k, the microscaling formats' rule: the
 * scale is 2^(floor(log2 max|x|) - 2), so that the largest magnitude lands in
 * [4, 8) and saturates at 6, the largest E2M1 value; the scale byte is that
 * exponent + 127, at least 0; a code is the sign of x and the E2M1 magnitude
 * nearest |x| / scale, ties to the even code (exact: the division is by a
 * power of two). A block with a NaN or an infinity gets byte 0xFF and zero
 * codes; a block of zeros byte 0.
 *
 * M >= 1; K >= 32 with K % 32 == 0; 0 <= R <= QUANTIZE_W4A4_MAX_R; every
 * tensor below 2^31 bytes. Alignment: x, lora_down, act 16 bytes, lora_act_in
 * 2, workspace 16. No output may overlap an input or another output.
 *
 * workspace: quantize_mxfp4_workspace(M, K, R) bytes of device memory that
 * nothing else uses until the call's work on `stream` has finished (0: NULL is
 * fine). Fewer: GEMM_W4A4_ESCRATCH. The call allocates and synchronises
 * nothing. Results do not depend on what the workspace holds.
 */
int quantize_mxfp4_act(const uint16_t* x, const uint16_t* lora_down, uint8_t* act, uint8_t* ascales,
                       uint16_t* lora_act_in, int M, int K, int R, void* workspace,
                       int64_t workspace_bytes, void* stream);
int quantize_mxfp4_act_f16(const uint16_t* x, const uint16_t* lora_down, uint8_t* act, uint8_t* ascales,
                           uint16_t* lora_act_in, int M, int K, int R, void* workspace,
                           int64_t workspace_bytes, void* stream);
/* Workspace bytes for (M, K, R) on the current device, or GEMM_W4A4_EINVAL (host only). */
int64_t quantize_mxfp4_workspace(int M, int K, int R);

/*
 * gemm_mxfp4_few / gemm_mxfp4_few_f16 — gemm_mxfp4's operation for few rows
 * (1 <= M <= GEMM_MXFP4_FEW_MAX_M): the weights are streamed once past all
 * rows instead of being tiled for many. Arguments, layouts, sizes, alignments
 * and return codes are gemm_mxfp4's / gemm_mxfp4_f16's; the results agree
 * with theirs up to the order of the float32 sums, not byte for byte. No
 * workspace; deterministic. The faster of the two up to 64 rows, or as fast, but
 * for 16 rows or more, M % 4 == 0, N % 8 == 0, K % 128 == 0, with so many columns
 * that gemm_mxfp4's tiles fill the chip (64 x 3072 x 18432: 27.6 us against 15.5; 64 x 12288 x 12288 37.4 and 42.4,
 * 33 x 3072 x 12288 13.5 and 36.3).
 */
#define GEMM_MXFP4_FEW_MAX_M 64
int gemm_mxfp4_few(const uint8_t* act, const uint8_t* ascales,
                   const uint8_t* wgt, const uint8_t* wscales,
                   const float* wcscale, const float* bias,
                   const uint16_t* lora_act_in, const uint16_t* lora_up,
                   uint16_t* out, int M, int N, int K, int R, void* stream);
int gemm_mxfp4_few_f16(const uint8_t* act, const uint8_t* ascales,
                       const uint8_t* wgt, const uint8_t* wscales,
                       const float* wcscale, const float* bias,
                       const uint16_t* lora_act_in, const uint16_t* lora_up,
                       uint16_t* out, int M, int N, int K, int R, void* stream);

/*
 * rotary_axes — rotary positions over several axes (time, height, width, ...)
 * applied to heads x [batch, tokens, heads, head_dim]. The P pairs of a head
 * (P = the sum of sections, 2P <= head_dim) are dealt to the axes in order,
 * sections[a] pairs to axis a. Pair j on axis a turns by
 *
 *     t = positions[batch, token, a] * inv_freq[j]        (radians)
 *     (u, w) -> (u cos t - w sin t, u sin t + w cos t)
 *
 * where (u, w) are elements (2j, 2j+1) when interleaved, else (j, j + P).
 * Elements from 2P on are copied. `inverse` turns by -t, which
 * takes the gradient of out to that of x: a rotation's transpose is the opposite
 * rotation. The angle is reduced
 * to one turn in float64, so it holds at every position (within 2^-22 turns for
 * frequencies up to 1); rotation in float32, rounded once.
 *
 * Strides are in elements; the last dimension is dense; positions' axes are
 * dense (stride 1), with a stride per batch (0: shared) and per token. out may
 * be x itself with the same strides (in place); any other overlap, or
 * overlap with positions or inv_freq, is GEMM_W4A4_EOVERLAP. Strides are
 * non-negative and out's may not make two elements share memory
 * (GEMM_W4A4_EINVAL). x and out 2-byte, positions and inv_freq 4-byte aligned;
 * interleaved needs an even head_dim (GEMM_W4A4_EINVAL) and pairs that start on
 * 4 bytes (GEMM_W4A4_EALIGN).
 * At most 65535 batches, head_dim up to ROTARY_MAX_HEAD_DIM (GEMM_W4A4_EINVAL).
 * batch, tokens and heads may be 0: nothing is enqueued.
 */
#define ROTARY_AXES_MAX 4
#define ROTARY_MAX_HEAD_DIM 256
typedef struct {
  const void* x;             /* 16-bit type, see f16 */
  void* out;
  const int32_t* positions;
  const float* inv_freq;     /* [P] */
  int batch, tokens, heads, head_dim;
  int axes;                  /* 1 .. ROTARY_AXES_MAX */
  int sections[ROTARY_AXES_MAX];   /* pairs per axis, each >= 0 */
  int64_t x_stride[3];       /* batch, token, head */
  int64_t out_stride[3];
  int64_t pos_stride[2];     /* batch, token */
  int interleaved, inverse;
  int f16;                   /* 0: bfloat16, 1: binary16 */
} rotary_axes_t;
int rotary_axes(const rotary_axes_t* args, void* stream);

/*
 * cross_attention — attention of q [batch, q_len, q_heads, head_dim] to keys
 * and values [batch, kv_len, kv_heads, head_dim] of another length:
 *
 *     out[b, i, h] = sum_j softmax_j(scale * q[b,i,h] . k[b,j,g]) v[b,j,g],
 *     g = h / (q_heads / kv_heads),  j < kv_lens[b]
 *
 *   kv_lens   int32 [batch] on the device, or NULL: kv_len keys everywhere.
 *             Values outside 0 .. kv_len are taken as the nearest of the two.
 *             Keys and values from kv_lens[b] on are never read.
 *   lse       float [batch, q_heads, q_len], written when not NULL: the natural
 *             log of the sum of exp(scale * q . k) (joins attentions over
 *             parts of the keys)
 * A row without keys gives out 0 and lse -inf. Scores, softmax statistics and
 * sums are float32; the weights exp(...) are rounded to the 16-bit type for
 * the product with v.
 *
 * scale: positive, at most 1e30. head_dim: a multiple of 8, 8 ..
 * CROSS_ATTENTION_MAX_HEAD_DIM; q_heads a multiple of kv_heads; q_len * q_heads
 * and kv_len at most 2^31 - CROSS_ATTENTION_PAST_END, batch * q_len * q_heads below
 * 2^31, batch * kv_heads below 2^23. Strides in elements, multiples of 8 (a dimension of
 * size 1 excepted), non-negative, k's and v's token strides below 2^23; the
 * last dimension is dense; all four tensors 16-byte aligned. q, k and v may
 * repeat memory (stride 0); out may not (GEMM_W4A4_EINVAL) and out and lse may
 * overlap nothing else (GEMM_W4A4_EOVERLAP). batch, q_len or q_heads 0:
 * nothing is enqueued; kv_len 0: k and v may be NULL.
 *
 * workspace: cross_attention_workspace bytes of device memory, 16-byte
 * aligned, that nothing else uses until the call's work on `stream` has
 * finished (0: NULL is fine). Fewer: GEMM_W4A4_ESCRATCH. Few rows split the
 * keys over workgroups and join the parts from there in a second launch, in a
 * fixed order. Deterministic; no allocation, no synchronisation.
 */
#define CROSS_ATTENTION_MAX_HEAD_DIM 128
#define CROSS_ATTENTION_PAST_END 1024
typedef struct {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;
  const int32_t* kv_lens;
  int batch, q_len, kv_len, q_heads, kv_heads, head_dim;
  int64_t q_stride[3];       /* batch, token, head */
  int64_t k_stride[3];
  int64_t v_stride[3];
  int64_t out_stride[3];
  float scale;
  int f16;                   /* 0: bfloat16, 1: binary16 */
  void* workspace;
  int64_t workspace_bytes;
} cross_attention_t;
int cross_attention(const cross_attention_t* args, void* stream);
/* Workspace bytes of this call on the current device (sizes and strides only; no
 * pointer is read), or GEMM_W4A4_EINVAL (host only). */
int64_t cross_attention_workspace(const cross_attention_t* args);

/*
 * block_norm — the norms after and before a block with its gate and residual in
 * between, on rows x and y [batch, tokens, width]:
 *
 *     z        = post_norm ? norm(y) * post_weight : y
 *     residual = residual_scale * x + gate * z
 *     out      = (norm(residual) * weight + bias) * (1 + scale) + shift
 *
 * norm(v) is (v - mean) / sqrt(var + eps) over the row (layer; var the mean of
 * the squared differences) or v / sqrt(mean of v^2 + eps). Without y, out is the norm of
 * x; residual, gate and post_norm are then not given and residual_scale is 1
 * (GEMM_W4A4_EINVAL). gate, scale, shift, weight, bias and post_weight may
 * each be NULL: left out. residual may be NULL: not written.
 *
 * All float32 from the 16-bit inputs to the two results, each rounded once: out
 * follows from the residual as it was before its rounding. Rows whose squares
 * pass float32's range have the result that they have in exact arithmetic; a row
 * with an infinity or a NaN has NaN as torch's would.
 *
 * width 1 .. BLOCK_NORM_MAX_WIDTH, odd ones too; batch * tokens below 2^31; eps 1e-12 .. 1;
 * residual_scale finite. Strides in elements, non-negative, the last dimension dense;
 * all tensors 2-byte aligned. gate, scale and shift have strides of their own
 * (0: one vector for the batch or for all tokens) and may be slices of one
 * tensor. out and residual may not make two rows share memory; each may be x
 * or y itself with the same strides (in place); otherwise the memory from its first to
 * its last element may hold nothing of an input or of the other
 * (GEMM_W4A4_EOVERLAP). batch or tokens 0: nothing is enqueued.
 * No workspace; deterministic.
 */
#define BLOCK_NORM_MAX_WIDTH 16384
typedef struct {
  const void* x;             /* 16-bit type, see f16 */
  const void* y;
  const void* gate;
  const void* scale;
  const void* shift;
  const void* weight;        /* [width], as bias and post_weight */
  const void* bias;
  const void* post_weight;
  void* out;
  void* residual;
  int batch, tokens, width;
  int64_t x_stride[2];       /* batch, token */
  int64_t y_stride[2];
  int64_t gate_stride[2];
  int64_t scale_stride[2];
  int64_t shift_stride[2];
  int64_t out_stride[2];
  int64_t residual_stride[2];
  float residual_scale, eps;
  int layer;                 /* 1: the layer norm, 0: without the mean */
  int post_norm;
  int f16;                   /* 0: bfloat16, 1: binary16 */
} block_norm_t;
int block_norm(const block_norm_t* args, void* stream);

/*
 * lora_adapters — low-rank adapters of many requests beside a projection that they
 * share: for every row m with adapter a = adapter[m],
 *
 *     out[m] = y[m] + scaling[a] * (x[m] @ down[a]^T) @ up[a]
 *
 *   x        16-bit  [rows, K]            the projection's input
 *   y        16-bit  [rows, N]            its result
 *   down     16-bit  [adapters, rank, K]  dense, one rank per row
 *   up       16-bit  [adapters, rank, N]  dense, likewise
 *   adapter  int32   [rows] on the device; outside 0 .. adapters - 1: none, out[m] = y[m]
 *   scaling  float   [adapters] on the device, or NULL: 1
 *   ranks    int32   [adapters] on the device, or NULL: rank for all. Rows of down and up
 *                    from ranks[a] on are not used; values outside 0 .. rank are
 *                    taken as the nearest of the two
 *
 * One 16-bit type (f16). Sums in float32; x @ down^T stays in float32 (its product
 * with up in two 16-bit parts); one rounding, to out. Rows may lie in any
 * order; rows of a request, or of requests with one adapter, beside each other share its reads.
 *
 * rows up to LORA_ADAPTERS_MAX_ROWS; rank 1 .. LORA_ADAPTERS_MAX_RANK; K a multiple
 * of 8; K and N up to 2^30; any N. Row strides in elements, not negative, x's a multiple of 8; x and
 * down 16-byte, y, up and out 2-byte, the others 4-byte aligned. out may be y itself
 * with the same stride (in place); it may overlap nothing else, and its rows not each
 * other (GEMM_W4A4_EINVAL). rows 0: nothing is enqueued.
 *
 * workspace: lora_adapters_workspace bytes, 16-byte aligned, that nothing else uses
 * until the call's work on `stream` has finished. Fewer: GEMM_W4A4_ESCRATCH. Results do not
 * depend on what it holds. Deterministic; no allocation, no synchronisation.
 */
#define LORA_ADAPTERS_MAX_RANK 128
#define LORA_ADAPTERS_MAX_ROWS 3145728
typedef struct {
  const void* x;             /* 16-bit type, see f16 */
  const void* y;
  const void* down;
  const void* up;
  void* out;
  const int32_t* adapter;
  const float* scaling;
  const int32_t* ranks;
  int rows, K, N, adapters, rank;
  int64_t x_stride, y_stride, out_stride;   /* of rows */
  int f16;                   /* 0: bfloat16, 1: binary16 */
  void* workspace;
  int64_t workspace_bytes;
} lora_adapters_t;
int lora_adapters(const lora_adapters_t* args, void* stream);
/* Workspace bytes of this call (sizes only; no pointer is read), or GEMM_W4A4_EINVAL (host only). */
int64_t lora_adapters_workspace(const lora_adapters_t* args);

/*
 * cache_append — keys and values of new tokens, k and v [tokens, heads,
 * head_dim], into a paged cache, k_cache and v_cache [pages, page_size, heads,
 * head_dim]: token t goes to place slots[t] % page_size of page slots[t] / page_size.
 * Slots outside 0 .. pages * page_size - 1 are left out (padding: -1). The slots of
 * a call's tokens must differ from each other: of two tokens with one slot either may stay, or
 * a part of each. Nothing else of the cache changes.
 *
 * tokens up to 2^30; head_dim a multiple of 8, 8 .. CROSS_ATTENTION_MAX_HEAD_DIM; fewer than
 * 2^20 heads; pages * page_size below 2^31. Strides in elements, multiples of 8
 * (a dimension of size 1 excepted), non-negative, the last dimension dense; tensors 16-byte,
 * slots 8-byte aligned. k and v may repeat memory; a cache may not, and may overlap nothing
 * else. Both caches may lie in one buffer (a page of the one beside a page of the
 * other) with the same strides. tokens or pages 0: nothing is enqueued.
 */
typedef struct {
  const void* k;             /* 16-bit values of any type */
  const void* v;
  void* k_cache;
  void* v_cache;
  const int64_t* slots;      /* [tokens] on the device */
  int tokens, heads, head_dim, pages, page_size;
  int64_t k_stride[2];       /* token, head */
  int64_t v_stride[2];
  int64_t k_cache_stride[3]; /* page, token, head */
  int64_t v_cache_stride[3];
} cache_append_t;
int cache_append(const cache_append_t* args, void* stream);

/*
 * packed_attention — attention within sequences of different lengths that lie one
 * after the other in q [tokens, q_heads, head_dim] and k, v [tokens, kv_heads,
 * head_dim]: sequence s is the tokens starts[s] .. starts[s + 1] - 1,
 *
 *     out[i, h] = sum_j softmax_j(scale * q[i,h] . k[j,g]) v[j,g],   g = h / (q_heads / kv_heads),
 *
 * over the tokens j of i's sequence, with causal those up to i itself.
 *
 *   starts    int32 [seqs + 1] on the device, rising (equal: an empty sequence). Values outside
 *             0 .. tokens are taken as the nearest of the two, a sequence that ends before it
 *             starts as empty; what sequences that overlap give is not defined.
 *   lse       float [q_heads, tokens], written when not NULL: the natural log of the sum
 *             of exp(scale * q . k)
 *
 * Rows of out and lse in no sequence (before the first start, from the last on) stay as they
 * are. What k and v hold for tokens that a row does not see does not matter to it, infinities
 * and NaN included. Arithmetic as for cross_attention.
 *
 * scale, head_dim, heads, strides (token, head) and alignment as for cross_attention, v's
 * token stride at least head_dim; tokens * q_heads at most 2^31 - CROSS_ATTENTION_PAST_END; seqs up to
 * PACKED_ATTENTION_MAX_SEQS; kv_heads below 2^20; tokens * q_heads / 128 + seqs * kv_heads below 2^24. tokens, seqs or q_heads 0: nothing is
 * enqueued. One launch, no workspace; deterministic.
 */
#define PACKED_ATTENTION_MAX_SEQS 4096
typedef struct {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;
  const int32_t* starts;
  int tokens, seqs, q_heads, kv_heads, head_dim;
  int64_t q_stride[2];       /* token, head */
  int64_t k_stride[2];
  int64_t v_stride[2];
  int64_t out_stride[2];
  float scale;
  int causal;
  int f16;                   /* 0: bfloat16, 1: binary16 */
} packed_attention_t;
int packed_attention(const packed_attention_t* args, void* stream);

/*
 * paged_attention — attention of the newest q_len tokens of each sequence, q [batch, q_len,
 * q_heads, head_dim], over its keys and values in a paged cache, k_cache and v_cache
 * [pages, page_size, kv_heads, head_dim] (cache_append):
 *
 *   table     int32 [batch, table_width] on the device: page table[b][i] holds the keys
 *             i * page_size .. of sequence b. Entries past its last key are not used.
 *             An entry outside 0 .. pages - 1 is no page: its keys are left out.
 *   lens      int32 [batch] on the device: keys of each sequence, the new tokens' own among
 *             them (append them first). Values outside 0 .. table_width * page_size
 *             are taken as the nearest of the two.
 *
 * New token i of sequence b sees the keys j <= lens[b] - q_len + i; a row that sees none gives out 0
 * and lse -inf. lse float [batch, q_heads, q_len], written when not NULL. Keys from
 * lens[b] on are never read; what keys and values hold that a row does not see does not matter to it.
 * Arithmetic as for cross_attention.
 *
 * page_size a multiple of PAGED_ATTENTION_PAGE_MULTIPLE; table_width * page_size and q_len below
 * 2^30 - CROSS_ATTENTION_PAST_END; batch * kv_heads times the tiles of 32 rows of each below 2^24; scale, head_dim, heads, strides (q and out: batch, token, head; caches: page,
 * token, head; table: batch), alignment and limits of rows as for cross_attention, v_cache's token
 * stride at least head_dim. Every 32 rows (token, query head of a key head) read the
 * keys anew, past 64 rows every 128. batch, q_len or q_heads 0: nothing is enqueued; pages or
 * table_width 0: no keys, caches and table may be NULL.
 *
 * workspace: paged_attention_workspace bytes, 16-byte aligned, that nothing else uses until the call's
 * work on `stream` has finished (0: NULL is fine). Fewer: GEMM_W4A4_ESCRATCH. Deterministic; no
 * allocation, no synchronisation.
 */
#define PAGED_ATTENTION_PAGE_MULTIPLE 16
typedef struct {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  void* out;
  float* lse;
  const int32_t* table;
  const int32_t* lens;
  int batch, q_len, q_heads, kv_heads, head_dim, pages, page_size, table_width;
  int64_t q_stride[3];       /* batch, token, head */
  int64_t k_stride[3];       /* page, token, head */
  int64_t v_stride[3];
  int64_t out_stride[3];
  int64_t table_stride;
  float scale;
  int f16;                   /* 0: bfloat16, 1: binary16 */
  void* workspace;
  int64_t workspace_bytes;
} paged_attention_t;
int paged_attention(const paged_attention_t* args, void* stream);
/* Workspace bytes of this call (sizes only; no pointer is read), or GEMM_W4A4_EINVAL (host only). */
int64_t paged_attention_workspace(const paged_attention_t* args);

/* Static string for a return code (never NULL). */
const char* gemm_w4a4_strerror(int code);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_W4A4_H */
