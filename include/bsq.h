/*
 * bsq.h -- block-scaled quantize + GEMM for MI355X (gfx950).  C ABI.
 *
 * What is computed (source pages):
 *  - NVFP4 pretraining post, section "NVFP4 pretraining recipe":
 *      ingredient 1  16-element micro-blocks (1x16) along the reduction dim;
 *      ingredient 2  E4M3 block scale factors under a per-tensor FP32 scale;
 *      ingredient 3  16-point Random Hadamard Transform on WGRAD inputs only;
 *      ingredient 4  16x16 2D weight scaling, so FPROP and the transposed
 *                    DGRAD see identical values;
 *      ingredient 5  round-to-nearest-even for weights/activations,
 *                    stochastic rounding for gradients;
 *    and the data-flow paragraph after Figure 1: the FPROP, DGRAD and WGRAD
 *    GEMMs consume NVFP4 operands and emit BF16.
 *  - HN page opcode84 (Triton on Blackwell quote, OCP MX spec link): MXFP8
 *    (E4M3 elements) and MXFP4 (E2M1 elements) with one E8M0 power-of-two
 *    scale per 32 elements, applied inside the matrix unit.
 *  - NVFP4 pretraining post, the paragraph after the example script (the FP8
 *    baseline run, quantization=te_fp8_delayedscaling) and section
 *    "Performance results" (Table 1, Figure 2: NVFP4 against that FP8
 *    baseline): the per-tensor FP8 format BSQ_FP8 below.
 *
 * Numerical definitions (bit-exact contract of the quantizers):
 *  - E2M1 magnitudes {0,0.5,1,1.5,2,3,4,6}, ties to the even code, saturate
 *    at 6; sign bit 0x8 kept (-0 -> 0x8).  Two codes per byte, the element
 *    with the even index in the low nibble.
 *  - E4M3 = OCP E4M3FN, subnormals kept, saturate at 448 (0x7E).
 *  - NVFP4 per-tensor scale: amax = max|x| (of the transformed values when the
 *    RHT applies); s_enc = 2688/amax (FP32; 1 if amax == 0; <= FLT_MAX);
 *    s_dec = 1/s_enc.  Block: sf = (a_b/6)*s_enc; S = E4M3(sf);
 *    enc = S ? min(s_enc/S, FLT_MAX) : 0; code = E2M1(x*enc).  FP32 IEEE
 *    RNE at every step, no fused multiply-add.
 *  - Per-tensor FP8 (BSQ_FP8): amax = max|x|; s_enc = 448/amax (FP32; 1 if
 *    amax == 0; <= FLT_MAX); s_dec = 1/s_enc; code = E4M3(x*s_enc), signed,
 *    RNE, saturating at 448.  No block scales; the column output is the same
 *    rule on x^T (the row codes transposed).  The delayed-scaling amax history
 *    of the baseline recipe spans training steps and is not modelled.
 *  - MX scale: e = floor(log2 a_b) - emax (emax 2 for E2M1, 8 for E4M3),
 *    -127 for an all-zero block, clamped to [-127,127], stored as e+127;
 *    element = E2M1/E4M3(x * 2^-e).
 *  - RHT: for each aligned 16-chunk y along the blocked dim: negate y_i where
 *    bit i of rht_signs is set, then butterflies h = 1,2,4,8
 *    (y_i, y_i+h) <- (y_i + y_i+h, y_i - y_i+h), then y *= 0.25 (FP32).
 *  - Stochastic rounding: element (r,c) of an output of shape [R',C'] in its
 *    own orientation has idx = r*C' + c; Philox4x32-10 (Salmon et al., SC'11)
 *    with key (seed lo, seed hi) and counter (lo(idx>>3), hi(idx>>3), offset,
 *    stream) gives 8 16-bit halves, the element takes half idx&7 (word
 *    (idx&7)>>1, low half first); stream 0 = rowwise, 1 = columnwise.  With
 *    lo <= |v| < hi the neighbouring E2M1 points, round up iff
 *    r16 < floor((|v|-lo)/(hi-lo) * 65536); |v| >= 6 -> 6.
 *
 * Conventions for every entry point:
 *  - All tensor pointers are DEVICE pointers, row-major and contiguous, and
 *    must be 16-byte aligned.  `x` is BF16.  The caller allocates every
 *    buffer; the library never allocates, frees or retains device memory and
 *    keeps no state between calls.
 *  - Every call is asynchronous on `stream` (a hipStream_t; NULL = the null
 *    stream) and never synchronizes the host.
 *  - Argument errors are detected before anything is launched: the call
 *    returns BSQ_EINVAL / BSQ_EUNSUPPORTED and no output is touched.  A launch
 *    failure returns BSQ_EHIP.  No exception crosses the ABI.
 *  - Inputs must be finite; NaN/Inf inputs give unspecified codes but never a
 *    fault.
 *  - Sizes: rows, cols, M, N, K >= 0; a zero-size call returns BSQ_OK and
 *    launches nothing except that amax outputs are set to 0.  An element
 *    count above 2^48 (rows * cols, n, M * K, N * K or M * ldc) returns
 *    BSQ_EINVAL.
 */
#ifndef BSQ_H
#define BSQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  BSQ_OK = 0,
  BSQ_EINVAL = 1,        /* null pointer, bad size, misalignment */
  BSQ_EUNSUPPORTED = 2,  /* combination the recipe does not define */
  BSQ_EHIP = 3           /* HIP launch error */
} bsq_status;

/* BSQ_FP8: per-tensor FP8, accepted by fp8_quantize_transpose (implied) and
 * bs_gemm only; the other quantizers return BSQ_EUNSUPPORTED for it. */
typedef enum { BSQ_NVFP4 = 0, BSQ_MXFP4 = 1, BSQ_MXFP8 = 2, BSQ_FP8 = 3 } bsq_format;
typedef enum { BSQ_RNE = 0, BSQ_SR = 1 } bsq_rounding;

/*
 * Rowwise NVFP4 of x[rows, cols] (BF16), blocks along cols.
 * Recipe ingredients 1, 2, 4, 5 (and 3 when rht != 0).
 *   block_rows : 1 (1x16 blocks) or 16 (16x16 tiles, rows % 16 == 0; the tile
 *                scale is written to each of its 16 rows).
 *   rnd        : BSQ_RNE or BSQ_SR (SR uses stream 0); SR with block_rows 16
 *                is BSQ_EUNSUPPORTED (it would break the transpose invariant).
 *   seed/offset: Philox key and counter word 2 for SR (ignored for RNE).
 *   rht        : nonzero = apply the 16-point RHT along cols first (amax is then
 *                taken over the transformed values); not with block_rows 16.
 *   amax_in    : NULL, or a device FP32 amax to use instead of computing it.
 *   codes      : out, uint8 [rows, cols/2], packed E2M1.
 *   scales     : out, uint8 [rows, cols/16], E4M3 block scales.
 *   amax_out   : out, device FP32 scalar: the amax used.  Required when
 *                amax_in is NULL (it is the reduction's accumulator); may be
 *                NULL otherwise.
 * Requires cols % 16 == 0.
 */
bsq_status nvfp4_quantize(const void* x, int64_t rows, int64_t cols, int block_rows,
                          bsq_rounding rnd, uint64_t seed, uint32_t offset,
                          int rht, uint16_t rht_signs, const float* amax_in,
                          uint8_t* codes, uint8_t* scales, float* amax_out,
                          void* stream);

/*
 * Rowwise MXFP4 (fmt BSQ_MXFP4, E2M1 elements) or MXFP8 (BSQ_MXFP8, E4M3
 * elements) of x[rows, cols] with one E8M0 scale per 32 elements along cols.
 * HN page opcode84 (MX formats; OCP MX spec).
 *   rnd    : BSQ_RNE, or BSQ_SR for MXFP4 only (stream 0).
 *   codes  : out, uint8 [rows, cols/2] (MXFP4) or [rows, cols] (MXFP8).
 *   scales : out, uint8 [rows, cols/32], E8M0.
 * Requires cols % 32 == 0.
 */
bsq_status mx_quantize(const void* x, int64_t rows, int64_t cols, bsq_format fmt,
                       bsq_rounding rnd, uint64_t seed, uint32_t offset,
                       uint8_t* codes, uint8_t* scales, void* stream);

/*
 * Both orientations from one read of x[rows, cols]:
 *   row = quantize(x)    -> codes_row [rows, cols/2 or cols], scales_row [rows, cols/B]
 *   col = quantize(x^T)  -> codes_col [cols, rows/2 or rows], scales_col [cols, rows/B]
 * B = 16 (NVFP4) or 32 (MX).  Recipe: ingredient 4 (the transposed DGRAD
 * operand of 2D-scaled weights), ingredient 3 (WGRAD operands are quantized
 * along tokens, with the RHT), data-flow paragraph.
 *   fmt        : BSQ_NVFP4, BSQ_MXFP4 or BSQ_MXFP8.
 *   block_rows : 1, or 16 for NVFP4 2D tiles (then row and col codes are the
 *                same values transposed and both scale arrays hold the same
 *                tile scales).
 *   rnd        : RNE or SR (SR: rowwise stream 0, columnwise stream 1); not SR
 *                with 2D tiles or MXFP8.
 *   rht_col    : nonzero = RHT along rows (the blocked dim of x^T) for the col
 *                output only; NVFP4 1x16 only; with the col output it needs
 *                cols < 2^26 (BSQ_EINVAL otherwise).
 *   amax_row / amax_col : out, device FP32 (NVFP4 only; ignored for MX).
 *                amax_row = max|x|; amax_col = max|RHT(x^T)| with rht_col,
 *                else equal to amax_row.
 * Either triple (codes_row, scales_row, amax_row) or (codes_col, scales_col,
 * amax_col) may be all-NULL to skip that orientation (not both).
 * Requires rows % 16 == 0 and cols % 16 == 0 (NVFP4) or rows % 32 == 0 and
 * cols % 32 == 0 (MX).
 */
bsq_status quantize_transpose(const void* x, int64_t rows, int64_t cols, bsq_format fmt,
                              int block_rows, bsq_rounding rnd, uint64_t seed, uint32_t offset,
                              int rht_col, uint16_t rht_signs,
                              uint8_t* codes_row, uint8_t* scales_row, float* amax_row,
                              uint8_t* codes_col, uint8_t* scales_col, float* amax_col,
                              void* stream);

/*
 * NVFP4 row and column outputs of x[rows, cols] under per-tensor amaxes the
 * caller already holds, typically from the producer of x (swiglu_amax,
 * swiglu_backward_amax below): the encode pass of quantize_transpose without
 * its amax pass.  Recipe ingredients 1-5 as for quantize_transpose with
 * fmt = BSQ_NVFP4; given the amaxes quantize_transpose would compute, the
 * codes and scales are the same bytes.
 *   block_rows, rnd, seed, offset, rht_col, rht_signs : as quantize_transpose.
 *   amax_row : in, device FP32 max|x|; required with the row outputs.
 *   amax_col : in, device FP32 amax of the col side (max|RHT(x^T)| with
 *              rht_col, else max|x|); required with the col outputs.  With
 *              block_rows 16 and both orientations it must be the same
 *              pointer as amax_row (one amax encodes both sides of a 16x16
 *              tile); BSQ_EINVAL otherwise.
 *   codes_row, scales_row / codes_col, scales_col : out, as quantize_transpose;
 *              either pair may be NULL to skip that orientation (not both).
 * Requires rows % 16 == 0 and cols % 16 == 0.
 */
bsq_status quantize_transpose_amax(const void* x, int64_t rows, int64_t cols, int block_rows,
                                   bsq_rounding rnd, uint64_t seed, uint32_t offset, int rht_col,
                                   uint16_t rht_signs, const float* amax_row, const float* amax_col,
                                   uint8_t* codes_row, uint8_t* scales_row, uint8_t* codes_col,
                                   uint8_t* scales_col, void* stream);

/*
 * SwiGLU forward of the MLP whose GEMMs the NVFP4 post measures (section
 * "Performance results": Llama 3 8B and Llama 3.1 405B, whose MLP is the
 * gate/up GEMM, SwiGLU, then the down GEMM), producing the BF16 input of the
 * down projection together with the amaxes its NVFP4 quantizer needs (the
 * data-flow paragraph after Figure 1: activations enter the next GEMM in
 * NVFP4).  The pages give no SwiGLU formula; the reading used:
 *   y_gu : in, BF16 [rows, 2f] = [G | U] (gate = first f columns).
 *   h    : out, BF16 [rows, f], h = BF16_RNE(silu(G) * U), silu(g) =
 *          g / (1 + exp(-g)); computed in FP32 (v_exp / v_rcp), so an element
 *          may differ from the exactly rounded value by one BF16 ulp.
 *   amax_row : out, device FP32 max|h| (or NULL).
 *   amax_col : out, device FP32: with rht_col, max|RHT(h^T)| (16-row chunks,
 *              rht_signs, the quantize_transpose rule); else max|h| (or NULL).
 *              Both amaxes equal what quantize_transpose computes on h.
 * With both amax pointers NULL only h is written.  h must not overlap y_gu.
 * Requires rows % 16 == 0, f % 16 == 0 and f < 2^25.
 */
bsq_status swiglu_amax(const void* y_gu, int64_t rows, int64_t f, int rht_col, uint16_t rht_signs,
                       void* h, float* amax_row, float* amax_col, void* stream);

/*
 * SwiGLU backward (the chain rule of h = silu(G) * U) producing the BF16
 * gradient of the gate/up GEMM output with the amaxes of its NVFP4 quantizer
 * (rowwise SR for DGRAD, columnwise SR + RHT for WGRAD: recipe ingredients 3
 * and 5).
 *   y_gu   : in, BF16 [rows, 2f] = [G | U], the forward's input.
 *   d_h    : in, BF16 [rows, f], gradient of h.
 *   d_y_gu : out, BF16 [rows, 2f] = [dG | dU], dU = BF16_RNE(dH * silu(G)),
 *            dG = BF16_RNE(dH * U * silu'(G)), silu'(g) = sigma(g) *
 *            (1 + g * (1 - sigma(g))); FP32 arithmetic, one BF16 ulp as for
 *            swiglu_amax.
 *   amax_row, amax_col : out, as for swiglu_amax, over d_y_gu.
 * d_y_gu must not overlap y_gu or d_h.  Requires rows % 16 == 0, f % 16 == 0
 * and f < 2^25.
 */
bsq_status swiglu_backward_amax(const void* y_gu, const void* d_h, int64_t rows, int64_t f,
                                int rht_col, uint16_t rht_signs, void* d_y_gu, float* amax_row,
                                float* amax_col, void* stream);

/*
 * FP32 master-weight update of the optimizer step: the data-flow paragraph
 * after Figure 1 of the NVFP4 post folds the BF16 GEMM outputs (here the
 * WGRAD output dW) into an FP32 master weight; the pages name no optimizer,
 * so the plain fold is used.  For each of the n elements:
 *   w32[i]    <- FP32(w32[i] - FP32(lr * grad[i]))   (two RNE roundings, no FMA)
 *   w_bf16[i] <- BF16_RNE(w32[i])                     (the copy the next step quantizes)
 *   amax      <- max |w_bf16|                         (device FP32, or NULL)
 * The amax is the per-tensor amax of the next 16x16 weight quantization
 * (quantize_transpose_amax with block_rows 16, as amax_row and amax_col).
 *   w32    : in/out, FP32 [n].       grad : in, BF16 [n].
 *   w_bf16 : out, BF16 [n].  The three arrays must not overlap.
 * Requires n % 8 == 0.
 */
bsq_status master_weight_update(float* w32, const void* grad, int64_t n, float lr, void* w_bf16,
                                float* amax, void* stream);

/*
 * Per-tensor FP8 (E4M3) of x[rows, cols] (BF16) in both orientations from
 * one amax pass and one encode pass: the FP8 baseline's operands for FPROP
 * (rowwise), DGRAD (W columnwise) and WGRAD (dY and X columnwise).
 *   codes_row : out, uint8 [rows, cols], E4M3 codes of x (or NULL).
 *   codes_col : out, uint8 [cols, rows], E4M3 codes of x^T, i.e. codes_row
 *               transposed (or NULL; not both NULL).
 *   amax      : out, device FP32 scalar max|x| (the reduction's accumulator;
 *               required).  The GEMM derives s_dec from it.
 * Requires rows % 16 == 0 and cols % 16 == 0.
 */
bsq_status fp8_quantize_transpose(const void* x, int64_t rows, int64_t cols, uint8_t* codes_row,
                                  uint8_t* codes_col, float* amax, void* stream);

/*
 * C[M, N] (BF16, row-major, row stride ldc >= N elements) =
 *     alpha * sum_k deq(A)[m, k] * deq(B)[n, k]
 * with A [M, K] and B [N, K] both K-major (quantized along K), FP32
 * accumulation and one BF16 round-to-nearest-even at the end.  Data-flow
 * paragraph: FPROP (A = X rowwise, B = W rowwise 2D), DGRAD (A = dY rowwise,
 * B = W columnwise 2D), WGRAD (A = dY columnwise, B = X columnwise, K = tokens).
 *   NVFP4: codes [M, K/2] + E4M3 scales [M, K/16] per operand and a device
 *          FP32 amax per operand; alpha = s_dec(a_amax) * s_dec(b_amax).
 *          Requires K % 16 == 0.
 *   MXFP4: codes [M, K/2], MXFP8: codes [M, K]; E8M0 scales [M, K/32];
 *          a_amax and b_amax are ignored (may be NULL); alpha = 1.
 *          Requires K % 32 == 0.
 *   FP8:   per-tensor E4M3 codes [M, K] (fp8_quantize_transpose); a_scales
 *          and b_scales are ignored (may be NULL); device FP32 a_amax and
 *          b_amax required; alpha = s_dec(a_amax) * s_dec(b_amax) with
 *          s_dec = 1/(448/amax).  Requires K % 32 == 0.
 * M and N may be any value >= 0.  C must not alias any input.
 * Workspace (NVFP4 only): when the 256 x 256 output tiles fill at least one
 * wave of the device's compute units and leave a last wave of at most half
 * of them (K % 512 == 0, K >= 4096), each tile of that last wave is computed
 * as two FP32 partial sums over the two halves of K, added in a second
 * kernel (the same order for every element: repeated calls give identical
 * bits; the sum differs from a one-pass accumulation only in FP32 rounding).
 * Their 512 KiB per tile come from the stream-ordered allocator
 * (hipMallocAsync / hipFreeAsync on `stream`); BSQ_EHIP if that fails.
 */
bsq_status bs_gemm(bsq_format fmt, int64_t M, int64_t N, int64_t K,
                   const uint8_t* a_codes, const uint8_t* a_scales, const float* a_amax,
                   const uint8_t* b_codes, const uint8_t* b_scales, const float* b_amax,
                   void* c, int64_t ldc, void* stream);

/*
 * bs_gemm for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments, checks and results (bit for bit) as bs_gemm; the NVFP4
 * split-last-wave workspace is the library's static per-device array of
 * 64 MiB (held by each device the library runs on until the process ends)
 * instead of the stream-ordered allocator, and no call allocates.  The
 * first call on a device looks up that array's address (make it outside
 * graph capture).  Returns BSQ_EUNSUPPORTED if the split would need more
 * than 64 MiB (more than 256 compute units).  Calls that overlap on one
 * device (other streams, other host threads) share the array and race.
 */
bsq_status bs_gemm_noalloc(bsq_format fmt, int64_t M, int64_t N, int64_t K,
                           const uint8_t* a_codes, const uint8_t* a_scales, const float* a_amax,
                           const uint8_t* b_codes, const uint8_t* b_scales, const float* b_amax,
                           void* c, int64_t ldc, void* stream);

/*
 * FP16 expansion of an NVFP4 operand (recipe ingredients 1-2: E2M1 codes
 * under E4M3 block scales), without its per-tensor scale:
 *   out[r, k] = v * S * 2^-7   (FP16, exact: v * S has at most 6 significant
 *                               bits and lies in [2^-10, 2688])
 * with v the E2M1 value of element (r, k) and S its block's E4M3 scale.
 *   codes  : in, uint8 [rows, cols/2] (8-byte aligned); scales : in, uint8 [rows, cols/16].
 *   out    : out, FP16 [rows, cols].
 * Requires cols % 16 == 0.  This is the B operand of bs_gemm_nvfp4_bx.
 */
bsq_status nvfp4_expand(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                        void* out, void* stream);

/*
 * The NVFP4 GEMM of bs_gemm (data-flow paragraph after Figure 1: FPROP,
 * DGRAD, WGRAD consume NVFP4 operands, emit BF16) with B handed over as its
 * FP16 expansion (nvfp4_expand of B's codes and scales): the kernel expands
 * only A.  The result is bit-identical to bs_gemm(BSQ_NVFP4, ...) on the
 * same operands whenever bs_gemm does not split its last wave over K (see
 * bs_gemm's workspace note).  For operands used by several GEMMs or much smaller than
 * the other operand (weights, the smaller WGRAD input), expanding once and
 * streaming FP16 costs less than expanding inside every output tile.
 *   a_codes [M, K/2], a_scales [M, K/16], a_amax : the NVFP4 A operand.
 *   b_x    : FP16 [N, K], nvfp4_expand of B;  b_amax : B's per-tensor amax.
 *   c      : BF16 [M, N], row stride ldc; alpha = s_dec(a_amax) * s_dec(b_amax).
 * BSQ_EUNSUPPORTED unless K % 128 == 0, K > 0, a_codes and b_x are 16-byte
 * aligned, a_scales 4-byte aligned, M * K / 2 < 2^32 and N * K * 2 < 2^32
 * (bs_gemm covers every other shape).
 */
bsq_status bs_gemm_nvfp4_bx(int64_t M, int64_t N, int64_t K, const uint8_t* a_codes,
                            const uint8_t* a_scales, const float* a_amax, const void* b_x,
                            const float* b_amax, void* c, int64_t ldc, void* stream);

/* ---------------------------------------------------------------------------
 * Around the MLP block: norms, gate and residual, and a mixture-of-experts MLP.
 * What surrounds the block-scaled products in a transformer layer.  The pages
 * give no formulas for these parts, so the usual definitions are used, written
 * out below.  All arithmetic is FP32 with one rounding at each store; no result
 * depends on the order of atomics.
 * ------------------------------------------------------------------------- */

/* Type of a residual stream or of router logits. */
typedef enum { BSQ_BF16 = 0, BSQ_F32 = 1 } bsq_dtype;
/* What a gate is broadcast over: FP32 [cols], FP32 [rows], or BF16 [rows, cols]. */
typedef enum { BSQ_GATE_NONE = 0, BSQ_GATE_CHANNEL = 1, BSQ_GATE_ROW = 2, BSQ_GATE_FULL = 3 } bsq_gate;
/* Score of a router logit. */
typedef enum { BSQ_SOFTMAX = 0, BSQ_SIGMOID = 1 } bsq_scoring;

/*
 * The step from one block to the next: norm of the block's output, its gate and
 * the scaled residual, and the norm that opens the next block, in one pass.
 *   n = o * rstd_post * w_post   (w_post NULL: n = o)
 *   r = alpha * x + gate * n
 *   h = BF16(r * rstd_pre * w_pre),  r before its rounding
 *   rstd = 1 / sqrt(mean over the row of v^2 + eps)
 *   x    : in, [rows, cols] of x_type.   o : in, BF16 [rows, cols], or NULL:
 *          then h = norm(x) only (w_post, gate and r must be absent too).
 *   gate : in, see bsq_gate (NULL with BSQ_GATE_NONE).
 *   w_post, w_pre : in, FP32 [cols].  w_pre NULL: no h, rstd_pre and amax.
 *   r    : out, [rows, cols] of x_type.  h : out, BF16 [rows, cols].
 *   rstd_post, rstd_pre : out, FP32 [rows] (what the backward takes), or NULL.
 *   amax : out, device FP32 max|h| for the NVFP4 quantizers, or NULL.
 * Outputs must not overlap inputs.  1 <= cols <= 16384 (BSQ_EUNSUPPORTED above),
 * eps > 0.  Pointers need their element's alignment only; whole 16-byte pieces
 * are used where cols % 8 == 0 and all of them are 16-byte aligned.
 */
bsq_status block_norm(const void* x, bsq_dtype x_type, const void* o, int64_t rows, int64_t cols,
                      const float* w_post, bsq_gate gate_kind, const void* gate, float alpha,
                      const float* w_pre, float eps, void* r, void* h, float* rstd_post,
                      float* rstd_pre, float* amax, void* stream);

/* Bytes of device workspace block_norm_backward needs for these sizes. */
bsq_status block_norm_backward_workspace(int64_t rows, int64_t cols, int64_t* bytes);

/*
 * Gradient of block_norm.  With rn = r * rstd_pre, on = o * rstd_post (w_post
 * NULL: on = o, its factor 1), a = d_h * w_pre:
 *   G      = d_r + rstd_pre * (a - rn * mean(a rn))
 *   d_x    = alpha * G (without o: G)            [rows, cols] of r_type
 *   d_gate = G * on * w_post, summed over what the gate is broadcast over
 *            (FP32 [cols] or [rows]; BF16 [rows, cols] for BSQ_GATE_FULL)
 *   b      = G * gate * w_post;  d_o = rstd_post * (b - on * mean(b on)), BF16
 *   d_w_pre = sum over rows of d_h rn;  d_w_post = sum over rows of G gate on (FP32)
 *   r    : in, block_norm's r (without o: its x).  d_r : in, or NULL (zero).
 *   d_h  : in, BF16; required with w_pre, NULL without.
 * Column sums are accumulated per workgroup and joined in a fixed order.
 * rows == 0 writes zeros to d_w_pre, d_w_post and a channel gate's d_gate.
 *   workspace : device memory, 16-byte aligned, at least the bytes of
 *               block_norm_backward_workspace.
 */
bsq_status block_norm_backward(const void* r, bsq_dtype r_type, const void* o, const void* d_r,
                               const void* d_h, int64_t rows, int64_t cols, const float* w_post,
                               bsq_gate gate_kind, const void* gate, float alpha, const float* w_pre,
                               const float* rstd_post, const float* rstd_pre, void* d_x, void* d_o,
                               void* d_gate, float* d_w_pre, float* d_w_post, void* workspace,
                               int64_t workspace_bytes, void* stream);

/*
 * Rows of the expert-ordered buffers of moe_route: enough for every routing of
 * tokens * k assignments to groups padded to `align` rows.  align == 1: tokens *
 * k; else a multiple of 512, so that a quantized reduction over the rows keeps
 * 16-byte aligned scale rows.
 */
bsq_status moe_rows(int64_t tokens, int experts, int k, int align, int64_t* rows);

/* Bytes of device workspace moe_route needs. */
bsq_status moe_route_workspace(int64_t tokens, int experts, int k, int64_t* bytes);

/*
 * The router.  Per token: the k experts with the largest logit + bias (FP32
 * sum), in descending order, ties to the lowest expert; an expert whose logit or
 * sum is -inf or NaN is masked and never taken.  Weights, times scale:
 *   softmax, normalize : softmax over the selected logits
 *   softmax            : softmax over all logits but those that are -inf or NaN
 *                        themselves (one that only the bias masks keeps its share,
 *                        and its gradient)
 *   sigmoid, normalize : sigmoid(l) over the sum of the selected sigmoids
 *   sigmoid            : sigmoid(l)
 * (the bias steers the selection only, and is added to the logit: a correction
 * bias trained to be added to the score goes to moe_route_score_bias, which takes
 * other experts under the same numbers).  A slot without a candidate left gets
 * expert -1, weight 0 and row -1.  Rows: the assignments sorted by expert, then
 * token, then slot, each expert's group padded to a multiple of align rows.
 *   logits  : in, [tokens, experts] of type.  bias : in, FP32 [experts] or NULL.
 *   rows    : length of src, at least moe_rows (BSQ_EINVAL otherwise).
 *   experts_out : out, int32 [tokens, k].    weights : out, FP32 [tokens, k].
 *   offsets : out, int32 [experts + 1], first row of each padded group and the end.
 *   row_of  : out, int32 [tokens, k], row of the assignment.
 *   src     : out, int32 [rows], token * k + slot of the row, -1 in the padding
 *             and past the last group.
 *   workspace : device memory, 4-byte aligned (moe_route_workspace bytes).
 * 1 <= k <= min(experts, 16), experts <= 512 (BSQ_EUNSUPPORTED above), 1 <= align
 * <= 512, rows < 2^31.
 */
bsq_status moe_route(const void* logits, bsq_dtype type, int64_t tokens, int experts, int k,
                     const float* bias, bsq_scoring scoring, int normalize, float scale, int align,
                     int64_t rows, int32_t* experts_out, float* weights, int32_t* offsets,
                     int32_t* row_of, int32_t* src, void* workspace, int64_t workspace_bytes,
                     void* stream);

/*
 * moe_route with the selection bias of routers balanced without an auxiliary loss:
 * per token the k experts with the largest score + score_bias (FP32 sum), the score
 * being sigmoid(l), or softmax(l) over all experts whose logit is not masked, as
 * FP32 (within a few units in the last place of the exact value, so scores closer
 * than that can change places).  Masks, ties, weights (without the bias), rows and
 * outputs as for moe_route; score_bias is FP32 [experts], not NULL.
 */
bsq_status moe_route_score_bias(const void* logits, bsq_dtype type, int64_t tokens, int experts, int k,
                                const float* score_bias, bsq_scoring scoring, int normalize, float scale,
                                int align, int64_t rows, int32_t* experts_out, float* weights,
                                int32_t* offsets, int32_t* row_of, int32_t* src, void* workspace,
                                int64_t workspace_bytes, void* stream);

/*
 * Gradient of moe_route's weights with respect to its logits; the selection is
 * constant.  Logits of no slot get 0, except for softmax without normalize (there
 * 0 for logits of -inf or NaN and for tokens without any expert).
 *   experts_in : in, moe_route's experts.  d_weights : in, FP32 [tokens, k].
 *   d_logits   : out, [tokens, experts] of type.
 */
bsq_status moe_route_backward(const void* logits, bsq_dtype type, int64_t tokens, int experts, int k,
                              const int32_t* experts_in, const float* d_weights, bsq_scoring scoring,
                              int normalize, float scale, void* d_logits, void* stream);

/*
 * Token rows to expert order: out[p] = x[src[p] / k], zeros where src[p] is not
 * in [0, tokens * k).  Its gradient is moe_combine without weights.
 *   x : in, BF16 [tokens, cols].  src : in, int32 [rows].  out : out, BF16 [rows, cols].
 * The row movers take cols <= 2^30 (BSQ_EUNSUPPORTED above).
 */
bsq_status moe_gather(const void* x, int64_t tokens, int64_t cols, int k, const int32_t* src,
                      int64_t rows, void* out, void* stream);

/*
 * Expert rows back to tokens: out[t] = sum over the slots j, in order, of
 * weights[t, j] * y[row_of[t, j]], slots whose row is not in [0, rows) left out.
 *   y : in, BF16 [rows, cols].  row_of : in, int32 [tokens, k].
 *   weights : in, FP32 [tokens, k], or NULL (1).  out : out, BF16 [tokens, cols].
 */
bsq_status moe_combine(const void* y, int64_t rows, int64_t cols, const int32_t* row_of,
                       const float* weights, int64_t tokens, int k, void* out, void* stream);

/*
 * Gradient of moe_combine: d_y[p] = weights[a] * d_out[a / k] with a = src[p]
 * (zeros where a is not in [0, tokens * k)), d_weights[a] = <d_out[a / k], y[p]>
 * with p = row_of[a], 0 where p is not in [0, rows) or src[p] is not a.  src and
 * row_of come from one moe_route; a buffer cut to a capacity (fewer rows, src cut
 * alike) or slots taken out of either are slots without a row.
 */
bsq_status moe_combine_backward(const void* d_out, const void* y, int64_t tokens, int64_t cols, int k,
                                const int32_t* src, const int32_t* row_of, const float* weights,
                                int64_t rows, void* d_y, float* d_weights, void* stream);

/*
 * Products grouped by expert, the rows ragged (FPROP and DGRAD of an expert
 * MLP, prompts and single tokens): for the rows p of group e, offsets[e] <= p <
 * offsets[e + 1],
 *   C[p, n] = alpha_e * sum_k deq(A)[p, k] * deq(B_e)[n, k]
 * and zeros in the rows of no group (before offsets[0] and from offsets[experts]
 * on).  FP32 accumulation, one BF16 rounding; MXFP8: the matrix instruction adds
 * eight neighbouring products (k = 8 i .. 8 i + 7) with an error of up to 2^-13 of
 * the largest each, in bs_gemm too.  Operands as for bs_gemm: A [rows, K], B
 * [experts, N, K], contiguous.
 *   fmt     : BSQ_NVFP4 (K % 16 == 0), BSQ_MXFP4 or BSQ_MXFP8 (K % 32 == 0);
 *             BSQ_FP8 is BSQ_EUNSUPPORTED.
 *   offsets : in, device int32 [experts + 1], ascending (values outside [0,
 *             rows] are read as the nearest bound).  Groups may be empty.
 *   a_amax  : NVFP4: device FP32.  b_amax : NVFP4: device FP32 [b_amax_n],
 *             b_amax_n 1 or experts.  alpha as for bs_gemm; ignored for MX.
 * 1 <= experts <= 4096, rows < 2^31.  Codes must be 16-byte aligned.
 */
bsq_status bs_gemm_grouped(bsq_format fmt, int experts, const int32_t* offsets, int64_t rows, int64_t N,
                           int64_t K, const uint8_t* a_codes, const uint8_t* a_scales,
                           const float* a_amax, const uint8_t* b_codes, const uint8_t* b_scales,
                           const float* b_amax, int b_amax_n, void* c, int64_t ldc, void* stream);

/*
 * Products grouped by expert, the reduction ragged (WGRAD of an expert MLP):
 *   C[e, m, n] = alpha * sum over the rows p of group e of deq(A)[m, p] * deq(B)[n, p]
 * with A [M, rows], B [N, rows] quantized along the rows (the column outputs of
 * quantize_transpose on expert-ordered tensors); an empty group's C is zero.
 *   offsets : as above, multiples of the scale block (16 NVFP4, 32 MX; other
 *             values are read as the multiple below).  rows % block == 0.
 *   a_amax, b_amax : NVFP4: device FP32.   c : out, BF16 [experts, M, N].
 */
bsq_status bs_gemm_grouped_wgrad(bsq_format fmt, int experts, const int32_t* offsets, int64_t M, int64_t N,
                                 int64_t rows, const uint8_t* a_codes, const uint8_t* a_scales,
                                 const float* a_amax, const uint8_t* b_codes, const uint8_t* b_scales,
                                 const float* b_amax, void* c, void* stream);

/* ---------------------------------------------------------------------------
 * 8-bit integers: another baseline of the block's products, with a scale for each
 * token (row of A) and each output channel (row of B) instead of one per tensor or
 * block.  The pages give no formulas, so the usual definitions are used.
 * ------------------------------------------------------------------------- */

/*
 * Codes of the rows of x[rows, cols] (BF16), one scale per row:
 *   amax = max|x| of the row; s_enc = 127 * (1/amax), two roundings (1 if amax == 0;
 *   <= FLT_MAX);
 *   scale = 1/s_enc; code = RNE(x * s_enc), in [-127, 127]
 * (FP32 IEEE RNE at every step).  NaN and infinities touch their own row only: a row
 * with NaN has scale NaN, one with infinities and no NaN scale infinity and codes 0, so
 * that either's products are NaN.
 *   codes  : out, int8 [rows, cols].  scales : out, FP32 [rows].
 * Any rows, any cols (cols == 0: scales of 1).
 */
bsq_status int8_quantize(const void* x, int64_t rows, int64_t cols, int8_t* codes, float* scales,
                         void* stream);

/* Bytes of device workspace int8_quantize_transpose needs. */
bsq_status int8_quantize_transpose_workspace(int64_t rows, int64_t cols, int64_t* bytes);

/*
 * int8_quantize of x and of x^T, for products over either dimension (FPROP, DGRAD
 * and WGRAD of a training step):
 *   codes_row [rows, cols], scales_row [rows]; codes_col [cols, rows], scales_col [cols].
 * Either pair may be NULL (not both).  workspace: device memory, 4-byte aligned.
 */
bsq_status int8_quantize_transpose(const void* x, int64_t rows, int64_t cols, int8_t* codes_row,
                                   float* scales_row, int8_t* codes_col, float* scales_col,
                                   void* workspace, int64_t workspace_bytes, void* stream);

/*
 * C[m, n] = BF16(FP32(sum_k A[m, k] B[n, k]) * (a_scales[m] * b_scales[n]) + bias[n])
 * with A int8 [M, K] and B int8 [N, K], the sum exact, so that the result depends on
 * the operands alone.  K == 0: the bias (or zeros).
 *   bias : in, FP32 [N] or NULL.   c : out, BF16 [M, N], row stride ldc >= N.
 * K < 2^17 (the sums are 32 bits): BSQ_EUNSUPPORTED above.  C must not alias an input.
 */
bsq_status int8_gemm(int64_t M, int64_t N, int64_t K, const int8_t* a_codes, const float* a_scales,
                     const int8_t* b_codes, const float* b_scales, const float* bias, void* c,
                     int64_t ldc, void* stream);

/* Bytes of device workspace int8_linear needs (the codes and scales of x). */
bsq_status int8_linear_workspace(int64_t M, int64_t K, int64_t* bytes);

/*
 * The serving form: C = int8_gemm of int8_quantize(x) with weights quantized
 * beforehand, for one token or many.
 *   x : in, BF16 [M, K].   w_codes, w_scales, bias, c, ldc : as for int8_gemm's B.
 *   workspace : device memory, 16-byte aligned.
 */
bsq_status int8_linear(const void* x, int64_t M, int64_t N, int64_t K, const int8_t* w_codes,
                       const float* w_scales, const float* bias, void* c, int64_t ldc,
                       void* workspace, int64_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Orthogonalised weight updates (Newton-Schulz products), beside
 * master_weight_update.
 * ------------------------------------------------------------------------- */

/* Bytes of device workspace orthogonalize and muon_update need (BSQ_EUNSUPPORTED for
 * sizes they do not take: rows or cols of 2^22 or more, batch above 65,535). */
bsq_status orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols, int64_t* bytes);

/*
 * For each matrix x[rows, cols] of a stack of `batch`:
 *   X = x / (||x||_F + eps); for each step's a, b, c: A = X X^T,
 *   X <- (a I + b A + c A^2) X;  out = BF16(X)
 * (on the transpose where rows > cols, which is the same).  The products take FP16
 * matrices under a power of two (each rounding at most 2^-11 of the value) and sum in
 * FP32; X itself is held to 22 bits, the diagonals of A and the polynomials in FP32,
 * the norm in FP64.  Five steps of the usual coefficients are 3e-4 to 1e-3 (relative,
 * Frobenius) from the exact result on gradients, and at most 2e-3 on a matrix of any rank
 * and any spread of its singular values; 5e-3 for fewer than 16 rows or columns, and where
 * steps are taken in pairs (the smaller side, in multiples of 64, above 256, and the larger
 * at least 4/3 of it).  Each further step multiplies what the last bits of X and of the
 * sums leave along singular values of zero by its a: eight steps are at most 8e-3 up to
 * 4,096 rows.  Coefficients must keep singular values below 8.  A zero matrix gives zeros; a
 * matrix with NaN or infinities gives NaN of its own.
 *   x     : in, [batch, rows, cols] of type.   out : out, BF16 [batch, rows, cols].
 *   coefs : in, HOST array of 3 * steps floats, 1 <= steps <= 32.   eps > 0.
 *   workspace : device memory, 256-byte aligned.
 */
bsq_status orthogonalize(const void* x, bsq_dtype type, int64_t batch, int64_t rows, int64_t cols,
                         int steps, const float* coefs, float eps, void* out, void* workspace,
                         int64_t workspace_bytes, void* stream);

/*
 * One optimizer step of a stack of weight matrices, in place on w32 and momentum:
 *   momentum <- mu * momentum + grad;   u = grad + mu * momentum (nesterov) or momentum
 *   w32 <- (1 - lr * weight_decay) * w32 - lr * scale * orthogonalize(u)
 *   w_bf16 <- BF16_RNE(w32);  amax <- max|w_bf16| over the stack
 * (FP32; orthogonalize's result in FP32, or rounded to FP16 here).  amax is the per-tensor amax of
 * the next weight quantization, as for master_weight_update.
 *   w32, momentum : in/out, FP32 [batch, rows, cols].  grad : in, BF16.
 *   w_bf16 : out, BF16.  amax : out, device FP32 or NULL.  No two may overlap.
 */
bsq_status muon_update(float* w32, float* momentum, const void* grad, int64_t batch, int64_t rows,
                       int64_t cols, float lr, float mu, int nesterov, float weight_decay, float scale,
                       int steps, const float* coefs, float eps, void* w_bf16, float* amax,
                       void* workspace, int64_t workspace_bytes, void* stream);

/* Static, human-readable name of a status code; host-side, thread-safe. */
const char* bsq_status_string(bsq_status status);

#ifdef __cplusplus
}
#endif

#endif /* BSQ_H */
