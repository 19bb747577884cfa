/*
 * mx.h — C ABI of the MXFP4 block-scaled Hadamard-32 hot path for AMD MI355X (gfx950).
 *
 * The library (libmx.so) quantizes bf16/fp32 tensors into MXFP4 (E2M1 elements sharing one
 * E8M0 power-of-two scale per block of 32 elements, or per 32x32 tile) with an optional
 * 32-point Walsh-Hadamard rotation, and multiplies MXFP4 operands with gfx950's block-scaled
 * matrix cores for the three GEMMs of a linear layer (forward, input gradient, weight
 * gradient). For decoding it has the product of a few tokens, adapters beside it, and a cache of
 * keys and values with the attention over it.
 *
 * Sources (web pages; cited by title and section):
 *  [P1] "Block-Scaled MXFP4 With Stochastic Hadamard Rounding Matches BF16 Convergence on 70B
 *       Pre-Training" (lazytensor.com news item), paragraphs 1-2: one shared 8-bit power-of-two
 *       exponent (E8M0) per block of 32 4-bit E2M1 values; a 32-element block-diagonal
 *       Walsh-Hadamard transform applied in registers before the values are packed to 4 bits.
 *  [P2] "Pretraining large language models with MXFP4" (arXiv 2605.09825, abstract): FP4 in
 *       Fprop, Dgrad and Wgrad; deterministic Hadamard rotations stabilise the Wgrad path.
 *  [P3] "Stable FP4 Training via Transposition-Invariant Block Quantization" (arXiv 2607.24953
 *       review): section "Why FP4 training is the current frontier" (E2M1 bits, per-block scale
 *       from the block max, P = round(X/S), reconstruction P*S); section "The aha: transposition
 *       scrambles the blocks" (the GEMM orientations, 1-D re-blocking under transposition);
 *       section "The fix, and its supporting cast" (32x32 blocks, scale rounded up to a power of
 *       two so nothing clips, stochastic rounding with E[round(x)] = x).
 *  [P4] "Training LLMs with MXFP4" (arXiv 2502.20586, abstract): stochastic rounding plus a
 *       random Hadamard transform (random +/-1 signs) to bound its variance.
 *
 * Conventions shared by every entry point:
 *  - Every tensor pointer is DEVICE memory owned by the caller. The library allocates no
 *    device memory, keeps no global state and never synchronises; all work is enqueued on
 *    `stream` (a hipStream_t passed as void*, NULL = the null stream).
 *  - `opts` is a HOST pointer, read during the call only.
 *  - The return value reports argument validation and launch errors. A non-OK status means
 *    nothing was enqueued. Faults during execution surface at the caller's next
 *    synchronisation of `stream`.
 *  - Dimensions are element counts; every dimension along which blocks are formed must be a
 *    positive multiple of 32 (MX_ERR_SHAPE otherwise). A zero-sized tensor is MX_OK and
 *    enqueues nothing.
 *  - Packed codes: two E2M1 codes per byte, the element with the even index along the packed
 *    (block) axis in the low nibble. A code is (sign << 3) | m, m in 0..7 indexing the
 *    magnitudes {0, 0.5, 1, 1.5, 2, 3, 4, 6}. The sign bit is copied from the value, so a
 *    negative value that rounds to zero is code 0x8.
 *  - Scales: one byte per block, value 2^(byte-127); byte 0xFF (NaN) marks a block whose
 *    maximum was not finite (its codes are then all zero).
 */
#ifndef MX_H
#define MX_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MX_OK = 0,
  MX_ERR_NULL = 1,        /* a required pointer is NULL */
  MX_ERR_SHAPE = 2,       /* a dimension is negative, not a multiple of 32, or ld too small */
  MX_ERR_UNSUPPORTED = 3, /* an option combination the path does not define */
  MX_ERR_LAUNCH = 4,      /* the HIP runtime refused the launch */
  MX_ERR_ARG = 5          /* an enum/option value out of range */
} mx_status;

typedef enum { MX_F32 = 0, MX_BF16 = 1 } mx_dtype;

/* Scale exponent e of a block with maximum magnitude amax = m * 2^E, m in [1, 2):
 *  MX_SCALE_FLOOR: e = E - 2 (the OCP rule: floor(log2 amax) minus E2M1's largest exponent);
 *                  elements whose scaled magnitude exceeds 6 saturate to 6.
 *  MX_SCALE_CEIL : the least e with amax <= 6 * 2^e ("truncation-free": the scale is rounded
 *                  up to a power of two, so no element clips) [P3, "The fix ..."].
 * amax = 0 gives e = -127. e is clamped to [-127, 127]; the scale byte is e + 127. */
typedef enum { MX_SCALE_FLOOR = 0, MX_SCALE_CEIL = 1 } mx_scale_rule;

/* Rounding of v = x * 2^-e to E2M1:
 *  MX_ROUND_RNE: nearest grid point, ties to the even code, |v| >= 6 saturates to 6.
 *  MX_ROUND_SR : with lo <= |v| < hi adjacent grid points and f = (|v| - lo) / (hi - lo), the
 *                magnitude rounds up to hi iff r < f * 2^16, where r is the 16-bit random field
 *                of the element; so E[round(v)] = v up to 2^-16 of a grid step [P3, "The fix
 *                ..."; P4]. r comes from Philox4x32-10 (Salmon et al., SC'11) keyed by
 *                (seed & 0xffffffff, seed >> 32) at counter (i >> 3 as two 32-bit words, 0, 0);
 *                element i takes 16-bit field (i & 7) of the 128-bit output: word (i & 7) >> 1,
 *                low half for even i. i is the row-major index r * cols + c of the element in
 *                the SOURCE tensor, whatever the block shape or output layout. */
typedef enum { MX_ROUND_RNE = 0, MX_ROUND_SR = 1 } mx_round;

typedef struct {
  int32_t scale_rule; /* mx_scale_rule */
  int32_t round;      /* mx_round */
  int32_t hadamard;   /* 0 or 1: rotate every 32-block before scaling [P1 paragraph 2] */
  uint32_t sign_mask; /* random +/-1 diagonal D: bit j set negates block position j before the
                         transform [P4]; 0 = the deterministic transform [P2] */
  uint64_t seed;      /* Philox key for MX_ROUND_SR; ignored for MX_ROUND_RNE */
} mx_quant_opts;

/* 1x32 blocks [P1 paragraph 1; P3 "Why FP4 ..."].
 * x: [rows][ld] row-major, dtype MX_BF16 or MX_F32, ld >= cols (elements).
 * axis = 1: blocks run along a row (the common case).      codes [rows][cols/2],
 *           scales [rows][cols/32]; needs cols % 32 == 0.
 * axis = 0: blocks run down a column (e.g. along tokens for the weight gradient); the output
 *           is the K-major layout of the transpose: codes [cols][rows/2],
 *           scales [cols][rows/32]; needs rows % 32 == 0.
 * Per block, in this order: widen to fp32; if opts->hadamard, negate the positions selected by
 * sign_mask and apply the unnormalised 32-point Sylvester-Hadamard transform
 * H[i][j] = (-1)^popcount(i & j) as five fp32 butterfly stages of span 1, 2, 4, 8, 16;
 * block maximum; scale exponent; v = x * 2^-e in fp32; round; pack.
 * Alignment: x and every source row (ld * element size) 16 bytes; codes 16 bytes (a code row
 * is a multiple of 16 bytes, so any row slice of an aligned buffer qualifies); axis = 0 also
 * needs cols % 8 == 0.
 * Errors (nothing is launched): MX_ERR_NULL for a NULL x, codes, scales or opts;
 * MX_ERR_SHAPE for negative sizes, ld < cols or a multiple-of-32 / row-alignment rule;
 * MX_ERR_ARG for a bad dtype, axis or option value, or a misaligned pointer;
 * MX_ERR_LAUNCH if the kernel launch fails. rows == 0 or cols == 0 is a no-op. */
mx_status mx_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                      int32_t axis, const mx_quant_opts* opts, uint8_t* codes, uint8_t* scales,
                      void* stream);

/* 32x32 blocks, transposition invariant [P3, "The fix ...": block (i, j) of X is block (j, i)
 * of X^T with the same values, maximum and scale]. rows and cols must be multiples of 32;
 * opts->hadamard must be 0 (MX_ERR_UNSUPPORTED otherwise).
 * codes  [rows][cols/2], scales   [rows/32][cols/32]      (required)
 * codes_t[cols][rows/2], scales_t [cols/32][rows/32]      (optional, may be NULL)
 * codes_t/scales_t hold the SAME rounding decisions in the K-major layout of X^T, so the
 * transposed GEMM consumes them without re-quantization.
 * Alignment: x and every source row 16 bytes, codes and codes_t 16 bytes. Errors as for
 * mx_quantize, plus MX_ERR_NULL when exactly one of codes_t / scales_t is NULL. */
mx_status mx_quantize_2d(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                         const mx_quant_opts* opts, uint8_t* codes, uint8_t* scales,
                         uint8_t* codes_t, uint8_t* scales_t, void* stream);

/* out[r][c] = E2M1(code) * 2^(scale - 127) in fp32 ("reconstructed as P*S", [P3 "Why FP4
 * ..."]); out is [rows][cols] contiguous. block_rows = 1 reads scales [rows][cols/32];
 * block_rows = 32 reads 2-D scales [rows/32][cols/32]. If inv_hadamard (block_rows == 1 only),
 * each 32-block is then mapped back by (1/32) * D * H: the same five fp32 butterfly stages,
 * a multiply by 1/32, and the sign flips of sign_mask.
 * Alignment: codes 4 bytes, out 16 bytes; cols % 32 == 0 (rows % 32 == 0 for block_rows = 32).
 * MX_ERR_UNSUPPORTED for inv_hadamard with block_rows = 32. */
mx_status mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                        int32_t block_rows, int32_t inv_hadamard, uint32_t sign_mask, float* out,
                        void* stream);

/* Block-scaled MXFP4 GEMMs [P2 abstract; P3 "The aha ..."; P4 abstract].
 * All three compute C[m][n] = 2^alpha_exp * sum_k A[m][k] * B[n][k] with both operands packed
 * K-major (codes [rows][K/2]) and fp32 accumulation. A scale granularity g of 1 means scales
 * [rows][K/32]; g = 32 means 2-D scales [rows/32][K/32] (from mx_quantize_2d); g = 64 means
 * [rows/64][K/32] (64x64 tiles from mx_quantize_2d_blocks, each byte covering two 32-k blocks).
 * The operand's row count must be a multiple of g. alpha_exp = -5
 * undoes the factor 32 of two unnormalised Hadamard rotations along K (the caller guarantees
 * both operands used the same sign_mask); otherwise 0. out_dtype MX_BF16 (round to nearest
 * even) or MX_F32; ldc >= the output row length, in elements.
 *   fprop: Y  [T][N] = X  [T][K] . W [N][K]^T   (reduce over K)
 *   dgrad: dX [T][K] = dY [T][N] . Wt[K][N]^T   (reduce over N; Wt = W blocked along N)
 *   wgrad: dW [N][K] = dYt[N][T] . Xt[K][T]^T   (reduce over tokens T)
 * M, N multiples of 32, K a multiple of 32; the operand codes and C 16-byte aligned, ldc a
 * multiple of 8 elements. One 256-row operand tile must stay below 2 GiB (256 * K / 2 < 2^31).
 * Errors (nothing is launched): MX_ERR_SHAPE, MX_ERR_ARG (granularity, out_dtype, alpha_exp
 * outside [-126, 127], alignment), MX_ERR_NULL; MX_ERR_LAUNCH if the launch fails or the shape
 * exceeds the 32-bit offsets above. M == 0 or N == 0 is a no-op; K == 0 writes zeros.
 * Accuracy: the E2M1 x E2M1 products with their scales are summed exactly within one 64-k
 * matrix instruction, and the K/64 instruction results are added in fp32, one accumulator per
 * output: the error is that of those additions, at worst (K/64) * 2^-24 * sum_k |a_k b_k|, and
 * within the tolerance |C - exact| <= 2^-20 * sum_k |a_k b_k| on the tested workloads (K up to
 * 28672) for fp32 output; bf16 output is the rounding of such a value. */
mx_status mx_gemm_fprop(const uint8_t* xq, const uint8_t* xs, int32_t gx, const uint8_t* wq,
                        const uint8_t* ws, int32_t gw, int64_t T, int64_t N, int64_t K,
                        int32_t alpha_exp, int32_t out_dtype, void* y, int64_t ldy, void* stream);
mx_status mx_gemm_dgrad(const uint8_t* dyq, const uint8_t* dys, int32_t gdy, const uint8_t* wtq,
                        const uint8_t* wts, int32_t gwt, int64_t T, int64_t K, int64_t N,
                        int32_t alpha_exp, int32_t out_dtype, void* dx, int64_t ldx, void* stream);
mx_status mx_gemm_wgrad(const uint8_t* dytq, const uint8_t* dyts, int32_t gdy, const uint8_t* xtq,
                        const uint8_t* xts, int32_t gx, int64_t N, int64_t K, int64_t T,
                        int32_t alpha_exp, int32_t out_dtype, void* dw, int64_t ldw, void* stream);

/* Fprop with the output quantized in the epilogue [P1 paragraph 1: the Walsh-Hadamard rotation
 * and stochastic rounding run inside the GEMM epilogue, before the output tile is packed to
 * 4 bits]. Y = 2^alpha_exp * X . W^T is formed in fp32 exactly as mx_gemm_fprop forms it and,
 * instead of being stored, quantized as mx_quantize(Y, axis = 1, opts) would quantize that fp32
 * tensor: 1x32 blocks along N, yq [T][N/2], ys [T][N/32], stochastic-rounding index t * N + n.
 * Arguments as for mx_gemm_fprop; opts as for mx_quantize. K must be a positive multiple of 128
 * (MX_ERR_UNSUPPORTED otherwise); yq 4-byte aligned. The fp32 values are not bit-identical to
 * those of a separate fp32 GEMM with a different accumulation order, so the codes equal the
 * quantization of some fp32 Y within the GEMM bound of mx_gemm_fprop. */
mx_status mx_gemm_fprop_quant(const uint8_t* xq, const uint8_t* xs, int32_t gx, const uint8_t* wq,
                              const uint8_t* ws, int32_t gw, int64_t T, int64_t N, int64_t K,
                              int32_t alpha_exp, const mx_quant_opts* opts, uint8_t* yq,
                              uint8_t* ys, void* stream);

/* MXFP8 [P3, "The fix, and its supporting cast": the query and key projections are quantized
 * in MXFP8 rather than FP4]. Blocks, scales, options and stochastic-rounding fields are those
 * of the MXFP4 path; the elements are 8-bit OCP floating point (the pages do not fix the
 * encoding):
 *  MX_E4M3: sign, 4 exponent bits (bias 7), 3 mantissa bits; exponent 15 with mantissa 7 is
 *           NaN and there is no infinity, so the largest magnitude is 448 = 1.75 * 2^8;
 *  MX_E5M2: sign, 5 exponent bits (bias 15), 2 mantissa bits; exponent 31 is inf / NaN, the
 *           largest magnitude is 57344 = 1.75 * 2^15.
 * Exponent field 0 is subnormal. A code is one byte, the sign in bit 7 (copied from the value).
 * Scale exponent, with amax = m * 2^E, m in [1, 2): MX_SCALE_FLOOR e = E - emax (emax = 8 or
 * 15, the exponent of the largest magnitude; values beyond it saturate); MX_SCALE_CEIL the
 * least e with amax <= largest * 2^e. MX_ROUND_RNE rounds to the nearest representable value
 * with ties to the even code; MX_ROUND_SR rounds up iff r < f * 2^16 as for E2M1; |v| >= the
 * largest magnitude gives the largest code. */
typedef enum { MX_E4M3 = 0, MX_E5M2 = 1 } mx_fp8_format;

/* 1x32 MXFP8 quantize; arguments as for mx_quantize plus fmt (mx_fp8_format).
 * axis = 1: codes [rows][cols] (one byte per element), scales [rows][cols/32];
 * axis = 0: codes [cols][rows], scales [cols][rows/32] (the K-major layout of the transpose).
 * Alignment: x and source rows 16 bytes; codes 8 bytes (axis = 1) or 16 bytes (axis = 0);
 * axis = 0 also needs cols % 8 == 0. Errors as for mx_quantize; MX_ERR_ARG for a bad fmt. */
mx_status mx_quantize_mxfp8(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                            int32_t axis, int32_t fmt, const mx_quant_opts* opts, uint8_t* codes,
                            uint8_t* scales, void* stream);

/* MXFP8 GEMM on gfx950's block-scaled matrix cores: C[m][n] = 2^alpha_exp * sum_k A[m][k] *
 * B[n][k], fp32 accumulation, with A codes [M][K] of format afmt and B codes [N][K] of format
 * bfmt (one byte per element, K-major), scales [M][K/32] and [N][K/32]. Fprop, Dgrad and Wgrad
 * are this call on the operands of the respective orientation (as for the MXFP4 calls).
 * M, N multiples of 32; K a positive multiple of 128 (MX_ERR_UNSUPPORTED otherwise, except
 * K == 0, which writes zeros); operand codes and C 16-byte aligned; ldc a multiple of 8
 * elements; 256 * K < 2^31. out_dtype, alpha_exp and errors as for mx_gemm_fprop.
 * Accuracy: |C - exact| <= 2^-10 * sum_k |a_k b_k| for fp32 output (K <= 65536), and bf16
 * output is the rounding of a value within that bound. The bound is the matrix core's: within
 * each group of 8 consecutive products of one 64-k instruction, every product is truncated
 * toward zero to a multiple of 2^(E - 13), 2^E the leading power of two of the group's largest
 * product, and the truncated products are summed exactly and rounded to fp32 once (derived
 * from single-instruction measurements on gfx950). A group loses less than 7 * 2^-13 of its
 * largest product, and the K/64 fp32 additions of the instruction results add at most
 * (K/64) 2^-24 sum |a_k b_k|. (MXFP4 products are summed exactly: the 2^-20 rule of
 * mx_gemm_fprop.) */
mx_status mx_gemm_mxfp8(const uint8_t* aq, const uint8_t* as, int32_t afmt, const uint8_t* bq,
                        const uint8_t* bs, int32_t bfmt, int64_t M, int64_t N, int64_t K,
                        int32_t alpha_exp, int32_t out_dtype, void* c, int64_t ldc, void* stream);

/* Square tiles of other sizes [P3, "The fix ...": Table 4 compares 8x8, 32x32 and 64x64
 * blocks, the smaller with more scale metadata]. As mx_quantize_2d with tile edge block = 8, 32
 * or 64: one scale per tile from the tile maximum, every element rounded once and written to
 * both code layouts (codes [rows][cols/2], codes_t [cols][rows/2], as for mx_quantize_2d).
 * Scales: block = 8: scales [rows/8][cols/8], scales_t [cols/8][rows/8];
 *         block = 32: exactly mx_quantize_2d;
 *         block = 64: in the layout the GEMMs read with g = 64, scales [rows/64][cols/32] and
 *                     scales_t [cols/64][rows/32], each tile's byte stored for both of its
 *                     32-wide halves.
 * 8x8 tiles cannot feed the block-scaled matrix cores, whose scale blocks are 32 elements along
 * K; they are a quantization (and mismatch) format here. rows and cols must be multiples of
 * max(block, 32); opts->hadamard must be 0. Alignment: x and source rows 16 bytes, codes and
 * codes_t 16 bytes, scales and scales_t 4 bytes. Errors as for mx_quantize_2d, plus MX_ERR_ARG
 * for another block. */
mx_status mx_quantize_2d_blocks(const void* x, int32_t dtype, int64_t rows, int64_t cols,
                                int64_t ld, int32_t block, const mx_quant_opts* opts,
                                uint8_t* codes, uint8_t* scales, uint8_t* codes_t,
                                uint8_t* scales_t, void* stream);

/* Scale-difference map of 1x32 blocking [P3, "The aha: transposition scrambles the blocks",
 * Figure 1]: map[r][c] = e_row - e_col, where e_row is the scale exponent (scale_rule, as for
 * mx_quantize) of the 1x32 block along row r that holds element (r, c), how X enters the forward
 * product, and e_col that of the 1x32 block down column c, how X enters the transposed product.
 * int8, saturated to [-127, 127]; -128 where either block's maximum is not finite. With 32x32
 * tiles the two exponents are one and the same, so the map of that quantizer is zero.
 * x: [rows][ld] bf16 or fp32, rows and cols multiples of 32; map [rows][cols] contiguous, 8-byte
 * aligned. Errors: MX_ERR_SHAPE, MX_ERR_ARG (dtype, scale_rule, alignment), MX_ERR_NULL. */
mx_status mx_scale_mismatch_map(const void* x, int32_t dtype, int64_t rows, int64_t cols,
                                int64_t ld, int32_t scale_rule, int8_t* map, void* stream);

/* RMS norm with the residual's addition, row by row over x [rows][cols]:
 *   s = x + residual (in fp32, rounded to dtype; s = x when residual is NULL),
 *   rho = 1 / sqrt(mean(s^2) + eps),   y = s * rho * gamma.
 * x, residual, sum and y have type dtype (MX_BF16 or MX_F32) and leading dimensions ldx, ldr, lds
 * and ldy in elements; gamma [cols] has type gamma_dtype. sum receives s, the new residual stream;
 * rstd [rows] (fp32) receives rho, which mx_rmsnorm_backward reads. residual, sum and rstd may be
 * NULL (ldr and lds are then ignored). The norm takes the rounded s, so it can be recomputed from
 * the stored sum. The sum of squares, rho and y are formed in 64 bits and every output is rounded
 * once, to the nearest value, so a row's outputs depend on that row alone (not on how many rows
 * share the call). A row that holds an infinity or a NaN gives NaNs (or zeros beside an infinity),
 * as the formula does. sum and y may each be x or residual itself (same leading dimension), not
 * both the same one; rows of theirs that share memory in another way are refused.
 * cols is a multiple of 32 and at most 32768 (MX_ERR_UNSUPPORTED beyond); pointers to rows and
 * gamma 16-byte aligned, rstd 4-byte, every leading dimension * element size a multiple of 16
 * bytes. Errors (nothing is launched): MX_ERR_NULL for a NULL x, gamma or y; MX_ERR_SHAPE for
 * negative sizes, a leading dimension below cols or the multiple-of rules; MX_ERR_ARG for a bad
 * type, a misaligned pointer, an eps that is negative or not finite, or outputs that overlap an
 * operand. rows == 0 or cols == 0 is a
 * no-op. */
mx_status mx_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr, int32_t dtype,
                     int64_t rows, int64_t cols, const void* gamma, int32_t gamma_dtype, float eps,
                     void* sum, int64_t lds, void* y, int64_t ldy, float* rstd, void* stream);

/* mx_rmsnorm with y quantized in 1x32 blocks along the row, MXFP4 or MXFP8: codes, scales, opts
 * and fmt as for mx_quantize (axis = 1) and mx_quantize_mxfp8 (axis = 1), stochastic-rounding
 * index r * cols + c. The values that are quantized are the unrounded y: with opts->hadamard the
 * signs and the 32-point transform are applied in 64 bits, and each value is rounded once, to its
 * code. y is optional here (NULL: only the codes are written; ldy ignored). Alignment of codes:
 * 16 bytes (MXFP4), 8 bytes (MXFP8). Errors as for mx_rmsnorm, plus those of the quantizers for
 * opts, fmt, codes and scales. */
mx_status mx_rmsnorm_quant(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                           int32_t dtype, int64_t rows, int64_t cols, const void* gamma,
                           int32_t gamma_dtype, float eps, void* sum, int64_t lds, void* y,
                           int64_t ldy, float* rstd, const mx_quant_opts* opts, uint8_t* codes,
                           uint8_t* scales, void* stream);
mx_status mx_rmsnorm_quant_mxfp8(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                 int32_t dtype, int64_t rows, int64_t cols, const void* gamma,
                                 int32_t gamma_dtype, float eps, void* sum, int64_t lds, void* y,
                                 int64_t ldy, float* rstd, int32_t fmt, const mx_quant_opts* opts,
                                 uint8_t* codes, uint8_t* scales, void* stream);

/* Backward pass of mx_rmsnorm (the quantizers are the identity, straight-through). From dy (the
 * gradient of y), dsum (the gradient that reaches the stored sum from further on; may be NULL), s
 * (the stored sum) and rstd:  u = dy * gamma, z = s * rstd, c = mean over the row of u * z,
 *   dx = rstd * (u - z * c) + dsum     (the gradient of x and of residual alike),
 *   dgamma[j] = sum over the rows of dy * z   (fp32; may be NULL).
 * fp32 throughout, dx rounded to dtype at the end; the order of every sum is fixed by the sizes.
 * dx may be dsum itself (same leading dimension), or without dgamma dy or s. With dgamma, workspace
 * holds at least mx_rmsnorm_backward_workspace(rows, cols) bytes (0 for small tensors of few
 * rows), 16-byte aligned; its contents are scratch, and calls that may run at the same time need
 * one each. Sizes, alignment and errors as for mx_rmsnorm; MX_ERR_ARG also for a workspace that is
 * too small and for dx that shares memory with dy or s when there is a dgamma. rows == 0 writes a
 * zero dgamma. */
int64_t mx_rmsnorm_backward_workspace(int64_t rows, int64_t cols);
mx_status mx_rmsnorm_backward(const void* dy, int64_t lddy, const void* dsum, int64_t ldds,
                              const void* s, int64_t lds, int32_t dtype, int64_t rows,
                              int64_t cols, const void* gamma, int32_t gamma_dtype,
                              const float* rstd, void* dx, int64_t lddx, float* dgamma,
                              void* workspace, int64_t workspace_bytes, void* stream);

/* Product of a few tokens with MXFP4 weights, the activations not quantized (decoding):
 *   y[t][n] = 2^alpha_exp * sum_k x'[t][k] * W[n][k]
 * x: [T][ldx], dtype MX_BF16 or MX_F32; W: codes wq [N][K/2] and scales ws of granularity gw (1,
 * 32 or 64), as for mx_gemm_fprop; y: [T][ldy], out_dtype. With hadamard = 1 every 32-block of x
 * is rotated like mx_quantize rotates it (signs of sign_mask, then the transform, in fp32), for
 * weights that were quantized rotated; alpha_exp = -5 then undoes the factor 32. T and N are
 * arbitrary (N a multiple of gw), K a multiple of 32. x and its rows (ldx * element size) 16-byte
 * aligned, wq 16-byte aligned, y aligned to its elements, ldy >= N. The weights are read once for
 * every 16 to 64 tokens; many more tokens are the GEMMs' work.
 * workspace: mx_gemv_workspace(...) bytes, 16-byte aligned, make many products of several tokens
 * faster (sums over parts of K); 0 bytes are wanted for one token. Its contents are scratch, and
 * calls that may run at the same time need one each. NULL does without, with other roundings.
 * Accuracy: fp32 accumulation. The products are exact, sums of 128 of them are formed by the
 * matrix core, which drops what lies below 2^-24 of a sum's largest term, and joined in fp32:
 * |y - exact| <= (160 + K / 128) * 2^-24 * sum_k |x'_k W_k| before the rounding to bf16. bf16
 * tokens that are rotated for a bf16 y keep 16 bits of each x' (another 2^-17 of the sum), and of
 * fp32 or rotated values what lies below bf16's least subnormal, 2^-133, is rounded away. A weight
 * beyond bf16's range, 2^128 or more (scale bytes 253 and 254), counts as infinity: with fp32 or
 * rotated tokens, or zeros in x, its output may be NaN. Scale byte 255 is NaN.
 * Errors (nothing is launched): MX_ERR_SHAPE, MX_ERR_ARG (types, granularity, hadamard, alpha_exp
 * outside [-126, 127], alignment, a workspace that is too small, a y that overlaps x), MX_ERR_NULL,
 * MX_ERR_UNSUPPORTED (N above 2^26 or T above 2^19 rows, whatever the other sizes). T == 0 or N == 0 is a no-op; K == 0 writes zeros. */
int64_t mx_gemv_workspace(int32_t dtype, int64_t T, int64_t N, int64_t K, int32_t hadamard,
                          int32_t out_dtype);
mx_status mx_gemv(const void* x, int32_t dtype, int64_t ldx, const uint8_t* wq, const uint8_t* ws,
                  int32_t gw, int64_t T, int64_t N, int64_t K, int32_t hadamard,
                  uint32_t sign_mask, int32_t alpha_exp, int32_t out_dtype, void* y, int64_t ldy,
                  void* workspace, int64_t workspace_bytes, void* stream);

/* A paged cache of keys and values in 8 bits (decoding), and the sequences that one call is about.
 * Codes are E4M3 or E5M2 (fmt, as for mx_quantize_mxfp8); one E8M0 scale serves a block of 32 tokens
 * of one head. A page holds page_size tokens (a multiple of 32, at most 2048) of every head:
 *   kq [n_pages][heads][page_size][dim]          a token's channels next to one another
 *   vq [n_pages][heads][page_size / 32][dim][32] a channel's 32 tokens next to one another
 *   ks, vs [n_pages][heads][page_size / 32]
 * pages [seqs][table_width]: page p of a sequence holds its tokens p * page_size and following. An
 * entry outside [0, n_pages) is no page: its tokens are not written, read as zeros and not attended
 * to; so are tokens beyond the table. Sequences may share pages that nobody writes to.
 * lengths [seqs]: tokens of each sequence, those of the call among them. offsets [seqs + 1]: rows
 * offsets[b] .. offsets[b + 1] - 1 of the call's T rows are the newest tokens of sequence b, the last
 * of them at position lengths[b] - 1; NULL: one row each, row b (T == seqs then). Rows that belong to
 * no sequence (before the first, behind the last) are neither read nor written. offsets must not
 * fall; pages, lengths and offsets are device memory, whose contents are not checked, but no content
 * leads outside the tensors.
 * dim is 64, 128, 192 or 256. kq and vq 16-byte aligned, the tables 4-byte. */
typedef struct {
  uint8_t* kq;
  uint8_t* ks;
  uint8_t* vq;
  uint8_t* vs;
  const int32_t* pages;
  const int32_t* lengths;
  const int32_t* offsets;
  int64_t n_pages, seqs, table_width;
  int32_t heads, dim, page_size, fmt;
} mx_cache;

/* Rows of keys, values, queries or outputs of a call: [T][heads][dim], `token` and `head` elements
 * from one token and from one head to the next; channels contiguous. Pointers 16-byte aligned, both
 * distances multiples of 16 bytes, at least dim (heads), and neither makes rows overlap. */
typedef struct {
  const void* p;
  int64_t token, head;
} mx_rows;

/* Quantizes the keys and values of a call's T rows (dtype MX_BF16 or MX_F32) into the cache, round to
 * nearest even. A block that receives tokens takes the scale byte of their largest magnitude
 * (scale_rule, as for mx_quantize_mxfp8), or keeps its own where it already holds older tokens of the
 * sequence and that is larger; where it grows the older codes are rounded again, to code * 2^(old -
 * new). Scales are powers of two, so that changes a code only below the format's least normal. A
 * token with an infinity or NaN makes its block's scale 0xFF and its tokens' codes zero, for good.
 * Slots of a block behind its last token keep what they hold. Tokens that a later call writes over
 * (drafts that were refused: lengths may shrink) leave the scale that they made to a block that holds
 * older tokens too, and those the rounding to it, or the zeros of a 0xFF; a block that is written from its
 * first slot on starts anew. Two rows of a call must not fall into one block from two sequences.
 * Errors (nothing is launched): MX_ERR_NULL; MX_ERR_SHAPE (negative sizes, T != seqs without
 * offsets, a distance below the rules); MX_ERR_ARG (dtype, fmt, scale_rule, page_size, alignment,
 * rows inside the cache); MX_ERR_UNSUPPORTED (dim, more than 2^20 sequences, 2^24 rows, 65535 heads
 * or 2^31 - 1 pages). T == 0 or heads == 0 is a no-op. */
mx_status mx_cache_write(const mx_rows* k, const mx_rows* v, int32_t dtype, int64_t T,
                         const mx_cache* cache, int32_t scale_rule, void* stream);

/* The T newest tokens' keys and values back as code * 2^(scale - 127), rounded to dtype once; NaN
 * where the scale is 0xFF, zeros where there is no page, or no token (more rows than the sequence
 * has). Errors as for mx_cache_write, and MX_ERR_ARG for k and v that overlap each other or the
 * tables. */
mx_status mx_cache_read(const mx_rows* k, const mx_rows* v, int32_t dtype, int64_t T,
                        const mx_cache* cache, void* stream);

/* Causal attention of the T rows' q_heads query heads over the cache: query head h reads head
 * h / (q_heads / heads) of it, and the row of position i the tokens 0 .. i:
 *   out = sum_j p_j v_j,  p = softmax(scale * q . k_j).
 * q and out: dtype, [T][q_heads][dim]; lse (optional, [T][q_heads] fp32, contiguous): the natural
 * logarithm of the sum of exp(scale * q . k_j). A row that sees no token gets zeros and -infinity.
 * Keys and values are exact (down to bf16's least subnormal, 2^-133); q . k is formed in fp32 from
 * exact products (bf16 q, or fp32 q as three bf16 terms); the statistics and sums are fp32; the
 * probabilities keep 16 bits for a bf16 output and 24 for fp32. Tokens whose scale is 0xFF make the rows
 * that see them NaN (their lse with that of the keys), and only those. Codes of NaN or infinity, which
 * mx_cache_write does not leave, are not provided for.
 * Lengths are read on the device, and long contexts are divided there: a call may be captured and
 * replayed with other lengths, pages and offsets. The order of the sums depends on the lengths of all
 * sequences of the call.
 * workspace: mx_cache_attention_workspace(...) bytes, 16-byte aligned, scratch: calls that may run at
 * the same time need one each (or -1 for arguments that the call refuses).
 * Errors as for mx_cache_write; MX_ERR_SHAPE for q_heads that is no multiple of heads; MX_ERR_ARG for
 * a scale that is not finite, a workspace that is too small, and an out or lse that overlaps q, the
 * other or the tables; MX_ERR_UNSUPPORTED for more than 65535 query heads, 2^30 rows of all of them, or
 * 2^31 steps of a head if every sequence filled its table (a step is 64 tokens, 32 for dim above 128,
 * by 16, 32 or 64 rows). One call takes one of these numbers of rows, by the sequences' average:
 * prompts and single tokens are faster in calls of their own. */
int64_t mx_cache_attention_workspace(int64_t T, int64_t q_heads, const mx_cache* cache);
mx_status mx_cache_attention(const mx_rows* q, const mx_rows* out, float* lse, int32_t dtype,
                             int64_t T, int64_t q_heads, float scale, const mx_cache* cache,
                             void* workspace, int64_t workspace_bytes, void* stream);

/* Low-rank adapters of many requests beside a shared projection (mx_gemv's y, or any other base):
 *   out[t] = base[t] + scaling[e] * B[e] (A[e] x[t]),   e = index[t],
 * a [adapters][rank][K] and b [adapters][N][rank], contiguous, of x's type (MX_BF16 or MX_F32); index
 * [T] int32 in any order: a token whose index is outside [0, adapters) gets base alone. scaling
 * [adapters] fp32 may be NULL (1), and base may be NULL (0). x [T][ldx], base [T][ldb] and out [T][ldo]
 * have types and leading dimensions of their own; out may be base itself. K and rank are multiples of
 * 8, rank at most 128, T, N and the number of adapters arbitrary. x and its rows 16-byte aligned, a
 * and b 16-byte, base and out aligned to their elements (rows at 16-byte addresses are faster).
 * A x, the sum over the rank, scaling and the addition are fp32, rounded once, to out's type; A x of
 * bf16 operands has exact products. A token's output depends on its own adapter and the call's sizes,
 * not on the other tokens.
 * workspace: mx_lora_workspace(...) bytes (0 for a few tokens), 16-byte aligned, scratch: calls that
 * may run at the same time need one each.
 * Errors (nothing is launched): MX_ERR_SHAPE, MX_ERR_ARG (types, alignment, a workspace that is too
 * small, an out that overlaps x, a, b, index, scaling or, without being it, base), MX_ERR_NULL,
 * MX_ERR_UNSUPPORTED (rank above 128, T above 2^21, N, K or adapters above 2^26). T == 0 or N == 0 is
 * a no-op; no adapters, or K == 0 or rank == 0, leave base alone. */
int64_t mx_lora_workspace(int32_t dtype, int64_t T, int64_t N, int64_t K, int64_t adapters,
                          int64_t rank);
mx_status mx_lora(const void* x, int32_t dtype, int64_t ldx, const void* a, const void* b,
                  int64_t adapters, int64_t rank, const int32_t* index, const float* scaling,
                  const void* base, int32_t base_dtype, int64_t ldb, int64_t T, int64_t N, int64_t K,
                  int32_t out_dtype, void* out, int64_t ldo, void* workspace,
                  int64_t workspace_bytes, void* stream);

/* Human-readable name of a status code (static storage). */
const char* mx_status_string(int32_t status);

/* Library version, major * 10000 + minor * 100 + patch. */
int32_t mx_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MX_H */
