/*
 * nvfp4_amd_fp8.h -- C ABI of the library's 8-bit operators: the gated feed-forward
 * block of a layer that a 4-bit run keeps out of NVFP4, with its norm, in E4M3 with
 * one power-of-two scale per block of 128; dropout; and low-rank adapters beside a
 * frozen 8-bit projection.
 *
 * Quantized tensor.  For a logical tensor [rows][cols], cols the contraction
 * dimension, with KB = ceil(cols / 128):
 *   codes  : E4M3 (OCP "FN") bytes [rows][128 KB]; the columns past cols hold zeros;
 *   scales : E8M0 bytes (the value 2^(byte - 127)), K-block-major: one per 1 x 128
 *            block, [KB][rows rounded up to 16] (the padding is not read for a result),
 *            or with two_d one per 128 x 128 tile, [KB][ceil(rows / 128)].
 *   scale  = the smallest 2^e with amax <= 448 * 2^e, e in [-126, 127], amax the
 *            block's largest magnitude (1 for a block of zeros);
 *   code   = E4M3(v / scale), nearest-even (v / scale is exact but for underflow).
 * The K-block-major scales put the 128 or 256 scales that one K stage of a product
 * reads side by side, and transposing a tile-scaled tensor transposes its scales.
 *
 * Memory, streams and errors are those of nvfp4_amd.h: the caller owns every buffer,
 * nothing is allocated, all work is enqueued on the given stream in order, arguments
 * are checked before anything is enqueued.  Results do not depend on timing: no
 * floating-point atomics, partial sums are joined in a fixed order.  Inputs are
 * expected to be finite; an infinity or NaN in a quantizer's input becomes the NaN
 * code and leaves the other elements' blocks as they are (an infinity raises its own
 * block's scale).  In the norm and the gated block a token's NaNs leave the other tokens'
 * rows (yq, hq, dgq, duq, y, dx) as they are and reach only what sums over the tokens
 * (the weights' gradients); the padding holds zeros all the same.
 *
 * Limits: rows and cols at most 16776960, and at most that many 128 x 128 tiles
 * (FP4_ERR_SHAPE otherwise); element counts and byte offsets may pass 2^32.
 */
#ifndef NVFP4_AMD_FP8_H
#define NVFP4_AMD_FP8_H

#include "nvfp4_amd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* codes 16-byte aligned, scales 16-byte aligned; both may be NULL for an empty tensor. */
typedef struct fp8_tensor {
  uint8_t *codes;
  uint8_t *scales;
  int64_t rows;
  int64_t cols;
  int32_t two_d;
} fp8_tensor;

/* Bytes of the codes and scales of a rows x cols tensor.  Pure host arithmetic.
 * FP4_ERR_NULL, FP4_ERR_SHAPE. */
FP4_API fp4_status fp8_tensor_bytes(int64_t rows, int64_t cols, int32_t two_d, size_t *codes_bytes,
                                    size_t *scales_bytes);

/* Quantizes x [rows][cols] (row stride ld elements, any alignment of its elements)
 * into q (x's layout) and q_t (x^T, [cols][rows], blocks down the columns of x) in one
 * read of x.  Either may be NULL, not both; both take the same two_d, and with it the
 * same tile scales.  x must not overlap the outputs.
 * Errors: FP4_ERR_NULL, FP4_ERR_DTYPE, FP4_ERR_SHAPE (ld < cols), FP4_ERR_ALIGN (x not
 * aligned to its element, outputs as above), FP4_ERR_MISMATCH (a descriptor's shape,
 * or two_d that differs between them), FP4_ERR_HIP. */
FP4_API fp4_status fp8_quantize(const void *x, fp4_dtype dtype, int64_t rows, int64_t cols, int64_t ld,
                                const fp8_tensor *q, const fp8_tensor *q_t, hipStream_t stream);

/* Root-mean-square norm with the residual's addition and a quantized output:
 *   h    = x + residual, rounded to dtype (x itself without a residual)
 *   rstd = 1 / sqrt(mean(h^2) + eps), rounded to binary32
 *   y    = h * rstd * weight    ->  yq (1 x 128 blocks along the width)
 *                               ->  yq_t (y^T, blocks along the tokens; nullable)
 * x, residual, h [rows][cols] with row strides ldx, ldr, ldh; weight [cols] binary32.
 * residual and h are both NULL or both given; h may be x or residual (same stride).
 * rstd [rows] is nullable without yq_t, which reads it.  eps > 0.
 * Errors: FP4_ERR_NULL, FP4_ERR_DTYPE, FP4_ERR_SHAPE (strides, eps), FP4_ERR_ALIGN,
 * FP4_ERR_MISMATCH, FP4_ERR_MODE (a tile-scaled output), FP4_ERR_HIP. */
FP4_API fp4_status fp8_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, fp4_dtype dtype,
                                int64_t rows, int64_t cols, const float *weight, float eps, void *h, int64_t ldh,
                                const fp8_tensor *yq, const fp8_tensor *yq_t, float *rstd, hipStream_t stream);

/* Its gradient, from dy (the gradient of y, straight through the quantization), h and
 * rstd of the forward call and dh (the gradient that reaches h by the residual stream;
 * nullable):
 *   hhat = h * rstd,  v = dy * weight
 *   dx      = dh + rstd * (v - hhat * mean(v * hhat))      (also the residual's)
 *   dweight = sum over rows of dy * hhat                   (binary32, [cols])
 * dy, h, dh, dx [rows][cols] contiguous, of dtype; dx may be dy or dh.  ws:
 * fp8_rms_norm_ws_bytes(rows, cols) bytes, 16-byte aligned, overwritten.
 * Errors: FP4_ERR_NULL, FP4_ERR_DTYPE, FP4_ERR_SHAPE, FP4_ERR_ALIGN,
 * FP4_ERR_WORKSPACE, FP4_ERR_HIP. */
FP4_API fp4_status fp8_rms_norm_backward(const void *dy, const void *h, const void *dh, fp4_dtype dtype, int64_t rows,
                                         int64_t cols, const float *weight, const float *rstd, void *dx,
                                         float *dweight, void *ws, size_t ws_bytes, hipStream_t stream);
FP4_API fp4_status fp8_rms_norm_ws_bytes(int64_t rows, int64_t cols, size_t *bytes);

/* Dropout.  Of a tensor [rows][cols], element (r, c) is kept where its 16 random bits are at
 * least T = 2^16 p, rounded, and is then multiplied by 2^16 / (2^16 - T) (binary32), so that
 * its mean is its value; what is not kept counts as 0, also an infinity or NaN.  The bits are
 * half-word c & 7 (word (c & 7) / 2, low half first) of Philox4x32-10 with counter (g as two
 * words, o as two words) and key seed, g = r * ceil(cols / 8) + c / 8, o = offset + *step
 * (offset alone where step is NULL), both modulo 2^64.  Nothing of the mask is stored: every
 * call that is given the same p, seed, offset and *step and a tensor of the same shape, of
 * whatever strides, uses the same one.  step is device memory, 8-byte aligned, read when the
 * call's kernels run: a captured graph whose step is advanced between its replays draws a new
 * mask in each.  0 <= p < 1 - 2^-17 (at most T = 2^16 - 1).
 * offset + *step is one number: offset 1 at step 2 is offset 2 at step 1, so the offsets of a
 * run's dropouts belong further apart than its steps (layer << 40, say).  And nvfp4_amd.h's
 * stochastic rounding draws the same bits of the same seed and offset where cols is a multiple
 * of 8: the two take seeds, or offsets, of their own. */
typedef struct fp8_dropout_config {
  double p;
  uint64_t seed;
  uint64_t offset;
  const uint64_t *step;
} fp8_dropout_config;

/* y = residual + dropout(x), rounded once to dtype (dropout(x) alone without a residual,
 * which is also the gradient's call: dx = dropout(dy)).  x, residual, y [rows][cols] with row
 * strides ldx, ldr, ldy; y may be x or residual (same stride).
 * Errors: FP4_ERR_NULL, FP4_ERR_DTYPE, FP4_ERR_SHAPE (strides, p), FP4_ERR_ALIGN,
 * FP4_ERR_HIP. */
FP4_API fp4_status fp8_dropout(const void *x, int64_t ldx, const void *residual, int64_t ldr, fp4_dtype dtype,
                               int64_t rows, int64_t cols, const fp8_dropout_config *drop, void *y, int64_t ldy,
                               hipStream_t stream);

/* fp8_rms_norm with x dropped out before the residual's addition, h = residual + dropout(x)
 * rounded to dtype; residual and h are given.  The rest, and the errors, as there
 * (FP4_ERR_SHAPE also for p). */
FP4_API fp4_status fp8_dropout_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, fp4_dtype dtype,
                                        int64_t rows, int64_t cols, const fp8_dropout_config *drop,
                                        const float *weight, float eps, void *h, int64_t ldh, const fp8_tensor *yq,
                                        const fp8_tensor *yq_t, float *rstd, hipStream_t stream);
/* Its gradient: dresidual is fp8_rms_norm_backward's dx, and dx = dropout(dresidual) before
 * that is rounded.  Each of dx and dresidual may be dy or dh.  ws and errors as there. */
FP4_API fp4_status fp8_dropout_rms_norm_backward(const void *dy, const void *h, const void *dh, fp4_dtype dtype,
                                                 int64_t rows, int64_t cols, const fp8_dropout_config *drop,
                                                 const float *weight, const float *rstd, void *dx, void *dresidual,
                                                 float *dweight, void *ws, size_t ws_bytes, hipStream_t stream);

/* C[m][n] = sum_k deq(A)[m][k] * deq(B)[n][k], A [M][K], B [N][K], each with either
 * kind of scales, C of c_dtype with row stride ldc.
 * flags: 0 sums in binary32 throughout: the operands, exact in bf16 with their scales,
 *   go through the bf16 matrix instruction (magnitudes under 2^-126 may count as 0).
 *   FP8_GEMM_FAST takes the 8-bit matrix instruction, at twice the rate.  It cuts the
 *   eight products of k = 8 t .. 8 t + 7 off at 2^-13 of their largest power of two
 *   (towards zero) before their sum enters the binary32 accumulator: a relative error
 *   (2-norm) of C of about 1.5e-5 for normally and 2.6e-5 for Laplace distributed
 *   operands, against 1.7e-3 for the rounding of C to bf16.
 * ws: fp8_gemm_ws_bytes(M, N, K) bytes (0 for many shapes), 16-byte aligned,
 * overwritten; with less (or NULL, 0) the product runs without splitting K.  The plan is
 * fixed for (M, N, K), the flags, the workspace's size and the GPU's CU count.
 * Errors: FP4_ERR_MODE (unknown flags), FP4_ERR_NULL, FP4_ERR_MISMATCH (K differs),
 * FP4_ERR_SHAPE (ldc < N), FP4_ERR_DTYPE, FP4_ERR_ALIGN, FP4_ERR_HIP. */
#define FP8_GEMM_FAST (1u << 0)
FP4_API fp4_status fp8_gemm(const fp8_tensor *a, const fp8_tensor *b, void *c, fp4_dtype c_dtype, int64_t ldc,
                            uint32_t flags, void *ws, size_t ws_bytes, hipStream_t stream);
FP4_API fp4_status fp8_gemm_ws_bytes(int64_t M, int64_t N, int64_t K, size_t *bytes);

/* The gated feed-forward block, forward, for M tokens, width K and inner width F:
 *   g = x wg^T, u = x wu^T, each rounded to bf16
 *   h = silu(g) * u (binary32 from the rounded g and u)  ->  hq [M][F], 1 x 128 blocks
 *   y = hq wd^T, bf16 [M][K] (row stride ldy)
 * flags: those of fp8_gemm, for all of the block's products; the call without them takes 0,
 *   sums in binary32.  FP8_GEMM_FAST is the faster (twice, on many tokens) and the less
 *   exact: what it cuts off a sum moves some of the values that are rounded to bf16 and
 *   then to 8 bits to the next step.  y and the gradients are then off by 1.8e-3 to 2.4e-3
 *   (relative 2-norm, normally and Laplace distributed operands of many sizes), and with
 *   flags 0 by 1.66e-3, which is their own rounding to bf16.
 * xq [M][K] (1 x 128), wg, wu [F][K] and wd [K][F] (tile scales).  g and u [M][F] bf16
 * contiguous receive the projections for the backward pass; both NULL where none
 * follows.  ws: fp8_ffn_ws_bytes(M, K, F) bytes, 16-byte aligned, overwritten; the call
 * with flags takes fp8_ffn_fprop_ws_bytes(M, K, F, keep, flags), keep being whether it is
 * given g and u: often much less, as dh of the backward pass has no place in it.
 * Errors: FP4_ERR_MODE (unknown flags), FP4_ERR_NULL, FP4_ERR_MISMATCH (shapes, kinds of
 * scales), FP4_ERR_SHAPE, FP4_ERR_ALIGN, FP4_ERR_WORKSPACE, FP4_ERR_HIP. */
FP4_API fp4_status fp8_ffn_fprop(const fp8_tensor *xq, const fp8_tensor *wg, const fp8_tensor *wu,
                                 const fp8_tensor *wd, const fp8_tensor *hq, void *g, void *u, void *y, int64_t ldy,
                                 void *ws, size_t ws_bytes, hipStream_t stream);
FP4_API fp4_status fp8_ffn_fprop_flags(const fp8_tensor *xq, const fp8_tensor *wg, const fp8_tensor *wu,
                                       const fp8_tensor *wd, const fp8_tensor *hq, void *g, void *u, void *y,
                                       int64_t ldy, uint32_t flags, void *ws, size_t ws_bytes, hipStream_t stream);

/* Its gradients from dy (quantized in both layouts, dyq [M][K], dyq_t [K][M]), x^T
 * (xq_t [K][M]), the transposed weights (wg_t, wu_t [K][F], wd_t [F][K], tile scales)
 * and the forward call's g and u:
 *   dh = dy wd                     (binary32)
 *   du = dh * silu(g),  dg = dh * u * silu'(g),  h = silu(g) * u, each quantized in
 *        1 x 128 blocks: dgq, duq [M][F] along F; dgq_t, duq_t, hq_t [F][M] along M
 *   dx = dg wg + du wu             bf16 [M][K]
 *   dwg = dg^T x, dwu = du^T x     bf16 [F][K]
 *   dwd = dy^T h                   bf16 [K][F]
 * dx is one accumulation over both of its terms.  flags as for the forward call.
 * All outputs contiguous.  ws as for the forward call; the call with flags takes
 * fp8_ffn_backward_ws_bytes(M, K, F, flags) where g and u are aligned to 16 bytes, and
 * fp8_ffn_ws_bytes(M, K, F) is enough where they are not.  Errors: as there. */
typedef struct fp8_ffn_buffers {
  fp8_tensor dgq, duq, dgq_t, duq_t, hq_t;
} fp8_ffn_buffers;
FP4_API fp4_status fp8_ffn_backward(const fp8_tensor *dyq, const fp8_tensor *dyq_t, const fp8_tensor *xq_t,
                                    const fp8_tensor *wg_t, const fp8_tensor *wu_t, const fp8_tensor *wd_t,
                                    const void *g, const void *u, const fp8_ffn_buffers *bufs, void *dx, void *dwg,
                                    void *dwu, void *dwd, void *ws, size_t ws_bytes, hipStream_t stream);
FP4_API fp4_status fp8_ffn_backward_flags(const fp8_tensor *dyq, const fp8_tensor *dyq_t, const fp8_tensor *xq_t,
                                          const fp8_tensor *wg_t, const fp8_tensor *wu_t, const fp8_tensor *wd_t,
                                          const void *g, const void *u, const fp8_ffn_buffers *bufs, void *dx,
                                          void *dwg, void *dwu, void *dwd, uint32_t flags, void *ws, size_t ws_bytes,
                                          hipStream_t stream);
/* Each call's own, and what is enough for either with any flags.  Pure host arithmetic. */
FP4_API fp4_status fp8_ffn_fprop_ws_bytes(int64_t M, int64_t K, int64_t F, int32_t keep, uint32_t flags,
                                          size_t *bytes);
FP4_API fp4_status fp8_ffn_backward_ws_bytes(int64_t M, int64_t K, int64_t F, uint32_t flags, size_t *bytes);
FP4_API fp4_status fp8_ffn_ws_bytes(int64_t M, int64_t K, int64_t F, size_t *bytes);

/* Low-rank adapters beside a projection whose weight is shared: `count` pairs of a
 * [rank][K], rows lda elements apart, and b [N][rank], contiguous, both bf16, 16-byte aligned
 * and one pair after the other, with a factor scale [count] (binary32, device) each.  rank is
 * a multiple of 8 up to 128 (a smaller rank is stored with zeros in the rest), lda a multiple
 * of 8; the elements of a's rows from K on are not read for a result.  An adapter's tokens
 * belong next to each other where there are many: a tile of the result, up to 256 tokens,
 * takes its adapters one after the other. */
typedef struct fp8_lora {
  const void *a;
  const void *b;
  const float *scale;
  int64_t lda;
  int32_t count;
  int32_t rank;
} fp8_lora;

/* A flag of the adapters' calls: neighbouring tokens have different adapters (a batch of single
 * tokens of many requests, say).  Of 65 to 512 tokens a and b are then read once for each token,
 * and not an adapter after the other for each tile of the result.  Never wrong, in either case:
 * a matter of time, and of the last bits. */
#define FP8_LORA_MIXED (1u << 3)

/* y[m] = x[m] W^T + scale_i (dropout(x)[m] a_i^T) b_i^T,  i = index[m],  bf16 [M][N]
 * xq [M][K] (1 x 128), wq [N][K] (tile scales), index [M] int32 on the device: a token's
 * adapter; one outside [0, count) has none and adds nothing.  index NULL: every token has
 * adapter 0.  drop: the dropout of x's values in front of the adapters (NULL: none).  Both
 * terms are one binary32 sum, rounded once; the product with a_i is in binary32 and enters the
 * one with b_i whole, or with FP8_GEMM_FAST and many tokens as the sum of two bf16 (2^-17 of it
 * lost).  A token's infinities
 * and NaNs, and its adapter's, leave the other tokens' rows as they are (where b_i holds one,
 * the result is an infinity or NaN).  y must not overlap an input.
 * flags: those of fp8_gemm, for the product with W, and FP8_LORA_MIXED.  A token's results do
 * not depend on how many adapters there are.  ws: fp8_lora_fprop_ws_bytes(M, N, K, rank,
 * flags) bytes, 16-byte aligned, overwritten.
 * Errors: FP4_ERR_MODE (unknown flags), FP4_ERR_NULL, FP4_ERR_MISMATCH (shapes, kinds of
 * scales), FP4_ERR_SHAPE (strides, rank, count, p), FP4_ERR_ALIGN, FP4_ERR_WORKSPACE,
 * FP4_ERR_HIP.  Limits: count at most 65535, count * rank * (lda + N) at most 2^32. */
FP4_API fp4_status fp8_lora_fprop(const fp8_tensor *xq, const fp8_tensor *wq, const fp8_lora *lora,
                                  const int32_t *index, const fp8_dropout_config *drop, void *y, int64_t ldy,
                                  uint32_t flags, void *ws, size_t ws_bytes, hipStream_t stream);
FP4_API fp4_status fp8_lora_fprop_ws_bytes(int64_t M, int64_t N, int64_t K, int32_t rank, uint32_t flags,
                                           size_t *bytes);

/* Its gradients, the weight's own left out (it is frozen), from dy (dyq [M][N], 1 x 128),
 * the transposed weight (wq_t [K][N], tile scales), x (xq, which the forward call read) and
 * the same lora, index and drop:
 *   t = dropout(x) a_i^T,  dt = dy b_i       (binary32; t is computed again)
 *   dx[m] = dy[m] W + scale_i dropout'(dt[m] a_i)      bf16 [M][K], row stride lddx
 *   da_i  = scale_i sum over its tokens of dt[m]^T dropout(x)[m]    binary32 [count][rank][lda]
 *   db_i  = scale_i sum over its tokens of dy[m]^T t[m]             binary32 [count][N][rank]
 * dropout' multiplies by what dropout multiplied x by.  da and db are a's and b's layouts,
 * zeros in da's rows from K on and for an adapter without tokens.  The coefficients t and dt
 * enter the products of da and db as the sum of three bf16 (all of a binary32, but of values
 * below 2^-100, whose third is below bf16's range).
 * The outputs must not overlap each other or an input.
 * ws: fp8_lora_backward_ws_bytes(M, N, K, rank, count, flags) bytes.  Errors as for the
 * forward call. */
FP4_API fp4_status fp8_lora_backward(const fp8_tensor *dyq, const fp8_tensor *wq_t, const fp8_tensor *xq,
                                     const fp8_lora *lora, const int32_t *index, const fp8_dropout_config *drop,
                                     void *dx, int64_t lddx, float *da, float *db, uint32_t flags, void *ws,
                                     size_t ws_bytes, hipStream_t stream);
FP4_API fp4_status fp8_lora_backward_ws_bytes(int64_t M, int64_t N, int64_t K, int32_t rank, int32_t count,
                                              uint32_t flags, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_AMD_FP8_H */
