/*
 * awq_a8.h -- C ABI of libawq for 8-bit activations: the producers of a quantized layer's input
 * (RMS norm with the residual's addition, gated activation), with an output in 8 bits and a
 * scale per row, and the product of such activations with the packed 4-bit weight.
 *
 * The conventions of awq.h hold (device memory owned by the caller, argument errors returned
 * synchronously, every call asynchronous on `stream`, nothing allocated, no state kept).  These
 * calls carry no data-error flags: a row of the input that holds NaN or Inf gets the scale NaN,
 * so every product that reads it is NaN (its codes are undefined); in a 16- or 32-bit output
 * the row's own NaN or Inf shows.
 */
#ifndef AWQ_A8_H
#define AWQ_A8_H

#include "awq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of 8-bit activations, beside awq_dtype's F32 and BF16. */
#define AWQ_DTYPE_I8 2   /* int8, codes -127 .. 127 */
#define AWQ_DTYPE_E4M3 3 /* e4m3 without infinities (OCP), |code| <= 448 */

/* Or'ed into awq_w4a8's y_dtype, at most one: how e4m3 codes are summed. */
#define AWQ_W4A8_SUMS_F32 0x100    /* in fp32 */
#define AWQ_W4A8_SUMS_MATRIX 0x200 /* by the matrix unit's own 8-bit products */

/* Activations of awq_act_mul, beside awq.h's AWQ_ACT_GELU and AWQ_ACT_SILU. */
#define AWQ_ACT_NONE 2

/* ---------------------------------------------------------------------------------------
 * The norm in front of a quantized layer (its gamma is where awq_fold_rows leaves 1/s):
 *   h = x + r (h = x without R);   y = h / sqrt(mean_k h[k]^2 + eps) * gamma[k]
 * h and y are formed in fp32, the mean from h before its rounding.
 *   X      [M, K] of x_dtype (F32, BF16), row stride ldx
 *   R      [M, K] of r_dtype (F32, BF16), row stride ldr, or NULL (no residual)
 *   H      [M, K] of r_dtype, row stride ldh: h rounded once; may be R itself (ldh = ldr); NULL
 *          without R, and where h is not wanted
 *   gamma  [K] of g_dtype (F32, BF16)
 *   eps    finite and positive
 *   Y      [M, K] of y_dtype, row stride ldy: F32 or BF16 holds y rounded once; I8 or E4M3 holds
 *          round(y / scale) to nearest even in the type, with
 *          scale = max(max_k |y|, 2^-100) / Q,  Q = 127 (I8) or 448 (E4M3)
 *   scale  fp32 [M] for an 8-bit Y, else ignored
 * Any K.  H = R aside, outputs overlap no input and not each other (of this only exact starts are checked: Y on
 * H, an output on gamma, or on an operand in another type or row stride, are AWQ_ERR_INVALID_ARG).  A row whose
 * sum of squares is not finite in fp32 (|h| of 1.8e19 / sqrt(K) and more, NaN, Inf) has y NaN.
 * ------------------------------------------------------------------------------------- */
AWQ_API int awq_rmsnorm(const void* X, int x_dtype, int64_t M, int64_t K, int64_t ldx, const void* R,
                        int r_dtype, int64_t ldr, void* H, int64_t ldh, const void* gamma, int g_dtype,
                        float eps, void* Y, int y_dtype, int64_t ldy, float* scale, awq_stream_t stream);

/* ---------------------------------------------------------------------------------------
 * The activation in front of a quantized layer:  y[m, k] = act(G[m, k]) * U[m, k] / s[k]
 *   G, U   [M, K] of x_dtype (F32, BF16), row strides ldg, ldu (the halves of a fused gate/up
 *          output are two such views); U NULL: no gate's product
 *   act    AWQ_ACT_NONE, AWQ_ACT_GELU (0.5 x (1 + erf(x / sqrt 2))) or AWQ_ACT_SILU
 *          (x / (1 + exp(-x)))
 *   s      fp32 [K] or NULL: the runtime form of 1/s where no producer absorbed it; 2^-126 to 2^126,
 *          so that s and 1/s are normal numbers (not checked here: the search and the pack did that
 *          s is positive and finite, and what the search writes stays far inside)
 *   Y, y_dtype, ldy, scale   as awq_rmsnorm
 * With act NONE and neither U nor s this quantizes given activations.  y is formed in fp32,
 * with a relative error of at most, in units of 2^-24: NONE 8; SILU 18, and |x| more where Y is not
 * F32; GELU 28 + 2 x^2 (its tail is that ill-conditioned).  An activation below 2^-126 is within 2^-149 (SiLU), or
 * may be 0 (GELU).
 * Any K.  Y may be G or U where it has their type
 * and row stride, and overlaps them in no other way.
 * ------------------------------------------------------------------------------------- */
AWQ_API int awq_act_mul(const void* G, int x_dtype, int64_t M, int64_t K, int64_t ldg, const void* U,
                        int64_t ldu, const float* s, int act, void* Y, int y_dtype, int64_t ldy,
                        float* scale, awq_stream_t stream);

/* ---------------------------------------------------------------------------------------
 * The artefact of awq_pack laid out for awq_w4a8, once per weight (4.25 bits per weight, N
 * rounded up to 16, and 4 bytes per channel):
 *   wt     device memory of at least awq_w4a8_weight_bytes(N, K) bytes, 256-byte aligned, in three
 *          parts, each starting at a multiple of 256 bytes:
 *            codes  for column tile c (channels n = 16 c + l % 16) and group g, 16 bytes per
 *                   l < 64: the codes of k = 128 g + 16 (l / 16) .. + 15 and 64 further on, four
 *                   words of eight; byte b of a word holds code b (low nibble) and b + 4 (high)
 *            steps  uint32 [tiles][K/128][16]: fp16 scales * 2^-e (low half), fp16 zeros (high)
 *            powers fp32 [16 tiles]: 2^e, e per channel such that its largest step lies in
 *                   [2^10, 2^11)
 *   qweight, scales, zeros   as written by awq_pack (qweight 16-byte aligned)
 * N is at most 2^27 (AWQ_ERR_SHAPE).  awq_w4a8_weight_bytes is 0 for sizes that awq_w4a8_weight rejects.
 * ------------------------------------------------------------------------------------- */
AWQ_API size_t awq_w4a8_weight_bytes(int64_t N, int64_t K);
AWQ_API int awq_w4a8_weight(const int32_t* qweight, const uint16_t* scales, const uint16_t* zeros,
                            int64_t N, int64_t K, int32_t group, void* wt, size_t wt_bytes,
                            awq_stream_t stream);

/* ---------------------------------------------------------------------------------------
 * The W4A8 product:
 *   Y[m, n] = xscale[m] * sum_g scales[n, g] * sum_{k in g} Xq[m, k] (q[n, k] - zeros[n, g])
 * on the 8-bit matrix cores: a code q is an int8 byte as it stands, and as an e4m3 byte it is
 * exactly q 2^-9.  I8: the inner sums are exact integers.  E4M3: the products are exact, and a group's are
 * summed
 *   in fp32 for an F32 Y, and for a BF16 Y of up to 256 tokens (at half the matrix rate);
 *   by the matrix unit for a BF16 Y of more.  It adds sixteen at a time to 14 bits of the largest of them: off by at
 *     most 2^-9 of the sum of the magnitudes |x q| and z |x|, 2^-13 and less as a rule; more than a bf16 rounding
 *     where one large code with q = z stands beside small ones.
 * AWQ_W4A8_SUMS_F32 or AWQ_W4A8_SUMS_MATRIX in y_dtype ask for one of the two at any size; with I8 they
 * change nothing.  The sums z multiplies are within 2^-23 of fp32's.  The steps and the sum over groups
 * are fp32; Y is rounded once.
 *   Xq      [M, K] of x_dtype I8 or E4M3, row stride ldx, 16-byte aligned rows
 *   xscale  fp32 [M]
 *   wt      as written by awq_w4a8_weight for the same N and K
 *   Y       [M, N] of y_dtype F32 or BF16 (and a flag, see above), row stride ldy >= N
 *   ws      device memory of at least awq_w4a8_workspace_bytes(M, K, N) bytes, 16-byte aligned
 *           (NULL where that is 0); nothing in it has to start at zero, and calls that may run at
 *           the same time need one each
 * Y and ws overlap no input and not each other (an exact start is checked: AWQ_ERR_INVALID_ARG).
 * K is a multiple of 128; 128 rows of Xq and of Y span less than 2^31 bytes each; M ceil(N / 256) is below
 * 2^29 (AWQ_ERR_SHAPE; awq_w4a8_workspace_bytes is then 0).
 * ------------------------------------------------------------------------------------- */
AWQ_API size_t awq_w4a8_workspace_bytes(int64_t M, int64_t K, int64_t N);
AWQ_API int awq_w4a8(const void* Xq, int x_dtype, const float* xscale, int64_t M, int64_t K, int64_t ldx,
                     const void* wt, int64_t N, int32_t group, void* Y, int y_dtype, int64_t ldy, void* ws,
                     size_t ws_bytes, awq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* AWQ_A8_H */
