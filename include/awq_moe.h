/*
 * awq_moe.h -- C ABI of libawq for mixtures of experts whose weights are the packed 4-bit artefact: the router, and a
 * layer's experts for the tokens of a decode batch or a short prompt.
 *
 * The conventions of awq.h hold (device memory owned by the caller, argument errors returned synchronously, every call
 * asynchronous on `stream`, nothing allocated, no state kept).  Activations are F32, BF16, or I8 / E4M3 codes with a
 * scale per row (awq_a8.h).  No data-error flags: a token whose activations hold NaN or Inf, or whose row scale is NaN,
 * has a result that is not finite, and no other token's result changes.  Finite activations up to the largest number give
 * a finite result where the definition's sums of magnitudes, sum |x| D |q - z|, stay inside fp32 (in channels whose largest
 * step D is 2^-11 or more; below, that much sooner).
 */
#ifndef AWQ_MOE_H
#define AWQ_MOE_H

#include "awq_a8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a router's logit becomes a weight. */
#define AWQ_MOE_SOFTMAX 0 /* exp(v) / sum over all experts of exp */
#define AWQ_MOE_SIGMOID 1 /* 1 / (1 + exp(-v)) */

/* ---------------------------------------------------------------------------------------
 * The router: the k experts of each token with the largest logits, largest first, ties to the lowest index.
 *   logits   [M, E] of l_dtype (F32, BF16), row stride ldl, M at most 2^24, E 1024 (AWQ_ERR_SHAPE)
 *   k        1 .. E (AWQ_ERR_INVALID_ARG), at most 32 (AWQ_ERR_SHAPE)
 *   ids      int32 [M, k]
 *   weights  fp32 [M, k]: the score of the expert, and with renormalize != 0 divided by the sum of the k scores (scores
 *            that all underflow keep their ratios)
 * A logit of -Inf masks its expert: it is never chosen.  Where fewer than k experts are left, the rest of the row has id
 * -1 and weight 0.  A NaN counts as the largest logit; the weights of its row are NaN (sigmoid without renormalize: only
 * its own), as they are for +Inf with softmax.
 * ------------------------------------------------------------------------------------- */
AWQ_API int awq_moe_route(const void* logits, int l_dtype, int64_t M, int64_t E, int64_t ldl, int32_t k, int score,
                          int renormalize, int32_t* ids, float* weights, awq_stream_t stream);

/* ---------------------------------------------------------------------------------------
 * The experts of a layer:
 *   Y[m] = sum_j weights[m, j] D_e (act(G_e x[m]) * (U_e x[m])),  e = ids[m, j]
 *   X        [M, H] of x_dtype (F32, BF16, I8, E4M3), row stride ldx, 16-byte aligned rows
 *   xscale   fp32 [M] for I8 and E4M3, else ignored
 *   ids      int32 [M, k]; a value outside 0 .. E-1 is skipped (an expert that another device holds, or none), but
 *            counts where the kernels are chosen by M k / E; the same expert may stand more than once in a row
 *   weights  fp32 [M, k]
 *   gate_up  as written by awq_w4a8_weight for N = 2 I E and K = H: expert e's gate rows from 2 I e on, its up rows I
 *            further
 *   down     the same for N = H E and K = I: expert e's rows from H e on
 *   act      AWQ_ACT_SILU or AWQ_ACT_GELU
 *   Y        [M, H] of y_dtype (F32, BF16), row stride ldy; a token without an expert here gets 0
 *   ws       device memory of at least awq_moe_workspace_bytes bytes, 256-byte aligned; nothing in it has to start at
 *            zero, one laid out for M tokens serves fewer, and calls that may run at the same time need one each
 * H and I are multiples of 128 up to 2^20, M is at most 2^24, E 1024, k 32, 2 I E and H E 2^27 (AWQ_ERR_SHAPE; the
 * workspace's size is then 0).  Zero points are whole numbers, as awq_pack writes them.
 * Products are exact in the matrix cores (codes, and an F32 X as three bf16 terms; exact from 2^-90 up), sums fp32;
 * act(gate) * up is formed in fp32 and handed on in two bf16 terms (2^-17) for a BF16 Y, in three (exactly, from 2^-90 up)
 * for F32; Y is rounded once.  I8 sums are exact in a group; the others are rounded by the magnitudes |x| D (16 + q) and
 * |x| D (16 + z), not |x| D |q - z|: an activation with q = z beside small ones costs their sum up to 2^-19 D of its size.
 * The order of the sums depends on the sizes alone: equal calls give equal bits.
 * Y and ws overlap no input and not each other (an exact start is checked: AWQ_ERR_INVALID_ARG).
 * ------------------------------------------------------------------------------------- */
AWQ_API size_t awq_moe_workspace_bytes(int64_t M, int64_t E, int32_t k, int64_t H, int64_t I);
AWQ_API int awq_moe(const void* X, int x_dtype, const float* xscale, int64_t M, int64_t H, int64_t ldx,
                    const int32_t* ids, const float* weights, int32_t k, const void* gate_up, const void* down, int64_t E,
                    int64_t I, int32_t group, int act, void* Y, int y_dtype, int64_t ldy, void* ws, size_t ws_bytes,
                    awq_stream_t stream);

/* The whole layer from the router's logits: awq_moe with the ids and weights that awq_moe_route gives for them, bit for
 * bit.  The same workspace; k at most E. */
AWQ_API int awq_moe_layer(const void* X, int x_dtype, const float* xscale, int64_t M, int64_t H, int64_t ldx,
                          const void* logits, int l_dtype, int64_t ldl, int32_t k, int score, int renormalize,
                          const void* gate_up, const void* down, int64_t E, int64_t I, int32_t group, int act, void* Y,
                          int y_dtype, int64_t ldy, void* ws, size_t ws_bytes, awq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* AWQ_MOE_H */
