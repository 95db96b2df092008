/*
 * awq_lora.h -- C ABI of libawq for low-rank adapters of many requests beside a shared projection: the projection
 * (awq_w4a16, awq_w4a8, any other) runs once for the whole batch, and each row gets its own adapter's product added.
 *
 * The conventions of awq.h hold (device memory owned by the caller, argument errors returned synchronously, every call
 * asynchronous on `stream`, nothing allocated, no state kept).  No data-error flags: NaN and Inf in a row of X, in base
 * or in an adapter reach that row, or that adapter's rows, of Y, and no others.
 */
#ifndef AWQ_LORA_H
#define AWQ_LORA_H

#include "awq_a8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------------------
 *   Y[m] = base[m] + scale[a] * B[a] (A[a] x[m]),  a = ids[m]
 *   X      [M, K] of x_dtype F32 or BF16 (16-byte aligned rows), or I8 or E4M3 (8-byte aligned rows) with a scale per
 *          row, row stride ldx; K a multiple of 8
 *   xscale fp32 [M] for I8 and E4M3, else ignored
 *   A      BF16 [adapters, R, K], contiguous, 16-byte aligned
 *   B      BF16 [adapters, N, R], contiguous, 16-byte aligned; R a multiple of 8 up to 256
 *   ranks  int32 [adapters] or NULL (all R): the rows of A[a] and the columns of B[a] from ranks[a] on are not used,
 *          whatever they hold; a value below 0 counts as 0, one above R as R
 *   scale  fp32 [adapters] or NULL (1)
 *   ids    int32 [M]; a value outside 0 .. adapters-1 leaves the row as base is
 *   base   [M, N] of y_dtype, row stride ldb
 *   Y      [M, N] of y_dtype (F32, BF16), row stride ldy; may be base itself (ldy = ldb)
 *   ws     device memory of at least awq_lora_workspace_bytes bytes, 16-byte aligned; nothing in it has to start at
 *          zero, one laid out for M tokens serves fewer, and calls that may run at the same time need one each
 * Products are exact in the matrix cores (an F32 X as three bf16 terms), sums fp32.  scale (A x) is formed in fp32 and
 * handed on in two bf16 terms (2^-17) for a BF16 Y, in three (exactly) for F32; Y is rounded once.  A row's result does
 * not depend on which rows stand beside it, but for the order of the sums over K, which the sizes alone decide: equal
 * calls give equal bits.
 * M is below 2^24, N below 2^22, K and adapters below 2^31, ceil(M / 16) ceil(N / 256) below 2^23 (AWQ_ERR_SHAPE; the
 * workspace's size is then 0).  Apart from Y = base, Y and ws overlap no input and not each other (an exact start is
 * checked: AWQ_ERR_INVALID_ARG).
 * ------------------------------------------------------------------------------------- */
AWQ_API size_t awq_lora_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t R);
AWQ_API int awq_lora(const void* X, int x_dtype, const float* xscale, int64_t M, int64_t K, int64_t ldx, const void* A,
                     const void* B, int64_t adapters, int64_t R, const int32_t* ranks, const float* scale,
                     const int32_t* ids, const void* base, int64_t ldb, void* Y, int y_dtype, int64_t ldy, int64_t N,
                     void* ws, size_t ws_bytes, awq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* AWQ_LORA_H */
