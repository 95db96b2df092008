// Host side of the low-rank adapters: argument validation behind the C ABI declared in include/awq_lora.h.
#include <climits>
#include <cstdint>

#include "api_check.h"
#include "awq_lora.h"
#include "lora_internal.h"

namespace {

using namespace awq::api;

constexpr int64_t kMaxRank = 256, kMaxRows = 1 << 24, kMaxCols = 1 << 22;

// The sizes as the launches take them: fewer than 2^32 threads, and 32-bit tile counts.
bool lora_sizes(int64_t M, int64_t K, int64_t N, int64_t R) {
  if (M <= 0 || K <= 0 || N <= 0 || R <= 0 || M >= kMaxRows || N >= kMaxCols || K % 8 != 0 || R % 8 != 0 || R > kMaxRank)
    return false;
  return (M + 15) / 16 * ((N + 255) / 256) < (1 << 23) && K < (int64_t)INT32_MAX;
}

}  // namespace

extern "C" {

AWQ_API size_t awq_lora_workspace_bytes(int64_t M, int64_t K, int64_t N, int64_t R) {
  if (!lora_sizes(M, K, N, R)) return 0;
  // What no batch of up to M tokens exceeds, so that one workspace serves them all: lora_splits gives at most min(16, K / 512)
  // splits, and more than one only up to 512 blocks, of at most sixteen tokens each: splits M <= M + 511 * 16.
  const int64_t most = K / 512 < 1 ? 1 : K / 512 < 16 ? K / 512 : 16;
  const int64_t rows = M * most < M + 8192 ? M * most : M + 8192;
  return (size_t)(rows * R * 4);
}

AWQ_API int awq_lora(const void* X, int x_dtype, const float* xscale, int64_t M, int64_t K, int64_t ldx, const void* A,
                     const void* B, int64_t adapters, int64_t R, const int32_t* ranks, const float* scale,
                     const int32_t* ids, const void* base, int64_t ldb, void* Y, int y_dtype, int64_t ldy, int64_t N,
                     void* ws, size_t ws_bytes, awq_stream_t stream) {
  if (M <= 0 || K <= 0 || N <= 0 || R <= 0 || adapters <= 0 || A == nullptr || B == nullptr || ids == nullptr)
    return AWQ_ERR_INVALID_ARG;
  if ((!float_type(x_dtype) && !code_type(x_dtype)) || !float_type(y_dtype)) return AWQ_ERR_UNSUPPORTED;
  if (!lora_sizes(M, K, N, R) || adapters > (int64_t)INT32_MAX || mul3(adapters, R, K * 2) < 0 || mul3(adapters, R, N * 2) < 0)
    return AWQ_ERR_SHAPE;
  int st = check_rows(X, x_dtype, M, K, ldx);
  if (st == AWQ_OK) st = check_rows(base, y_dtype, M, N, ldb);
  if (st == AWQ_OK) st = check_rows(Y, y_dtype, M, N, ldy);
  if (st != AWQ_OK) return st;
  if (code_type(x_dtype) && (xscale == nullptr || !aligned(xscale, 4))) return AWQ_ERR_INVALID_ARG;
  if (!rows_aligned(X, x_dtype, ldx, code_type(x_dtype) ? 8 : 16) || !aligned(A, 16) || !aligned(B, 16) ||
      !aligned(ids, 4) || !aligned(ranks, 4) || !aligned(scale, 4))
    return AWQ_ERR_INVALID_ARG;
  const size_t need = awq_lora_workspace_bytes(M, K, N, R);
  if (ws == nullptr || ws_bytes < need) return AWQ_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return AWQ_ERR_INVALID_ARG;
  if (Y == base && ldy != ldb) return AWQ_ERR_INVALID_ARG;
  for (const void* in : {X, A, B, (const void*)xscale, (const void*)ids, (const void*)scale, (const void*)ranks})
    if (in != nullptr && (Y == in || ws == in)) return AWQ_ERR_INVALID_ARG;
  if (ws == Y || ws == base) return AWQ_ERR_INVALID_ARG;
  awq::LoraArgs a{};
  a.x = X, a.xscale = xscale, a.ids = ids, a.scale = scale, a.ranks = ranks, a.base = base, a.y = Y;
  a.a = static_cast<const uint16_t*>(A), a.b = static_cast<const uint16_t*>(B), a.t = static_cast<float*>(ws);
  a.M = M, a.K = K, a.N = N, a.ldx = ldx, a.ldb = ldb, a.ldy = ldy;
  a.n = (int)adapters, a.R = (int)R, a.splits = awq::lora_splits(M, K, R);
  a.ybf16 = y_dtype == AWQ_DTYPE_BF16;
  a.vec = rows_aligned(base, y_dtype, ldb, 16) && rows_aligned(Y, y_dtype, ldy, 16);
  return map_hip(awq::launch_lora(a, x_dtype, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
