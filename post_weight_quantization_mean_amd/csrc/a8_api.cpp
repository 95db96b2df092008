// Host side of the 8-bit activation path: argument validation behind the C ABI declared in
// include/awq_a8.h.  Validation is plain host code that runs before any HIP call.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "a8_internal.h"
#include "api_check.h"
#include "awq_a8.h"

namespace {

using awq::kGroup;
using namespace awq::api;

int check_out(const void* y, int y_type, int64_t M, int64_t K, int64_t ldy, const float* scale) {
  if (!float_type(y_type) && !code_type(y_type)) return AWQ_ERR_UNSUPPORTED;
  if (code_type(y_type) && (scale == nullptr || !aligned(scale, 4))) return AWQ_ERR_INVALID_ARG;
  return check_rows(y, y_type, M, K, ldy);
}

// eight elements of y per store: 32 or 16 bytes, or 8 of codes
bool out_vec(const void* y, int y_type, int64_t ldy) {
  return rows_aligned(y, y_type, ldy, code_type(y_type) ? 8 : 16);
}

constexpr int64_t kMaxTokenTiles = 1 << 29;  // below 2^32 threads: 256 per 64 tokens x 256 channels

// The sizes of a product of M tokens, as the plan's arithmetic and the launches take them.
bool w4a8_sizes(int64_t M, int64_t N, int64_t K, awq::W4a8Layout* L) {
  return M > 0 && w4a8_layout(N, K, L) && M < kMaxTokenTiles && M * ((N + 255) / 256) < kMaxTokenTiles &&
         mul3(M, K, 1) >= 0;
}

}  // namespace

extern "C" {

AWQ_API int awq_rmsnorm(const void* X, int x_dtype, int64_t M, int64_t K, int64_t ldx, const void* R, int r_dtype,
                        int64_t ldr, void* H, int64_t ldh, const void* gamma, int g_dtype, float eps, void* Y,
                        int y_dtype, int64_t ldy, float* scale, awq_stream_t stream) {
  if (M <= 0 || K <= 0 || gamma == nullptr || !(eps > 0.0f) || !std::isfinite(eps)) return AWQ_ERR_INVALID_ARG;
  if (!float_type(x_dtype) || !float_type(g_dtype) || (R != nullptr && !float_type(r_dtype)))
    return AWQ_ERR_UNSUPPORTED;
  if (!aligned(gamma, (uintptr_t)dsize(g_dtype)) || (R == nullptr && H != nullptr)) return AWQ_ERR_INVALID_ARG;
  int st = check_rows(X, x_dtype, M, K, ldx);
  if (st == AWQ_OK && R != nullptr) st = check_rows(R, r_dtype, M, K, ldr);
  if (st == AWQ_OK && H != nullptr) st = check_rows(H, r_dtype, M, K, ldh);
  if (st == AWQ_OK) st = check_out(Y, y_dtype, M, K, ldy, scale);
  if (st != AWQ_OK) return st;
  // an output exactly over an operand in another type or row stride: rows would overwrite other rows' operands
  auto crossed = [](const void* p, int pt, int64_t pl, const void* q, int qt, int64_t ql) {
    return p != nullptr && p == q && (pt != qt || pl != ql);
  };
  if (crossed(H, r_dtype, ldh, R, r_dtype, ldr) || crossed(H, r_dtype, ldh, X, x_dtype, ldx) ||
      crossed(Y, y_dtype, ldy, X, x_dtype, ldx) || crossed(Y, y_dtype, ldy, R, r_dtype, ldr) ||
      Y == H || Y == gamma || (H != nullptr && H == gamma))
    return AWQ_ERR_INVALID_ARG;
  const bool vec = K % 8 == 0 && rows_aligned(X, x_dtype, ldx, 16) && aligned(gamma, 16) &&
                   (R == nullptr || rows_aligned(R, r_dtype, ldr, 16)) &&
                   (H == nullptr || rows_aligned(H, r_dtype, ldh, 16)) && out_vec(Y, y_dtype, ldy);
  awq::RowArgs a{};
  a.x = X, a.b = R, a.h = H, a.col = gamma, a.y = Y, a.scale = scale;
  a.M = M, a.K = K, a.ldx = ldx, a.ldb = ldr, a.ldh = ldh, a.ldy = ldy;
  a.eps = eps, a.col_type = g_dtype, a.y_type = y_dtype;
  return map_hip(awq::launch_rmsnorm(a, x_dtype, R != nullptr ? r_dtype : awq::kNoOperand, vec,
                                     reinterpret_cast<hipStream_t>(stream)));
}

AWQ_API int awq_act_mul(const void* G, int x_dtype, int64_t M, int64_t K, int64_t ldg, const void* U, int64_t ldu,
                        const float* s, int act, void* Y, int y_dtype, int64_t ldy, float* scale,
                        awq_stream_t stream) {
  if (M <= 0 || K <= 0) return AWQ_ERR_INVALID_ARG;
  if (!float_type(x_dtype) || (act != AWQ_ACT_NONE && act != AWQ_ACT_GELU && act != AWQ_ACT_SILU))
    return AWQ_ERR_UNSUPPORTED;
  if (s != nullptr && !aligned(s, 4)) return AWQ_ERR_INVALID_ARG;
  int st = check_rows(G, x_dtype, M, K, ldg);
  if (st == AWQ_OK && U != nullptr) st = check_rows(U, x_dtype, M, K, ldu);
  if (st == AWQ_OK) st = check_out(Y, y_dtype, M, K, ldy, scale);
  if (st != AWQ_OK) return st;
  if ((Y == G && (y_dtype != x_dtype || ldy != ldg)) || (Y == U && (y_dtype != x_dtype || ldy != ldu)))
    return AWQ_ERR_INVALID_ARG;
  const bool vec = K % 8 == 0 && rows_aligned(G, x_dtype, ldg, 16) &&
                   (U == nullptr || rows_aligned(U, x_dtype, ldu, 16)) && (s == nullptr || aligned(s, 16)) &&
                   out_vec(Y, y_dtype, ldy);
  awq::RowArgs a{};
  a.x = G, a.b = U, a.col = s, a.y = Y, a.scale = scale;
  a.M = M, a.K = K, a.ldx = ldg, a.ldb = ldu, a.ldy = ldy;
  a.act = act, a.col_type = s != nullptr ? awq::kF32 : awq::kNoOperand, a.y_type = y_dtype;
  return map_hip(awq::launch_act_mul(a, x_dtype, vec, reinterpret_cast<hipStream_t>(stream)));
}

AWQ_API size_t awq_w4a8_weight_bytes(int64_t N, int64_t K) {
  awq::W4a8Layout L;
  return w4a8_layout(N, K, &L) ? L.total : 0;
}

AWQ_API int awq_w4a8_weight(const int32_t* qweight, const uint16_t* scales, const uint16_t* zeros, int64_t N,
                            int64_t K, int32_t group, void* wt, size_t wt_bytes, awq_stream_t stream) {
  if (qweight == nullptr || scales == nullptr || zeros == nullptr || N <= 0 || K <= 0) return AWQ_ERR_INVALID_ARG;
  if (group != kGroup) return AWQ_ERR_UNSUPPORTED;
  awq::W4a8Layout L;
  if (!w4a8_layout(N, K, &L)) return AWQ_ERR_SHAPE;
  if (!aligned(qweight, 16) || !aligned(scales, 2) || !aligned(zeros, 2)) return AWQ_ERR_INVALID_ARG;
  if (wt == nullptr || wt_bytes < L.total) return AWQ_ERR_WORKSPACE;
  if (!aligned(wt, kAlign)) return AWQ_ERR_INVALID_ARG;
  char* p = static_cast<char*>(wt);
  return map_hip(awq::launch_w4a8_weight(qweight, scales, zeros, N, K, reinterpret_cast<uint32_t*>(p),
                                         reinterpret_cast<uint32_t*>(p + L.steps),
                                         reinterpret_cast<float*>(p + L.powers),
                                         reinterpret_cast<hipStream_t>(stream)));
}

AWQ_API size_t awq_w4a8_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  awq::W4a8Layout L;
  if (!w4a8_sizes(M, N, K, &L)) return 0;
  return awq::w4a8_workspace(M, K, N);
}

AWQ_API int awq_w4a8(const void* Xq, int x_dtype, const float* xscale, int64_t M, int64_t K, int64_t ldx,
                     const void* wt, int64_t N, int32_t group, void* Y, int y_dtype, int64_t ldy, void* ws,
                     size_t ws_bytes, awq_stream_t stream) {
  if (Xq == nullptr || xscale == nullptr || wt == nullptr || Y == nullptr || M <= 0 || N <= 0 || K <= 0)
    return AWQ_ERR_INVALID_ARG;
  int sums = awq::kSumsDefault;
  if (y_dtype >= 0 && (y_dtype & ~0xff) == AWQ_W4A8_SUMS_F32) sums = awq::kSumsF32;
  if (y_dtype >= 0 && (y_dtype & ~0xff) == AWQ_W4A8_SUMS_MATRIX) sums = awq::kSumsMatrix;
  if (sums != awq::kSumsDefault) y_dtype &= 0xff;
  if (!code_type(x_dtype) || !float_type(y_dtype) || group != kGroup) return AWQ_ERR_UNSUPPORTED;
  awq::W4a8Layout L;
  if (!w4a8_sizes(M, N, K, &L)) return AWQ_ERR_SHAPE;
  int st = check_rows(Xq, x_dtype, M, K, ldx);
  if (st == AWQ_OK) st = check_rows(Y, y_dtype, M, N, ldy);
  if (st != AWQ_OK) return st;
  if (!rows_aligned(Xq, x_dtype, ldx, 16) || !aligned(xscale, 4) || !aligned(wt, kAlign)) return AWQ_ERR_INVALID_ARG;
  // tiles of up to 128 tokens use 32-bit offsets within their rows of Xq and of Y
  const int64_t xspan = mul3(awq::kW4a8TileM, ldx, 1), yspan = mul3(awq::kW4a8TileM, ldy, dsize(y_dtype));
  if (xspan < 0 || xspan >= (int64_t)INT32_MAX || yspan < 0 || yspan >= (int64_t)INT32_MAX) return AWQ_ERR_SHAPE;
  const size_t need = awq_w4a8_workspace_bytes(M, K, N);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return AWQ_ERR_WORKSPACE;
  if (need > 0 && !aligned(ws, 16)) return AWQ_ERR_INVALID_ARG;
  if (Y == Xq || Y == wt || Y == xscale || (need > 0 && (ws == Y || ws == Xq || ws == wt))) return AWQ_ERR_INVALID_ARG;
  const char* p = static_cast<const char*>(wt);
  awq::W4a8Args a{};
  a.x = Xq, a.xscale = xscale, a.y = Y;
  a.codes = reinterpret_cast<const uint32_t*>(p);
  a.steps = reinterpret_cast<const uint32_t*>(p + L.steps);
  a.powers = reinterpret_cast<const float*>(p + L.powers);
  a.M = M, a.K = K, a.N = N, a.ldx = ldx, a.ldy = ldy;
  a.e4m3 = x_dtype == AWQ_DTYPE_E4M3, a.ybf16 = y_dtype == AWQ_DTYPE_BF16, a.sums = sums;
  return map_hip(awq::launch_w4a8(a, ws, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
