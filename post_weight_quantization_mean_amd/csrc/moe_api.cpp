// Host side of the mixture of experts: argument validation behind the C ABI declared in include/awq_moe.h, and the passes
// over the tokens.
#include <climits>
#include <cstdint>

#include "api_check.h"
#include "awq_moe.h"
#include "moe_internal.h"

namespace {

using namespace awq::api;

static_assert(awq::kSoftmax == AWQ_MOE_SOFTMAX && awq::kSigmoid == AWQ_MOE_SIGMOID, "the ABI's scores");

// A launch takes fewer than 2^32 threads: 64 per token (router); a quarter per result of 2048 pairs (sum).
constexpr int64_t kMaxTokens = 1 << 24, kMaxWidth = 1 << 20;

bool route_sizes(int64_t M, int64_t E, int64_t k) {
  return M > 0 && M <= kMaxTokens && E > 0 && E <= awq::kMaxExperts && k > 0 && k <= awq::kMaxChosen;
}

int check_route(const void* logits, int l_dtype, int64_t M, int64_t E, int64_t ldl, int32_t k, int score) {
  if (M <= 0 || E <= 0 || k <= 0) return AWQ_ERR_INVALID_ARG;
  if (!float_type(l_dtype) || (score != AWQ_MOE_SOFTMAX && score != AWQ_MOE_SIGMOID)) return AWQ_ERR_UNSUPPORTED;
  if (!route_sizes(M, E, k)) return AWQ_ERR_SHAPE;
  if (k > E) return AWQ_ERR_INVALID_ARG;
  return check_rows(logits, l_dtype, M, E, ldl);
}

awq::RouteArgs route_args(const void* logits, int64_t M, int64_t E, int64_t ldl, int32_t k, int score, int renormalize,
                          int32_t* ids, float* weights) {
  awq::RouteArgs a{};
  a.logits = logits, a.ids = ids, a.weights = weights, a.M = M, a.ld = ldl;
  a.E = (int)E, a.k = k, a.score = score, a.renorm = renormalize != 0;
  return a;
}

struct MoeLayout {
  awq::W4a8Layout up, down;
  int64_t pass;                      // tokens of one pass
  size_t h, o, ids, weights, total;  // byte offsets in the workspace
};

bool moe_layout(int64_t M, int64_t E, int64_t k, int64_t H, int64_t I, MoeLayout* L) {
  if (!route_sizes(M, E, k) || H <= 0 || I <= 0 || H > kMaxWidth || I > kMaxWidth) return false;
  if (!w4a8_layout(2 * I * E, H, &L->up) || !w4a8_layout(H * E, I, &L->down)) return false;
  L->pass = awq::kMoePairs / k < M ? awq::kMoePairs / k : M;
  const int64_t pairs = L->pass * k;
  L->h = 0;
  L->o = align_up((size_t)(pairs * I * 6));
  L->ids = L->o + align_up((size_t)(pairs * H * 4));
  L->weights = L->ids + align_up((size_t)(M * k * 4));
  L->total = L->weights + align_up((size_t)(M * k * 4));
  return true;
}

struct Routing {  // given, or made from logits in the workspace
  const int32_t* ids;
  const float* weights;
  const void* logits;
  int l_dtype;
  int64_t ldl;
  int score, renormalize;
};

int run_moe(const void* X, int x_dtype, const float* xscale, int64_t M, int64_t H, int64_t ldx, const Routing& r, int32_t k,
            const void* gate_up, const void* down, int64_t E, int64_t I, int32_t group, int act, void* Y, int y_dtype,
            int64_t ldy, void* ws, size_t ws_bytes, awq_stream_t stream) {
  if (M <= 0 || H <= 0 || I <= 0 || E <= 0 || k <= 0 || gate_up == nullptr || down == nullptr) return AWQ_ERR_INVALID_ARG;
  if (r.logits == nullptr && (r.ids == nullptr || r.weights == nullptr)) return AWQ_ERR_INVALID_ARG;
  if ((!float_type(x_dtype) && !code_type(x_dtype)) || !float_type(y_dtype) || group != awq::kGroup ||
      (act != AWQ_ACT_GELU && act != AWQ_ACT_SILU))
    return AWQ_ERR_UNSUPPORTED;
  MoeLayout L;
  if (!moe_layout(M, E, k, H, I, &L)) return AWQ_ERR_SHAPE;
  int st = check_rows(X, x_dtype, M, H, ldx);
  if (st == AWQ_OK) st = check_rows(Y, y_dtype, M, H, ldy);
  if (st == AWQ_OK && r.logits != nullptr) st = check_route(r.logits, r.l_dtype, M, E, r.ldl, k, r.score);
  if (st != AWQ_OK) return st;
  if (code_type(x_dtype) && (xscale == nullptr || !aligned(xscale, 4))) return AWQ_ERR_INVALID_ARG;
  if (!rows_aligned(X, x_dtype, ldx, 16) || !aligned(gate_up, kAlign) || !aligned(down, kAlign) || !aligned(r.ids, 4) ||
      !aligned(r.weights, 4))
    return AWQ_ERR_INVALID_ARG;
  if (ws == nullptr || ws_bytes < L.total) return AWQ_ERR_WORKSPACE;
  if (!aligned(ws, kAlign)) return AWQ_ERR_INVALID_ARG;
  for (const void* in : {X, (const void*)xscale, (const void*)r.ids, (const void*)r.weights, r.logits, gate_up, down})
    if (in != nullptr && (Y == in || ws == in)) return AWQ_ERR_INVALID_ARG;
  if (ws == Y) return AWQ_ERR_INVALID_ARG;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  char* w = static_cast<char*>(ws);
  const int32_t* ids = r.ids;
  const float* weights = r.weights;
  awq::RouteArgs route{};
  bool here = false;  // routed inside the first kernel of the products
  if (r.logits != nullptr) {
    int32_t* wi = reinterpret_cast<int32_t*>(w + L.ids);
    float* ww = reinterpret_cast<float*>(w + L.weights);
    route = route_args(r.logits, M, E, r.ldl, k, r.score, r.renormalize, wi, ww);
    here = awq::moe_routes(M, k, (int)E);
    if (!here) {
      const hipError_t e = awq::launch_moe_route(route, r.l_dtype, s);
      if (e != hipSuccess) return map_hip(e);
    }
    ids = wi, weights = ww;
  }
  auto part = [](const void* wt, const awq::W4a8Layout& l) {
    const char* p = static_cast<const char*>(wt);
    return awq::ExpertWeights{reinterpret_cast<const uint32_t*>(p), reinterpret_cast<const uint32_t*>(p + l.steps),
                              reinterpret_cast<const float*>(p + l.powers)};
  };
  awq::MoeArgs a{};
  a.up = part(gate_up, L.up), a.down = part(down, L.down);
  a.h = reinterpret_cast<uint16_t*>(w + L.h), a.o = reinterpret_cast<float*>(w + L.o);
  a.ldx = ldx, a.ldy = ldy;
  a.k = k, a.E = (int)E, a.H = (int)H, a.I = (int)I, a.act = act;
  a.ybf16 = y_dtype == AWQ_DTYPE_BF16, a.terms = a.ybf16 ? 2 : 3;
  for (int64_t m = 0; m < M; m += L.pass) {  // the passes follow each other on the stream and share the workspace
    a.M = (int)(M - m < L.pass ? M - m : L.pass);
    a.x = static_cast<const char*>(X) + m * ldx * dsize(x_dtype);
    a.xscale = code_type(x_dtype) ? xscale + m : nullptr;
    a.ids = ids + m * k, a.weights = weights + m * k;
    a.y = static_cast<char*>(Y) + m * ldy * dsize(y_dtype);
    const hipError_t e = awq::launch_moe(a, here ? &route : nullptr, r.l_dtype, x_dtype, s);
    if (e != hipSuccess) return map_hip(e);
  }
  return AWQ_OK;
}

}  // namespace

extern "C" {

AWQ_API int awq_moe_route(const void* logits, int l_dtype, int64_t M, int64_t E, int64_t ldl, int32_t k, int score,
                          int renormalize, int32_t* ids, float* weights, awq_stream_t stream) {
  if (ids == nullptr || weights == nullptr) return AWQ_ERR_INVALID_ARG;
  const int st = check_route(logits, l_dtype, M, E, ldl, k, score);
  if (st != AWQ_OK) return st;
  if (!aligned(ids, 4) || !aligned(weights, 4) || (const void*)ids == weights || ids == logits || weights == logits)
    return AWQ_ERR_INVALID_ARG;
  return map_hip(awq::launch_moe_route(route_args(logits, M, E, ldl, k, score, renormalize, ids, weights), l_dtype,
                                       reinterpret_cast<hipStream_t>(stream)));
}

AWQ_API size_t awq_moe_workspace_bytes(int64_t M, int64_t E, int32_t k, int64_t H, int64_t I) {
  MoeLayout L;
  return moe_layout(M, E, k, H, I, &L) ? L.total : 0;
}

AWQ_API int awq_moe(const void* X, int x_dtype, const float* xscale, int64_t M, int64_t H, int64_t ldx,
                    const int32_t* ids, const float* weights, int32_t k, const void* gate_up, const void* down, int64_t E,
                    int64_t I, int32_t group, int act, void* Y, int y_dtype, int64_t ldy, void* ws, size_t ws_bytes,
                    awq_stream_t stream) {
  return run_moe(X, x_dtype, xscale, M, H, ldx, Routing{ids, weights, nullptr, 0, 0, 0, 0}, k, gate_up, down, E, I, group,
                 act, Y, y_dtype, ldy, ws, ws_bytes, stream);
}

AWQ_API int awq_moe_layer(const void* X, int x_dtype, const float* xscale, int64_t M, int64_t H, int64_t ldx,
                          const void* logits, int l_dtype, int64_t ldl, int32_t k, int score, int renormalize,
                          const void* gate_up, const void* down, int64_t E, int64_t I, int32_t group, int act, void* Y,
                          int y_dtype, int64_t ldy, void* ws, size_t ws_bytes, awq_stream_t stream) {
  if (logits == nullptr) return AWQ_ERR_INVALID_ARG;
  return run_moe(X, x_dtype, xscale, M, H, ldx, Routing{nullptr, nullptr, logits, l_dtype, ldl, score, renormalize}, k,
                 gate_up, down, E, I, group, act, Y, y_dtype, ldy, ws, ws_bytes, stream);
}

}  // extern "C"
