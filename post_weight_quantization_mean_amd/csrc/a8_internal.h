// Internal declarations of the 8-bit activation path (rows8.hip, w4a8.hip, a8_api.cpp).
#pragma once

#include "awq_internal.h"
#include "w4a8_plan.h"

namespace awq {

// Element types, the values of the ABI's codes; kNoOperand: an operand that is absent.
constexpr int kF32 = 0, kBf16 = 1, kI8 = 2, kE4m3 = 3, kNoOperand = -1;
constexpr int kActNone = 2;

// Blocks of a kernel that strides over its grid: as many as asked for, but fewer than 2^32 threads, a launch's limit.
inline unsigned blocks_of(int64_t blocks, int threads) {
  const int64_t most = 0xffffffffLL / threads;
  return (unsigned)(blocks < most ? blocks : most);
}

// ---- row operators (rmsnorm, act_mul) ----------------------------------------------------
struct RowArgs {
  const void* x;      // [M, K], ldx
  const void* b;      // second operand [M, K], ldb: the residual, or the gate's factor
  void* h;            // [M, K], ldh: x + b in b's type (norm), or null
  const void* col;    // [K]: gamma (norm) or s (activation), or null
  void* y;            // [M, K], ldy
  float* scale;       // [M] for an 8-bit y
  int64_t M, K, ldx, ldb, ldh, ldy;
  float eps;
  int act;            // activation
  int col_type, y_type;
};
// vec: every row of every operand starts 16-byte aligned (8-bit y: 8-byte), col 16-byte aligned,
// and K is a multiple of 8
hipError_t launch_rmsnorm(const RowArgs& a, int x_type, int b_type, bool vec, hipStream_t st);
hipError_t launch_act_mul(const RowArgs& a, int x_type, bool vec, hipStream_t st);

// ---- W4A8 --------------------------------------------------------------------------------
struct W4a8Layout {
  size_t steps, powers, total;  // byte offsets of the parts behind the codes
};
struct W4a8Args {
  const void* x;
  const float* xscale;
  const uint32_t* codes;
  const uint32_t* steps;
  const float* powers;
  void* y;
  int64_t M, K, N, ldx, ldy;
  bool e4m3, ybf16;
  int sums;  // e4m3 codes: kSumsDefault, kSumsF32, kSumsMatrix
};
hipError_t launch_w4a8_weight(const int32_t* qweight, const uint16_t* scales, const uint16_t* zeros, int64_t N,
                              int64_t K, uint32_t* codes, uint32_t* steps, float* powers, hipStream_t st);
constexpr int kW4a8TileM = 128;  // tokens of the largest tile
size_t w4a8_workspace(int64_t M, int64_t K, int64_t N);
hipError_t launch_w4a8(const W4a8Args& a, void* ws, hipStream_t st);

}  // namespace awq
