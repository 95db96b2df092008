// Internal declarations of the low-rank adapters (lora.hip, lora_api.cpp).
#pragma once

#include "a8_internal.h"

namespace awq {

struct LoraArgs {
  const void* x;         // [M, K], ldx
  const float* xscale;   // [M] for codes, else null
  const uint16_t* a;     // [n, R, K]
  const uint16_t* b;     // [n, N, R]
  const int32_t* ids;    // [M]
  const float* scale;    // [n] or null
  const int32_t* ranks;  // [n] or null
  const void* base;      // [M, N], ldb
  void* y;               // [M, N], ldy
  float* t;              // [splits, M, R]: scale (A x), in parts over K
  int64_t M, K, N, ldx, ldb, ldy;
  int n, R, splits;
  bool ybf16, vec;  // vec: rows of base and y start 16-byte aligned
};
int lora_splits(int64_t M, int64_t K, int64_t R);
hipError_t launch_lora(const LoraArgs& a, int x_type, hipStream_t st);

}  // namespace awq
