// Checks of arguments that the C entry points share.  Plain host code that runs before any HIP call.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "a8_internal.h"
#include "awq_a8.h"

namespace awq::api {

inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline bool float_type(int t) { return t == AWQ_DTYPE_F32 || t == AWQ_DTYPE_BF16; }
inline bool code_type(int t) { return t == AWQ_DTYPE_I8 || t == AWQ_DTYPE_E4M3; }
inline int64_t dsize(int t) { return t == AWQ_DTYPE_F32 ? 4 : t == AWQ_DTYPE_BF16 ? 2 : 1; }

// a * b * c, or -1 where it leaves int64 (all non-negative)
inline int64_t mul3(int64_t a, int64_t b, int64_t c) {
  int64_t ab = 0, abc = 0;
  if (__builtin_mul_overflow(a, b, &ab) || __builtin_mul_overflow(ab, c, &abc)) return -1;
  return abc;
}

// One [M, K] operand with row stride ld (elements) of a supported type.
inline int check_rows(const void* p, int type, int64_t M, int64_t K, int64_t ld) {
  if (p == nullptr || ld < K || !aligned(p, (uintptr_t)dsize(type))) return AWQ_ERR_INVALID_ARG;
  if (mul3(M, ld, dsize(type)) < 0) return AWQ_ERR_SHAPE;
  return AWQ_OK;
}

// Rows whose starts are n-byte aligned.
inline bool rows_aligned(const void* p, int type, int64_t ld, int64_t n) {
  return aligned(p, (uintptr_t)n) && (ld * dsize(type)) % n == 0;
}

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// A launch takes fewer than 2^32 threads: 512 per 32 channels at most.
constexpr int64_t kMaxN = 1 << 27;

// The parts of a weight of N channels as awq_w4a8_weight lays it out; false where it refuses the sizes.
inline bool w4a8_layout(int64_t N, int64_t K, W4a8Layout* L) {
  if (N <= 0 || N > kMaxN || K <= 0 || K % kGroup != 0) return false;
  const int64_t rows = w4a8_tiles(N) * 16;
  if (mul3(rows, K, 2) < 0) return false;
  L->steps = align_up((size_t)(rows * (K / 2)));
  L->powers = L->steps + align_up((size_t)(rows * (K / kGroup) * 4));
  L->total = L->powers + align_up((size_t)(rows * 4));
  return true;
}

inline int map_hip(hipError_t e) { return e == hipSuccess ? AWQ_OK : AWQ_ERR_HIP; }

}  // namespace awq::api
