// How a row of the norm and the activation is held in registers, by sizes and alignment alone.  Host code without HIP:
// which kernel a size takes can be asked from a plain C++ program.
#pragma once

#include <cstdint>

namespace awq {

struct RowLayout {
  int waves, units;  // waves per row (1: four rows per block), units of eight elements per lane; waves 0: two passes
};

// The fewest registers that hold the row: few units per lane leave more rows in flight, and lanes without a
// unit read for nothing (4096 rows, silu gate, K = 14336, bf16 -> e4m3: 4 waves x 8 units 68.6 us, 4 x 7 58.7,
// 8 x 4 53.9, 16 x 2 53.1; K = 4096, rmsnorm: 1 x 8 22.8 us, 4 x 2 21.2;
// 1000 rows of 20480, rmsnorm: 16 x 4 55.6 us, 16 x 3 32.6).  Rows of any alignment take the steps that are kept.
constexpr RowLayout row_layout(int64_t M, int64_t K, bool aligned) {
  const int64_t units = K / 8;
  if (units > 16 * 64 * 4) return {0, 0};
  if (units <= 128) return {1, 2};
  if (M <= 256 && units <= 2048) return {16, units <= 1024 ? 1 : 2};  // fewer rows than CUs: each over sixteen waves
  if (aligned && units <= 256) return {4, 1};
  if (units <= 512) return {4, 2};
  if (aligned && units <= 768) return {4, 3};
  if (units <= 1024) return {4, 4};
  if (aligned && units <= 1536) return {8, 3};
  if (units <= 2048) return {16, 2};
  if (units <= 3072) return {16, 3};
  return {16, 4};
}

}  // namespace awq
