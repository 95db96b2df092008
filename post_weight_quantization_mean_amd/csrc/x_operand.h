// Activations as operands of the bf16 matrix cores, exactly: bf16 as it stands, int8 and e4m3 codes converted (both fit
// bf16's eight bits), fp32 as three bf16 terms of eight bits each.
#pragma once

#include "a8_internal.h"

namespace awq {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t bits(float f) { return __builtin_bit_cast(uint32_t, f); }
__device__ __forceinline__ float flt(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ float half_lo(uint32_t h) { return (float)__builtin_bit_cast(_Float16, (uint16_t)h); }
// two fp32 to two bf16, rounded to nearest even, or cut to the upper halves (exact where eight bits hold the value)
__device__ __forceinline__ uint32_t pack_rne(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}
__device__ __forceinline__ uint32_t pack_cut(float a, float b) {
  return __builtin_amdgcn_perm(bits(b), bits(a), 0x07060302);
}
__device__ __forceinline__ float cut(float v) { return flt(bits(v) & 0xffff0000u); }

// Eight consecutive channels of one row.
template <int XT>
struct X8 {
  static constexpr int kWords = XT == kF32 ? 8 : XT == kBf16 ? 4 : 2, kTerms = XT == kF32 ? 3 : 1;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const char* p) {  // aligned to 16 bytes (8-bit codes: 8)
    if constexpr (kWords == 2) {
      const u32x2 v = *reinterpret_cast<const u32x2*>(p);
      w[0] = v[0], w[1] = v[1];
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const u32x4 v = reinterpret_cast<const u32x4*>(p)[i];
        w[4 * i] = v[0], w[4 * i + 1] = v[1], w[4 * i + 2] = v[2], w[4 * i + 3] = v[3];
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // The terms, whose sum is the eight channels.  fp32: the value cut to eight bits, what is left cut to eight, the rest;
  // every difference is exact.
  __device__ __forceinline__ void terms(bf16x8 (&t)[kTerms]) const {
    u32x4 o[kTerms];
    if constexpr (XT == kBf16) {
      o[0] = (u32x4){w[0], w[1], w[2], w[3]};
    } else if constexpr (XT == kF32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = flt(w[2 * i]), b = flt(w[2 * i + 1]);
        const float a1 = a - cut(a), b1 = b - cut(b);
        o[0][i] = pack_cut(a, b);
        o[1][i] = pack_cut(a1, b1);
        o[2][i] = pack_cut(a1 - cut(a1), b1 - cut(b1));
      }
    } else if constexpr (XT == kI8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int v = (int)w[i / 2] << (i % 2 ? 0 : 16);
        o[0][i] = pack_cut((float)(int8_t)(v >> 16), (float)(v >> 24));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[0][i] = __builtin_bit_cast(uint32_t, i % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i / 2], 1.0f, true)
                                                     : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i / 2], 1.0f, false));
    }
#pragma unroll
    for (int i = 0; i < kTerms; ++i) t[i] = __builtin_bit_cast(bf16x8, o[i]);
  }
};

// Eight fp32 values as T bf16 terms: all but the last cut, the last rounded (T = 2: 2^-17 of the value; 3: exact).
template <int T>
__device__ __forceinline__ void split_terms(const float (&v)[8], bf16x8 (&t)[T]) {
  u32x4 o[T];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = v[2 * i], b = v[2 * i + 1];
#pragma unroll
    for (int s = 0; s < T - 1; ++s) {
      o[s][i] = pack_cut(a, b);
      a -= cut(a), b -= cut(b);
    }
    o[T - 1][i] = pack_rne(a, b);
  }
#pragma unroll
  for (int s = 0; s < T; ++s) t[s] = __builtin_bit_cast(bf16x8, o[s]);
}

}  // namespace awq
