// The product of 8-bit activations with the packed 4-bit weight:
//   Y[m, n] = xscale[m] sum_g D[n, g] sum_{k in g} x[m, k] (q[n, k] - z[n, g])
// on the 8-bit matrix cores, which multiply a group's 128 channels of 16 tokens with 16 output channels in
// one instruction (e4m3: 16x16x128) or two (int8: 16x16x64).
//
// The codes need no conversion: 0 .. 15 as an int8 byte is the code, and as an e4m3 byte (bits b < 16:
// the subnormals b 2^-9 and the first normal binade, which continues them) exactly q 2^-9.  A word of eight
// codes becomes two operand words with three instructions.  The zero point is taken out of the sums:
//   sum x (q - z) = sum x q - z sum x.
// int8 sums are exact integers below 2^18; e4m3 products are exact in fp32 and their sums round as fp32's.
//
// The weight is laid out once (awq_w4a8_weight): the 16 bytes of lane l for one tile of 16 channels and one
// group are contiguous over the lanes, so a tile's group is one 1 KiB load of a wave, in operand order.
// Within a lane's 32 channels the sum over k runs in the order of the bytes, the same for both operands.
#include "a8_internal.h"

namespace awq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float h2f(uint32_t h) { return (float)__builtin_bit_cast(_Float16, (uint16_t)h); }
__device__ __forceinline__ uint16_t f2h(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
__device__ __forceinline__ uint16_t to_bf16(float x) {
  return (uint16_t)__builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){x, x}, bf16x2));
}

// ---- the weight's layout --------------------------------------------------------------------------
// One thread per word of the laid-out codes.
__global__ __launch_bounds__(256) void w4a8_codes_kernel(const uint32_t* __restrict__ qweight, int64_t N, int64_t K,
                                                         int64_t words, uint32_t* __restrict__ codes) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= words) return;
  const int64_t G = K / kGroup, tg = i / 256;
  const int l = (int)(i % 256) / 4, w = (int)(i % 4);
  const int64_t n = (tg / G) * 16 + l % 16, k = (tg % G) * kGroup + 32 * (l / 16) + 8 * w;
  uint32_t out = 0;
  if (n < N) {
    const uint32_t q = qweight[n * (K / 8) + k / 8];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      out |= ((q >> (4 * b)) & 15u) << (8 * b);
      out |= ((q >> (4 * b + 16)) & 15u) << (8 * b + 4);
    }
  }
  codes[i] = out;
}

// One thread per channel: the power of two that takes its largest step into [2^10, 2^11) (there a step
// times a zero point, at most 15 2^11, is a finite fp16, and only steps below 2^-25 of the largest lose
// bits), then its steps and zero points.
__global__ __launch_bounds__(256) void w4a8_steps_kernel(const uint16_t* __restrict__ scales,
                                                         const uint16_t* __restrict__ zeros, int64_t N, int64_t G,
                                                         int64_t rows, uint32_t* __restrict__ steps,
                                                         float* __restrict__ powers) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= rows) return;
  float top = 0.0f;
  if (n < N)
    for (int64_t g = 0; g < G; ++g) top = fmaxf(top, fabsf(h2f(scales[n * G + g])));
  int e = 0;
  if (top > 0.0f && top < __builtin_inff()) {
    frexpf(top, &e);  // top in [2^(e-1), 2^e)
    e -= 11;
  }
  const float down = ldexpf(1.0f, -e);
  for (int64_t g = 0; g < G; ++g) {
    uint32_t v = 0;
    if (n < N) v = f2h(h2f(scales[n * G + g]) * down) | (uint32_t)zeros[n * G + g] << 16;
    steps[((n / 16) * G + g) * 16 + n % 16] = v;
  }
  powers[n] = ldexpf(1.0f, e);
}

// ---- operand pieces ---------------------------------------------------------------------------------
// eight operand words (32 channels) of a lane from its four words of codes
__device__ __forceinline__ i32x8 unpack_codes(const u32x4 w) {
  i32x8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[2 * i] = (int)(w[i] & 0x0f0f0f0fu);
    r[2 * i + 1] = (int)((w[i] >> 4) & 0x0f0f0f0fu);
  }
  return r;
}

constexpr float kE4m3Unit = 0x1p-9f;  // an e4m3 byte b < 16 is b times this

// One group's products of 16 tokens and 16 channels: lane l gets channel l % 16 of tokens 4 (l / 16) + i
// (fp32; int8: exact integers; e4m3: times 2^-9 with codes as b).
template <bool E4M3>
__device__ __forceinline__ f32x4 group_product(const i32x8 a, const i32x8 b) {
  if constexpr (E4M3) {
    const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
  } else {
    const i32x4 z = {0, 0, 0, 0};
    const i32x4 alo = __builtin_shufflevector(a, a, 0, 1, 2, 3), ahi = __builtin_shufflevector(a, a, 4, 5, 6, 7);
    const i32x4 blo = __builtin_shufflevector(b, b, 0, 1, 2, 3), bhi = __builtin_shufflevector(b, b, 4, 5, 6, 7);
    i32x4 r = __builtin_amdgcn_mfma_i32_16x16x64_i8(alo, blo, z, 0, 0, 0);
    r = __builtin_amdgcn_mfma_i32_16x16x64_i8(ahi, bhi, r, 0, 0, 0);
    return (f32x4){(float)r[0], (float)r[1], (float)r[2], (float)r[3]};
  }
}

// ---- few tokens: the weight as a stream ----------------------------------------------------------------
// A block computes CT tiles of 16 channels for up to 16 TT tokens over all of K.  Its eight waves take the
// groups in turn, each with its own fp32 sums, which meet in LDS at the end in wave order.  Sum x per
// token and group is one more product, with ones, in the layout of the sums it corrects.  Rows past the
// last token repeat it and are not stored.
constexpr int kStWaves = 8;

template <bool E4M3, int TT, int CT>
__global__ __launch_bounds__(64 * kStWaves) void w4a8_stream_kernel(const W4a8Args p) {
  __shared__ float part[kStWaves][TT * CT * 256];
  const int lane = threadIdx.x & 63, j = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t G = p.K / kGroup, tiles = (p.N + 15) / 16;
  const int64_t t0 = (int64_t)blockIdx.x * CT, m0 = (int64_t)blockIdx.y * (16 * TT);
  const uint8_t* xrow[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int64_t m = m0 + 16 * t + c;
    xrow[t] = static_cast<const uint8_t*>(p.x) + (m < p.M ? m : p.M - 1) * p.ldx + 32 * j;
  }
  const uint32_t* wrow[CT];
  const uint32_t* srow[CT];
#pragma unroll
  for (int q = 0; q < CT; ++q) {
    const int64_t tile = t0 + q < tiles ? t0 + q : tiles - 1;  // past the last tile: loaded, not stored
    wrow[q] = p.codes + tile * G * 256 + 4 * lane;
    srow[q] = p.steps + tile * G * 16 + c;
  }
  i32x8 ones;
#pragma unroll
  for (int i = 0; i < 8; ++i) ones[i] = E4M3 ? 0x38383838 : 0x01010101;
  f32x4 tot[TT][CT];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int q = 0; q < CT; ++q) tot[t][q] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
  for (int64_t g = wave; g < G; g += kStWaves) {
    u32x4 w[CT], xa[TT][2];
    uint32_t dz[CT];
#pragma unroll
    for (int q = 0; q < CT; ++q) {
      w[q] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wrow[q] + g * 256));
      dz[q] = srow[q][g * 16];
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      xa[t][0] = *reinterpret_cast<const u32x4*>(xrow[t] + g * kGroup);
      xa[t][1] = *reinterpret_cast<const u32x4*>(xrow[t] + g * kGroup + 16);
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const i32x8 a = {(int)xa[t][0][0], (int)xa[t][0][1], (int)xa[t][0][2], (int)xa[t][0][3],
                       (int)xa[t][1][0], (int)xa[t][1][1], (int)xa[t][1][2], (int)xa[t][1][3]};
      const f32x4 sx = group_product<E4M3>(a, ones);
#pragma unroll
      for (int q = 0; q < CT; ++q) {
        const f32x4 s = group_product<E4M3>(a, unpack_codes(w[q]));
        const float d = h2f(dz[q] & 0xffffu) * (E4M3 ? 1.0f / kE4m3Unit : 1.0f);
        const float z = h2f(dz[q] >> 16) * (E4M3 ? kE4m3Unit : 1.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[t][q][i] = fmaf(d, fmaf(-z, sx[i], s[i]), tot[t][q][i]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int q = 0; q < CT; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][((t * 16 + 4 * j + i) * CT + q) * 16 + c] = tot[t][q][i];
  __syncthreads();
  for (int o = threadIdx.x; o < TT * CT * 256; o += 64 * kStWaves) {
    const int64_t m = m0 + o / (16 * CT), n = t0 * 16 + o % (16 * CT);
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kStWaves; ++w) s += part[w][o];
    if (m < p.M && n < p.N) {
      const float y = s * (p.xscale[m] * p.powers[n]);
      if (p.ybf16) static_cast<uint16_t*>(p.y)[m * p.ldy + n] = to_bf16(y);
      else static_cast<float*>(p.y)[m * p.ldy + n] = y;
    }
  }
}

template <bool E4M3>
hipError_t launch_stream(const W4a8Args& a, hipStream_t st) {
  const int64_t tiles = w4a8_tiles(a.N);
#define AWQ_ST(TTV, CTV)                                                                            \
  w4a8_stream_kernel<E4M3, TTV, CTV>                                                                \
      <<<dim3((unsigned)((tiles + CTV - 1) / CTV), (unsigned)((a.M + 16 * TTV - 1) / (16 * TTV))),  \
         64 * kStWaves, 0, st>>>(a)
  if (a.M <= 16) AWQ_ST(1, 1);
  else if (a.M <= 32) AWQ_ST(2, 1);
  else AWQ_ST(4, 1);
#undef AWQ_ST
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w4a8_weight(const int32_t* qweight, const uint16_t* scales, const uint16_t* zeros, int64_t N,
                              int64_t K, uint32_t* codes, uint32_t* steps, float* powers, hipStream_t st) {
  const int64_t rows = w4a8_tiles(N) * 16, words = rows * (K / 8);
  if ((words + 255) / 256 > 0x7fffffff) return hipErrorInvalidValue;
  w4a8_codes_kernel<<<(unsigned)((words + 255) / 256), 256, 0, st>>>(reinterpret_cast<const uint32_t*>(qweight), N, K,
                                                                     words, codes);
  w4a8_steps_kernel<<<(unsigned)((rows + 255) / 256), 256, 0, st>>>(scales, zeros, N, K / kGroup, rows, steps, powers);
  return hipGetLastError();
}

size_t w4a8_workspace(int64_t M, int64_t K, int64_t N) { return 0; }

hipError_t launch_w4a8(const W4a8Args& a, void* ws, hipStream_t st) {
  return a.e4m3 ? launch_stream<true>(a, st) : launch_stream<false>(a, st);
}

}  // namespace awq
