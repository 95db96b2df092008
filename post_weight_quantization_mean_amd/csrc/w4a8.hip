// The product of 8-bit activations with the packed 4-bit weight:
//   Y[m, n] = xscale[m] sum_g D[n, g] sum_{k in g} x[m, k] (q[n, k] - z[n, g])
// on the 8-bit matrix cores, which multiply a group's 128 channels of 16 tokens with 16 output channels in
// one instruction (e4m3: 16x16x128) or two (int8: 16x16x64).
//
// The codes need no conversion: 0 .. 15 as an int8 byte is the code, and as an e4m3 byte (bits b < 16:
// the subnormals b 2^-9 and the first normal binade, which continues them) exactly q 2^-9.  A word of eight
// codes becomes two operand words with three instructions.  The zero point is taken out of the sums:
//   sum x (q - z) = sum x q - z sum x.
// int8 sums are exact integers below 2^18; e4m3 products are exact, their sums as kE4m3Fast and kE4m3Wide say.
// A result is (sum 2^e) xscale: the first product is exact (e in -35 .. 6 and |sum| far from both ends), so a row
// whose scale is at either end of fp32 loses nothing.
//
// The weight is laid out once (awq_w4a8_weight): the 16 bytes of lane l for one tile of 16 channels and one
// group are contiguous over the lanes, so a tile's group is one 1 KiB load of a wave, in operand order.
// Lane l's 32 channels of a group are 16 (l / 16) .. + 15 and the same 64 further on, for both operands: one read of
// 16 bytes by the lanes of a row then covers 64 whole bytes (16 x 14336 -> 4096: 11.1 us against 12.4 with 32
// channels in a row per lane).
#include "a8_internal.h"
static_assert(awq::kW4a8Group == awq::kGroup, "one group size");

namespace awq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float h2f(uint32_t h) { return (float)__builtin_bit_cast(_Float16, (uint16_t)h); }
__device__ __forceinline__ uint16_t f2h(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
__device__ __forceinline__ uint16_t to_bf16(float x) {
  return (uint16_t)__builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){x, x}, bf16x2));
}

// ---- the weight's layout --------------------------------------------------------------------------
// A thread per word of the laid-out codes (several from 2^32 words on).
__global__ __launch_bounds__(256) void w4a8_codes_kernel(const uint32_t* __restrict__ qweight, int64_t N, int64_t K,
                                                         int64_t words, uint32_t* __restrict__ codes) {
  const int64_t G = K / kGroup;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) {
    const int64_t tg = i / 256;
    const int l = (int)(i % 256) / 4, w = (int)(i % 4);
    const int64_t n = (tg / G) * 16 + l % 16, k = (tg % G) * kGroup + 16 * (l / 16) + 64 * (w / 2) + 8 * (w % 2);
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
}

// Sixteen threads per channel: the power of two that takes its largest step into [2^10, 2^11) (there a step
// times a zero point, at most 15 2^11, is a finite fp16, and only steps below 2^-24 of the largest, subnormal then,
// lose bits), then its steps and zero points.  (4096 channels of 112 groups: 6 us; one thread each: 39.)
__global__ __launch_bounds__(256) void w4a8_steps_kernel(const uint16_t* __restrict__ scales,
                                                         const uint16_t* __restrict__ zeros, int64_t N, int64_t G,
                                                         uint32_t* __restrict__ steps, float* __restrict__ powers) {
  const int64_t n = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);  // the grid covers whole tiles of 16 channels
  const int part = threadIdx.x & 15;
  float top = 0.0f;
  if (n < N)
    for (int64_t g = part; g < G; g += 16) top = fmaxf(top, fabsf(h2f(scales[n * G + g])));
#pragma unroll
  for (int i = 1; i < 16; i *= 2) top = fmaxf(top, __shfl_xor(top, i, 16));
  int e = 0;
  if (top > 0.0f && top < __builtin_inff()) {
    frexpf(top, &e);  // top in [2^(e-1), 2^e)
    e -= 11;
  }
  const float down = ldexpf(1.0f, -e);
  for (int64_t g = part; g < G; g += 16) {
    uint32_t v = 0;
    if (n < N) v = f2h(h2f(scales[n * G + g]) * down) | (uint32_t)zeros[n * G + g] << 16;
    steps[((n / 16) * G + g) * 16 + n % 16] = v;
  }
  if (part == 0) powers[n] = ldexpf(1.0f, e);
}

#define AWQ_INLINE __attribute__((always_inline))

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

// How a group's products are formed.  The e4m3 matrix instruction adds 16 products at a time after
// shifting them to the largest one's exponent and keeps 14 bits there (measured; the sums of 16 then add in
// fp32): about 2^-13 of the largest product.  On activations with 1% of channels 10 to 50 times the others that
// adds 2e-4 (rms, relative) to a bf16 result's rounding of 1.7e-3; where a large code's q is its zero point, so that
// its product cancels, what is lost beside it can be more than that rounding.  And the results that round another way
// for it turn codes behind them: an MLP in e4m3 (40 tokens) ends 4.4e-3 from its value in 64 bits, 2.1e-3 with fp32 sums.
// kE4m3Wide converts both operands to bf16 (exactly) and adds in fp32, at half the matrix rate.  matrix_sums says which is
// taken.
constexpr int kInt8 = 0, kE4m3Fast = 1, kE4m3Wide = 2;

template <int KIND>
struct Operand {
  i32x8 b;  // 32 bytes
};
template <>
struct Operand<kE4m3Wide> {
  bf16x8 h[4];  // the same 32 values, 8 bytes at a time
};
template <int KIND>
__device__ __forceinline__ Operand<KIND> operand(const i32x8 b) {
  Operand<KIND> r;
  if constexpr (KIND == kE4m3Wide) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4 w;
#pragma unroll
      for (int d = 0; d < 4; ++d)
        w[d] = __builtin_bit_cast(uint32_t, d & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b[2 * s + d / 2], 1.0f, true)
                                                   : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b[2 * s + d / 2], 1.0f, false));
      r.h[s] = __builtin_bit_cast(bf16x8, w);
    }
  } else {
    r.b = b;
  }
  return r;
}

// One group's products of 16 tokens and 16 channels: lane l gets channel l % 16 of tokens 4 (l / 16) + i,
// as settled<KIND>(r[i]) (int8: exact integers; e4m3: times 2^-9 with codes as b).  In two parts, the second of
// which continues the first's sums (kE4m3Fast: all in the first).
template <int KIND>
__device__ __forceinline__ f32x4 product_begin(const Operand<KIND>& a, const Operand<KIND>& b) {
  const f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (KIND == kE4m3Fast) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.b, b.b, z, 0, 0, 0, 0, 0, 0);
  } else if constexpr (KIND == kE4m3Wide) {
    const f32x4 r = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.h[0], b.h[0], z, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.h[1], b.h[1], r, 0, 0, 0);
  } else {
    // the sums start at the bits of 1.5 2^23: |sum| < 2^22 more is that float plus the sum, so that a
    // full-rate subtraction stands for the conversion
    constexpr int kBits = 0x4b400000;
    const i32x4 zi = {kBits, kBits, kBits, kBits};
    const i32x4 alo = __builtin_shufflevector(a.b, a.b, 0, 1, 2, 3), blo = __builtin_shufflevector(b.b, b.b, 0, 1, 2, 3);
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_mfma_i32_16x16x64_i8(alo, blo, zi, 0, 0, 0));
  }
}
template <int KIND>
__device__ __forceinline__ f32x4 product_end(const Operand<KIND>& a, const Operand<KIND>& b, const f32x4 r) {
  if constexpr (KIND == kE4m3Fast) {
    return r;
  } else if constexpr (KIND == kE4m3Wide) {
    const f32x4 s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.h[2], b.h[2], r, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.h[3], b.h[3], s, 0, 0, 0);
  } else {
    const i32x4 ahi = __builtin_shufflevector(a.b, a.b, 4, 5, 6, 7), bhi = __builtin_shufflevector(b.b, b.b, 4, 5, 6, 7);
    return __builtin_bit_cast(
        f32x4, __builtin_amdgcn_mfma_i32_16x16x64_i8(ahi, bhi, __builtin_bit_cast(i32x4, r), 0, 0, 0));
  }
}
template <int KIND>
__device__ __forceinline__ f32x4 group_product(const Operand<KIND>& a, const Operand<KIND>& b) {
  return product_end<KIND>(a, b, product_begin<KIND>(a, b));
}
template <int KIND>
__device__ __forceinline__ float settled(float r) { return KIND == kInt8 ? r - 12582912.0f : r; }

__device__ __forceinline__ i32x8 join(const u32x4 lo, const u32x4 hi) {
  return (i32x8){(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// ---- few tokens: the weight as a stream ----------------------------------------------------------------
// A block computes CT tiles of 16 channels for up to 16 TT tokens over all of K.  Its WV waves take the
// groups in turn, D of them in flight in each wave, with fp32 sums of their own, which meet in LDS at the
// end in wave order.  Bound: up to 8 tokens by the weight's bytes and the time until they flow (1 x 4096 -> 28672:
// 12.3 us, 5.1 TB/s, what a copy reaches; 1 and 5 x 14336 -> 4096: 8.0, 256 blocks of seven groups a wave), in e4m3
// with fp32 sums by the conversions to bf16 where each block has two channel tiles (16.5 and 8.7); beyond, by
// the reads of X from L2 too, 2 KiB per wave, group and 16 tokens: with every token's lanes reading the first token
// instead, us, 16 x 14336 -> 4096 takes 7.9 for 10.8, 16 x 4096 -> 28672 12.4 / 15.2, 64 x 4096 -> 4096 5.3 / 7.1,
// 101 x 4096 -> 6144 9.0 / 13.0, 256 x 4096 -> 4096 10.1 / 14.6.  Sum x per token and group is one more product, with
// ones, in the layout of the
// sums it corrects.  Rows past the last token repeat it and are not stored.
template <int KIND, int TT, int CT, int WV, int D>
__global__ __launch_bounds__(64 * WV) void w4a8_stream_kernel(const W4a8Args p) {
  __shared__ float part[WV][CT * 256];
  const int lane = threadIdx.x & 63, j = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = (int)(p.K / kGroup);
  const int64_t tiles = (p.N + 15) / 16;
  const int64_t t0 = (int64_t)blockIdx.x * CT, m0 = (int64_t)blockIdx.y * (16 * TT);
  const uint8_t* xbase = static_cast<const uint8_t*>(p.x) + m0 * p.ldx;
  uint32_t xoff[TT];  // less than 2^31: host-checked
#pragma unroll
  for (int t = 0; t < TT; ++t)
    xoff[t] = (uint32_t)((m0 + 16 * t + c < p.M ? 16 * t + c : (int)(p.M - 1 - m0)) * p.ldx + 16 * j);
  const uint32_t* wrow[CT];
  const uint32_t* srow[CT];
#pragma unroll
  for (int q = 0; q < CT; ++q) {
    const int64_t tile = t0 + q < tiles ? t0 + q : tiles - 1;  // past the last tile: loaded, not stored
    wrow[q] = p.codes + tile * G * 256;
    srow[q] = p.steps + tile * G * 16;
  }
  constexpr bool E4M3 = KIND != kInt8;
  constexpr int kOne = E4M3 ? 0x38383838 : 0x01010101;
  const Operand<KIND> ones = operand<KIND>((i32x8){kOne, kOne, kOne, kOne, kOne, kOne, kOne, kOne});
  f32x4 tot[TT][CT];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int q = 0; q < CT; ++q) tot[t][q] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  struct Group {
    u32x4 w[CT], x[TT][2];
    uint32_t dz[CT];
  } buf[D];
  auto fetch = [&](Group& b, int i) AWQ_INLINE {  // this wave's i-th group
    const int64_t g = wave + i * WV;
#pragma unroll
    for (int q = 0; q < CT; ++q) {
      b.w[q] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wrow[q] + g * 256) + (unsigned)lane);
      b.dz[q] = (srow[q] + g * 16)[(unsigned)c];
    }
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) b.x[t][h] = *reinterpret_cast<const u32x4*>(xbase + g * kGroup + 64 * h + xoff[t]);
  };
  auto use = [&](const Group& b) AWQ_INLINE {
    Operand<KIND> w[CT];
    float d[CT], z[CT];
    auto unpack = [&](int q) AWQ_INLINE {
      w[q] = operand<KIND>(unpack_codes(b.w[q]));
      d[q] = h2f(b.dz[q] & 0xffffu) * (E4M3 ? 1.0f / kE4m3Unit : 1.0f);
      z[q] = h2f(b.dz[q] >> 16) * (E4M3 ? kE4m3Unit : 1.0f);
    };
    // one token tile: each channel tile's codes are unpacked just before its product (int8, 1 x 4096 -> 28672: 12.6
    // us against 13.2); several: all of them first (101 x 4096 -> 6144: 13.7 against 14.0)
    if constexpr (TT > 1) {
#pragma unroll
      for (int q = 0; q < CT; ++q) unpack(q);
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const Operand<KIND> a = operand<KIND>(join(b.x[t][0], b.x[t][1]));
      const f32x4 sx = group_product<KIND>(a, ones);
#pragma unroll
      for (int q = 0; q < CT; ++q) {
        if constexpr (TT == 1) unpack(q);
        const f32x4 s = group_product<KIND>(a, w[q]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          tot[t][q][i] = fmaf(d[q], fmaf(-z[q], settled<KIND>(sx[i]), settled<KIND>(s[i])), tot[t][q][i]);
      }
    }
  };
  const int n = (G - wave + WV - 1) / WV;  // this wave's groups (none or fewer where G < wave)
#pragma unroll
  for (int i = 0; i < D; ++i)
    if (i < n) fetch(buf[i], i);
  int i0 = 0;
  for (; i0 + 2 * D <= n; i0 += D)
#pragma unroll
    for (int i = 0; i < D; ++i) {
      use(buf[i]);
      fetch(buf[i], i0 + i + D);
    }
#pragma unroll
  for (int i = 0; i < D; ++i) {
    if (i0 + i < n) use(buf[i]);
    if (i0 + i + D < n) fetch(buf[i], i0 + i + D);
  }
#pragma unroll
  for (int i = 0; i < D; ++i)
    if (i0 + i + D < n) use(buf[i]);
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    if (t > 0) __syncthreads();
#pragma unroll
    for (int q = 0; q < CT; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][((4 * j + i) * CT + q) * 16 + c] = tot[t][q][i];
    __syncthreads();
    for (int o = threadIdx.x; o < CT * 256; o += 64 * WV) {
      const int64_t m = m0 + 16 * t + o / (16 * CT), nn = t0 * 16 + o % (16 * CT);
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < WV; ++w) s += part[w][o];
      if (m < p.M && nn < p.N) {
        const float y = s * p.powers[nn] * p.xscale[m];
        if (p.ybf16) static_cast<uint16_t*>(p.y)[m * p.ldy + nn] = to_bf16(y);
        else static_cast<float*>(p.y)[m * p.ldy + nn] = y;
      }
    }
  }
}

template <int KIND>
hipError_t launch_stream(const W4a8Args& a, const Plan& pl, hipStream_t st) {
  const int64_t tiles = w4a8_tiles(a.N);
  const dim3 grid((unsigned)((tiles + pl.ct - 1) / pl.ct), (unsigned)((a.M + 16 * pl.tm - 1) / (16 * pl.tm)));
  if (pl.tm == 1 && pl.ct == 2) w4a8_stream_kernel<KIND, 1, 2, 8, 2><<<grid, 512, 0, st>>>(a);
  else if (pl.tm == 1) w4a8_stream_kernel<KIND, 1, 1, 16, 2><<<grid, 1024, 0, st>>>(a);
  else if (pl.ct == 2) w4a8_stream_kernel<KIND, 2, 2, 8, 1><<<grid, 512, 0, st>>>(a);
  else if (pl.ct == 3 && pl.waves == 8) w4a8_stream_kernel<KIND, 2, 3, 8, 1><<<grid, 512, 0, st>>>(a);
  else if (pl.ct == 3) w4a8_stream_kernel<KIND, 2, 3, 4, 1><<<grid, 256, 0, st>>>(a);
  else if (pl.waves == 8) w4a8_stream_kernel<KIND, 2, 4, 8, 1><<<grid, 512, 0, st>>>(a);
  else w4a8_stream_kernel<KIND, 2, 4, 4, 1><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

// ---- many tokens: tiles -----------------------------------------------------------------------------
// sums[m][g]: sum of row m's codes of group g, formed in fp32 and kept as two fp16, high = rne(s) and low =
// rne(s - high), zero for g in G .. Gp - 1.  high leaves at most 2^-11 of s's binade, low 2^-12 of what high left:
// s to 2^-23, twice fp32's own half step (an int8 sum, and an e4m3 sum of up to 23 bits, is exact).  A third part would
// hold all 24 bits, for one more round of products every eight groups and twice the workspace; each e4m3 sum of
// 128 products beside it rounds many times that.  Eight lanes per group, 16 bytes each.
template <bool E4M3>
__global__ __launch_bounds__(256) void w4a8_sums_kernel(const uint8_t* __restrict__ x, int64_t M, int64_t ldx,
                                                        int64_t G, int64_t Gp, uint32_t* __restrict__ sums) {
  const int piece = threadIdx.x & 7;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 8; i < M * Gp; i += (int64_t)gridDim.x * 32) {
    const int64_t m = i / Gp, g = i - m * Gp;
    float s = 0.0f;
    if (g < G) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(x + m * ldx + g * kGroup + 16 * piece);
      if constexpr (E4M3) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(v[d], false), b = __builtin_amdgcn_cvt_pk_f32_fp8(v[d], true);
          s += (a[0] + a[1]) + (b[0] + b[1]);
        }
      } else {
        int t = 0;
#pragma unroll
        for (int d = 0; d < 4; ++d) t = __builtin_amdgcn_sdot4((int)v[d], 0x01010101, t, false);
        s = (float)t;
      }
    }
    s += dpp<kDppXor1>(s);
    s += dpp<kDppXor2>(s);
    s += dpp<kDppHalfMirror>(s);
    if (piece == 0) {
      const uint16_t hi = f2h(s);
      sums[i] = hi | (uint32_t)f2h(s - h2f(hi)) << 16;
    }
  }
}

// A block of four waves, one per SIMD, computes 16 TM tokens x 256 channels, and two blocks share a CU; wave wn has
// all the tokens and 64 of the channels and takes one group a step.  The tokens' bytes (128 per row and group)
// and the groups' steps come into LDS by DMA in four stages; the codes, which no other wave of the block needs,
// come straight into registers in operand order, one or two groups ahead.  The barrier of step g says that stages g
// and g + 1 have landed, so that the last products of a step run beside the reads for the first ones of
// the next; stage g + 2 is under way and g + 3 is requested.
// Rows of 128 bytes hold their 16-byte pieces at piece ^ (row % 8) ^ (row / 8 % 2): the reads of sixteen
// rows' same piece then use every bank once.
//
// Per group and 16 x 16 outputs the matrix unit works 32 cycles on the product and the vector unit 8
// on the steps' multiply-adds (int8: 16); unpacking adds 12 instructions per channel tile and wave,
// spread over TM products.  The zero points would cost as many multiply-adds
// again; their sum over groups is a product of its own, sum_g sums[m, g] (D z)[n, g], and runs on the matrix
// cores in fp16 with both operands as high and low parts (sums to 2^-23, D z 15 bits: exact), one
// instruction of 16 cycles for eight groups.
//
// 4096 x 4096 -> 28672, by box: e4m3 434 to 462 us (2.1 to 2.2 PFLOP/s), int8 484 to 520 (1.9 to 2.0), e4m3 in fp32
// sums 830 to 875 (1.1: bf16's matrix rate, with 64-token tiles and both operands converted in every wave).  A loop of
// nothing but such products and multiply-adds runs at 4.0 (e4m3) and 2.9 (int8), a library product without steps at 3.1 and 2.55.  The clock is
// down to 1.7 .. 2.0 GHz under this load.  4096 x 11008 -> 4096, e4m3, 169 us: 149 without the codes' loads, 132
// without the copies into LDS, 117 without both, 102 without the zero points' part too: what bounds it is the
// operands' way from L2 (32 KiB a block and step, and the power it takes), then the products.
template <int TM>
constexpr int kTileStage = 16 * TM * 128 + 1024;

__device__ __forceinline__ int row_swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }
#define AWQ_LDS_A8 __attribute__((address_space(3)))

template <int KIND, int TM>
__global__ __launch_bounds__(256, 2) void w4a8_tile_kernel(const W4a8Args p, const uint32_t* __restrict__ sums,
                                                           int64_t Gp, int mtiles, int ntiles) {
  constexpr bool E4M3 = KIND != kInt8;
  constexpr int STAGE = kTileStage<TM>, SOFF = 16 * TM * 128;
  constexpr int NDMA = TM / 2 + 1;  // copies per wave and stage
  // groups that the codes are requested ahead: two, but for the case whose registers one fills (256 tiles of 64 tokens, G =
  // 86: 60.4 us against 62.6; 896 of 128: 439.9 / 442.5; four ahead: no change)
  constexpr int AHEAD = TM == 8 && KIND == kInt8 ? 1 : 2;
  __shared__ __attribute__((aligned(1024))) uint8_t st0[STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t st1[STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t st2[STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t st3[STAGE];
  const int lane = threadIdx.x & 63, j = lane >> 4, c = lane & 15;
  const int wn = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = (int)(p.K / kGroup);
  // Blocks go to the eight XCDs in turn; each XCD takes a contiguous run of tiles, which walk bands
  // of eight token tiles, so that the 64 tiles in work there (two blocks on each of 32 CUs) are about eight by eight
  // and share their operands in the XCD's L2.
  const int total = mtiles * ntiles, per = (total + 7) / 8;
  const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
  const int band = __builtin_amdgcn_readfirstlane(id / (8 * ntiles)), in = id - band * 8 * ntiles;
  const int bh = mtiles - 8 * band < 8 ? mtiles - 8 * band : 8;
  const int col = __builtin_amdgcn_readfirstlane(in / bh), tile0 = 16 * col;  // first channel tile
  const int64_t m0 = (int64_t)(8 * band + in - col * bh) * (16 * TM);
  const int tiles = (int)w4a8_tiles(p.N);
  const int nt = tiles - tile0 < 16 ? tiles - tile0 : 16;
  const int rows = p.M - m0 < 16 * TM ? (int)(p.M - m0) : 16 * TM;

  // rows and tiles past the end read as zero (the resources end there)
  const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(static_cast<const uint8_t*>(p.x) + m0 * p.ldx), (short)0, (int)((rows - 1) * p.ldx + p.K),
      0x00020000);
  const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint32_t*>(p.codes + (int64_t)tile0 * G * 256), (short)0, nt * G * 1024, 0x00020000);
  const __amdgpu_buffer_rsrc_t sr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint32_t*>(p.steps + (int64_t)tile0 * G * 16), (short)0, nt * G * 64, 0x00020000);
  uint32_t xoff[TM / 2];
#pragma unroll
  for (int i = 0; i < TM / 2; ++i) {
    const int row = 4 * TM * wn + 8 * i + (lane >> 3);
    xoff[i] = (uint32_t)(row * p.ldx + 16 * ((lane & 7) ^ row_swizzle(row)));
  }
  const uint32_t soff = (uint32_t)((4 * wn + j) * G * 64 + c * 4);  // the steps of this wave's own four tiles
  // A request past the last group repeats the last one (nothing uses it): scalar offsets stay below the
  // resources' ends, and rows past the last are out of range by their vector offset.
  auto dma = [&](uint8_t* st, int g) AWQ_INLINE {
    g = g < G ? g : G - 1;
#pragma unroll
    for (int i = 0; i < TM / 2; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (AWQ_LDS_A8 void*)(st + (4 * TM * wn + 8 * i) * 128), 16,
                                               (int)xoff[i], g * 128, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(sr, (AWQ_LDS_A8 void*)(st + SOFF + wn * 256), 4, (int)soff, g * 64, 0, 0);
  };
  u32x4 codes[AHEAD][4];  // the codes of the next steps, step g's in codes[g % AHEAD]
  auto load_codes = [&](u32x4* cw, int g) AWQ_INLINE {
    g = g < G ? g : G - 1;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int tl = 4 * wn + q < nt ? 4 * wn + q : nt - 1;  // past the last tile: loaded again, not stored
      cw[q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, lane * 16, (tl * G + g) * 1024, 0));
    }
  };
  // the zero points' operands of eight groups: row sums (past the last row: zero) and steps (past the last
  // group, whose sum is zero: the last one's)
  const __amdgpu_buffer_rsrc_t zr = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint32_t*>(sums + m0 * Gp), (short)0, (int)(rows * Gp * 4), 0x00020000);
  struct Zero {
    u32x2 sum[TM];
    uint32_t step[4][2];
  } z0, z1;
  auto load_zero = [&](Zero& z, int b) AWQ_INLINE {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int g = 8 * b + 2 * j + h;
        z.step[q][h] = __builtin_amdgcn_raw_buffer_load_b32(sr, ((4 * wn + q) * G + (g < G ? g : G - 1)) * 64 + c * 4, 0, 0);
      }
#pragma unroll
    for (int t = 0; t < TM; ++t)
      z.sum[t] = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_raw_buffer_load_b64(zr, (int)((16 * t + c) * Gp + 8 * b + 2 * j) * 4, 0, 0));
  };
  load_zero(z0, 0);
  load_zero(z1, 1);
  __builtin_amdgcn_sched_barrier(0);
  dma(st0, 0);
  dma(st1, 1);
  dma(st2, 2);
  f32x4 tot[TM][4];
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) tot[t][q] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  // minus the zero points' part: lane quarter j multiplies groups 8 b + 2 j and + 1, four products each.
  // The operands of eight groups are requested two rounds ahead, the first ones before the stages' copies.
  for (int b = 0; b < (int)Gp / 8; ++b) {
    f16x8 zq[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      u32x4 w;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t v = z0.step[q][h];
        const float dz = -h2f(v & 0xffffu) * h2f(v >> 16);
        const uint32_t hi = f2h(dz), lo = f2h(dz - h2f(hi));
        w[2 * h] = hi | hi << 16;
        w[2 * h + 1] = lo | lo << 16;
      }
      zq[q] = __builtin_bit_cast(f16x8, w);
    }
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      const f16x8 a = __builtin_bit_cast(f16x8, (u32x4){z0.sum[t][0], z0.sum[t][0], z0.sum[t][1], z0.sum[t][1]});
#pragma unroll
      for (int q = 0; q < 4; ++q) tot[t][q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, zq[q], tot[t][q], 0, 0, 0);
    }
    z0 = z1;
    load_zero(z1, b + 2);
  }
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) load_codes(codes[i], i);
  // this lane's pieces of row c of a token tile (tiles are 16 rows: the same swizzle in each)
  const int a0 = c * 128 + 16 * (j ^ row_swizzle(c));
  const int a1 = c * 128 + 16 * ((j + 4) ^ row_swizzle(c));
  i32x8 an;         // the next token tile's bytes
  uint32_t dn[4];   // the next step's steps and zero points
  auto read_a = [&](const uint8_t* st, int t) AWQ_INLINE {
    an = join(*reinterpret_cast<const u32x4*>(st + a0 + t * 2048), *reinterpret_cast<const u32x4*>(st + a1 + t * 2048));
  };
  auto read_d = [&](const uint8_t* st) AWQ_INLINE {
#pragma unroll
    for (int q = 0; q < 4; ++q) dn[q] = *reinterpret_cast<const uint32_t*>(st + SOFF + (4 * wn + q) * 64 + c * 4);
  };
  // own copies but the newest NDMA landed, own reads of the stage before done; after the barrier that
  // holds for every wave
  auto sync = [&] () AWQ_INLINE {
    __builtin_amdgcn_sched_barrier(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    constexpr int NEWER = NDMA + (AHEAD > 1 ? 4 : 0);
    static_assert(NEWER < 16, "the low four bits of vmcnt");
    __builtin_amdgcn_s_waitcnt(NEWER | (0x7 << 4) | (0xf << 8));  // vmcnt; no wait for LDS and exports
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
  };
  // Step g: stages now (g), next (g + 1) and free (g - 1, then g + 3).
  auto step = [&](int g, u32x4* cw, const uint8_t* now, const uint8_t* next, uint8_t* free) AWQ_INLINE {
    Operand<KIND> w[4];
    float d[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      w[q] = operand<KIND>(unpack_codes(cw[q]));
      d[q] = h2f(dn[q] & 0xffffu) * (E4M3 ? 1.0f / kE4m3Unit : 1.0f);
      asm volatile("" : "+v"(d[q]));  // fp32 from here on: v_fmac_f32 in place, not v_fma_mix_f32 from fp16
    }
    sync();
    load_codes(cw, g + AHEAD);
    __builtin_amdgcn_sched_barrier(0);
    dma(free, g + 3);
    __builtin_amdgcn_sched_barrier(0);
    // a token tile's multiply-adds run between the next tile's products, so that no product is waited for
    f32x4 s[4];
    auto add = [&](int t, int q) AWQ_INLINE {
#pragma unroll
      for (int i = 0; i < 4; ++i) tot[t][q][i] = fmaf(d[q], settled<KIND>(s[q][i]), tot[t][q][i]);
    };
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      const Operand<KIND> a = operand<KIND>(an);
      f32x4 r[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        r[q] = product_begin<KIND>(a, w[q]);
        if (q == 0) {
          if (t + 1 < TM) {
            read_a(now, t + 1);
          } else {
            read_a(next, 0);
            read_d(next);
          }
        }
        if (t > 0 && (KIND == kE4m3Fast || q < 2)) add(t - 1, q);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (KIND != kE4m3Fast) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          r[q] = product_end<KIND>(a, w[q], r[q]);
          if (t > 0 && q < 2) add(t - 1, 2 + q);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) s[q] = r[q];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) add(TM - 1, q);
  };
  __builtin_amdgcn_sched_barrier(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  constexpr int NEWER0 = 2 * NDMA + 4 * AHEAD;
  __builtin_amdgcn_s_waitcnt((NEWER0 & 15) | ((NEWER0 >> 4) << 14) | (0x7 << 4) | (0xf << 8));  // stage 0
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_sched_barrier(0);
  read_a(st0, 0);
  read_d(st0);
  int g = 0;
  for (; g + 4 <= G; g += 4) {
    step(g, codes[0], st0, st1, st3);
    step(g + 1, codes[1 % AHEAD], st1, st2, st0);
    step(g + 2, codes[2 % AHEAD], st2, st3, st1);
    step(g + 3, codes[3 % AHEAD], st3, st0, st2);
  }
  if (g < G) step(g, codes[0], st0, st1, st3);
  if (g + 1 < G) step(g + 1, codes[1 % AHEAD], st1, st2, st0);
  if (g + 2 < G) step(g + 2, codes[2 % AHEAD], st2, st3, st1);
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt and lgkmcnt 0: no copy or load outlives the block
  // stores through a resource that ends with the last row's last channel: rows past M are dropped there,
  // channels past N by the lane mask (128 rows of Y span less than 2^31 bytes: host-checked)
  const int n0 = tile0 * 16;
  const int es = p.ybf16 ? 2 : 4;
  const __amdgpu_buffer_rsrc_t yr = __builtin_amdgcn_make_buffer_rsrc(
      static_cast<char*>(p.y) + (m0 * p.ldy + n0) * es, (short)0, (int)(((rows - 1) * p.ldy + p.N - n0) * es),
      0x00020000);
  const __amdgpu_buffer_rsrc_t mr =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(p.xscale + m0), (short)0, rows * 4, 0x00020000);
  const int ldyb = (int)p.ldy * es;
  float pw[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int n = n0 + (4 * wn + q) * 16 + c;
    pw[q] = p.powers[n < tiles * 16 ? n : tiles * 16 - 1];
  }
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float xs = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(mr, (16 * t + 4 * j + i) * 4, 0, 0));  // 0 past M
#pragma unroll
      for (int q = 0; q < 4; ++q) tot[t][q][i] = tot[t][q][i] * pw[q] * xs;
    }
  if (p.ybf16) {
    // through LDS, so that a wave stores whole rows of 256 channels (written from the products' layout,
    // a store would fill 32 bytes of a line); rows of 528 bytes keep the writes free of bank conflicts
    constexpr int ROW = 528, RPS = 4 * TM;  // bytes of a row, rows per stage buffer
    static_assert(RPS * ROW <= STAGE, "a stage buffer holds a quarter of the tile");
    uint8_t* const pool[4] = {st0, st1, st2, st3};
    __syncthreads();  // every wave is done with the stages
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint16_t*>(pool[16 * t / RPS] + (16 * t % RPS + 4 * j + i) * ROW + (64 * wn + 16 * q + c) * 2) =
              to_bf16(tot[t][q][i]);
    __syncthreads();
    // 32 lanes a row; 16-byte stores where every row of Y starts at a multiple of 16 bytes
    const int cb = (lane & 31) * 8;
    const bool wide = ((reinterpret_cast<uintptr_t>(p.y) | (uintptr_t)ldyb) & 15u) == 0 && n0 + cb + 8 <= p.N;
#pragma unroll
    for (int r = 0; r < 2 * TM; ++r) {
      const int row = 2 * wn + (lane >> 5);  // of eight
      const u32x4 v = *reinterpret_cast<const u32x4*>(pool[8 * r / RPS] + (8 * r % RPS + row) * ROW + cb * 2);
      const int yo = (8 * r + row) * ldyb + cb * 2;
      if (wide) {
        __builtin_amdgcn_raw_buffer_store_b128(v, yr, yo, 0, 0);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n0 + cb + e < p.N)
            __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(v[e / 2] >> (16 * (e & 1))), yr, yo + 2 * e, 0, 0);
      }
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int nc = (4 * wn + q) * 16 + c;
      if (n0 + nc < p.N) {
        const int yo = 4 * j * ldyb + nc * 4;
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(tot[t][q][i]), yr, yo + (16 * t + i) * ldyb, 0, 0);
      }
    }
  }
}

// ---- some tokens: tiles that share their groups among blocks ----------------------------------------------
// Where 16 TM x 256 tiles are fewer than CUs, each tile's groups are divided among blocks: block
// (column, split, row) sums groups split n .. split n + n - 1 into fp32 parts that a second kernel adds in
// split order (one split: straight into Y).  A block has few groups, so what it takes is latency, the
// memory's and that of a product behind whose result its multiply-adds wait: two sets of four waves take
// the even and the odd groups of the block (their sums meet in LDS at the end), each from its own ring of
// three stages that LDS DMA fills with a group's tokens, codes and steps, two stages ahead.
// The zero points come off per group, with the rows' sums from one more product with ones.
template <int TM>
constexpr int kSplitStage = 16 * TM * 128 + 16 * 1024 + 1024;

template <int KIND, int TM>
__global__ __launch_bounds__(512, 2) void w4a8_split_kernel(const W4a8Args p, float* __restrict__ parts, int mtiles,
                                                            int ntiles, int splits, int per_split) {
  constexpr bool E4M3 = KIND != kInt8;
  constexpr int STAGE = kSplitStage<TM>, BOFF = 16 * TM * 128, SOFF = BOFF + 16 * 1024;
  constexpr int NDMA = TM / 2 + 4 + 1;  // copies per wave and stage
  __shared__ __attribute__((aligned(1024))) uint8_t st0[2 * STAGE], st1[2 * STAGE], st2[2 * STAGE];
  const int lane = threadIdx.x & 63, j = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wn = wave & 3, set = wave >> 2;
  const int G = (int)(p.K / kGroup);
  // each XCD (blocks go to the eight in turn) takes a contiguous run: the rows of one column and split, which
  // share their codes, then the next split, then the next column
  const int total = mtiles * ntiles * splits, per = (total + 7) / 8;
  const int id = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || id >= total) return;
  const int cs = __builtin_amdgcn_readfirstlane(id / mtiles);
  const int col = __builtin_amdgcn_readfirstlane(cs / splits), split = cs - col * splits;
  const int tile0 = 16 * col;
  const int64_t m0 = (int64_t)(id - cs * mtiles) * (16 * TM);
  const int tiles = (int)w4a8_tiles(p.N);
  const int nt = tiles - tile0 < 16 ? tiles - tile0 : 16;
  const int rows = p.M - m0 < 16 * TM ? (int)(p.M - m0) : 16 * TM;
  const int g0 = split * per_split, n = G - g0 < per_split ? G - g0 : per_split;  // this block's groups, at least one

  const int base = set * STAGE;  // this set's half of a stage buffer
  uint32_t xoff[TM / 2], woff[4];
#pragma unroll
  for (int i = 0; i < TM / 2; ++i) {
    const int row = 4 * TM * wn + 8 * i + (lane >> 3);
    xoff[i] = (uint32_t)(row * p.ldx + 16 * ((lane & 7) ^ row_swizzle(row)));
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) woff[q] = (uint32_t)((4 * wn + q) * G * 1024 + lane * 16);
  const uint32_t soff = (uint32_t)((4 * wn + j) * G * 64 + c * 4);
  // Rows and tiles past the end read as zero (the resources end there); past the block's last group the
  // resources are empty, so that every step has the same number of copies and none reads for nothing.
  auto dma = [&](uint8_t* st, int i) AWQ_INLINE {
    const bool in = 2 * i + set < n;
    const int g = in ? g0 + 2 * i + set : 0;
    const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(static_cast<const uint8_t*>(p.x) + m0 * p.ldx), (short)0,
        in ? (int)((rows - 1) * p.ldx + p.K) : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint32_t*>(p.codes + (int64_t)tile0 * G * 256), (short)0, in ? nt * G * 1024 : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t sr = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint32_t*>(p.steps + (int64_t)tile0 * G * 16), (short)0, in ? nt * G * 64 : 0, 0x00020000);
#pragma unroll
    for (int k = 0; k < TM / 2; ++k)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (AWQ_LDS_A8 void*)(st + (base + (4 * TM * wn + 8 * k) * 128)), 16,
                                               (int)xoff[k], g * 128, 0, 0);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, (AWQ_LDS_A8 void*)(st + (base + BOFF + (4 * wn + q) * 1024)), 16,
                                               (int)woff[q], g * 1024, 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(sr, (AWQ_LDS_A8 void*)(st + (base + SOFF + wn * 256)), 4, (int)soff, g * 64, 0, 0);
  };
  dma(st0, 0);
  dma(st1, 1);
  f32x4 tot[TM][4];
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) tot[t][q] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int kOne = E4M3 ? 0x38383838 : 0x01010101;
  const Operand<KIND> ones = operand<KIND>((i32x8){kOne, kOne, kOne, kOne, kOne, kOne, kOne, kOne});
  const int a0 = base + c * 128 + 16 * (j ^ row_swizzle(c));
  const int a1 = base + c * 128 + 16 * ((j + 4) ^ row_swizzle(c));
  i32x8 an;                // the next token tile's bytes
  u32x4 cw[4];             // the next step's codes
  uint32_t dn[4];          // and its steps and zero points
  auto read_a = [&](const uint8_t* st, int t) AWQ_INLINE {
    an = join(*reinterpret_cast<const u32x4*>(st + (a0 + t * 2048)), *reinterpret_cast<const u32x4*>(st + (a1 + t * 2048)));
  };
  auto read_w = [&](const uint8_t* st) AWQ_INLINE {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      cw[q] = *reinterpret_cast<const u32x4*>(st + (base + BOFF + (4 * wn + q) * 1024 + lane * 16));
      dn[q] = *reinterpret_cast<const uint32_t*>(st + (base + SOFF + (4 * wn + q) * 64 + c * 4));
    }
  };
  auto sync = [&](auto newer) AWQ_INLINE {  // own copies but the newest landed, own reads done; then everybody's
    constexpr int NEWER = decltype(newer)::value;
    static_assert(NEWER < 16, "the low four bits of vmcnt");
    __builtin_amdgcn_sched_barrier(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(NEWER | (0x7 << 4));
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
  };
  // Step i: stages now (i), next (i + 1) and free (i - 1, then i + 2).  The barrier is in the middle: it
  // says that stage i + 1 has landed, whose first operands the second half reads, and that nobody reads
  // stage i - 1 any more.
  auto step = [&](const uint8_t* now, const uint8_t* next, uint8_t* free, int i) AWQ_INLINE {
    Operand<KIND> w[4];
    float d[4], z[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      w[q] = operand<KIND>(unpack_codes(cw[q]));
      d[q] = h2f(dn[q] & 0xffffu);
      z[q] = d[q] * h2f(dn[q] >> 16);  // step times zero point
      if (E4M3) d[q] *= 1.0f / kE4m3Unit;
      asm volatile("" : "+v"(d[q]), "+v"(z[q]));  // fp32 from here on: v_fmac_f32 in place
    }
    // a token tile's multiply-adds run behind the next tile's products
    f32x4 sx, r[4];
    auto add = [&](int t) AWQ_INLINE {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = settled<KIND>(sx[e]);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          tot[t][q][e] = fmaf(d[q], settled<KIND>(r[q][e]), fmaf(-z[q], x, tot[t][q][e]));
      }
    };
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      const Operand<KIND> a = operand<KIND>(an);
      if (t == TM / 2) {
        sync(std::integral_constant<int, 0>{});
        dma(free, i + 2);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (t + 1 < TM) {
        read_a(now, t + 1);
      } else {
        read_a(next, 0);
        read_w(next);
      }
      const f32x4 nx = group_product<KIND>(a, ones);
      f32x4 nr[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) nr[q] = group_product<KIND>(a, w[q]);
      if (t > 0) add(t - 1);
      sx = nx;
#pragma unroll
      for (int q = 0; q < 4; ++q) r[q] = nr[q];
      __builtin_amdgcn_sched_barrier(0);
    }
    add(TM - 1);
    __builtin_amdgcn_sched_barrier(0);
  };
  sync(std::integral_constant<int, NDMA>{});
  read_a(st0, 0);
  read_w(st0);
  const int pairs = (n + 1) / 2;
  int i = 0;
  for (; i + 3 <= pairs; i += 3) {
    step(st0, st1, st2, i);
    step(st1, st2, st0, i + 1);
    step(st2, st0, st1, i + 2);
  }
  if (i < pairs) step(st0, st1, st2, i);
  if (i + 1 < pairs) step(st1, st2, st0, i + 1);
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt and lgkmcnt 0: no copy outlives the block
  // each set gives the other the sums of half the token tiles through LDS (a tile's four values a lane, lane by
  // lane) and finishes the other half
  __syncthreads();
  static_assert(TM * 8192 <= 2 * STAGE, "a stage buffer holds half the sums of one set");
  auto slot = [&](uint8_t* st, int t, int q) AWQ_INLINE {
    return reinterpret_cast<f32x4*>(st + ((t * 4 + wn) * 4 + q) * 1024 + lane * 16);
  };
  constexpr int H = TM / 2;
  if (set == 0) {
#pragma unroll
    for (int t = 0; t < H; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) *slot(st0, t, q) = tot[H + t][q];
  } else {
#pragma unroll
    for (int t = 0; t < H; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) *slot(st1, t, q) = tot[t][q];
  }
  __syncthreads();
  // (the even groups' sums first in both halves)
  f32x4 fin[H][4];
#pragma unroll
  for (int t = 0; t < H; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) fin[t][q] = set == 0 ? tot[t][q] + *slot(st1, t, q) : *slot(st0, t, q) + tot[H + t][q];
  const int r0 = 16 * H * set + 4 * j;  // this lane's first row
  const int64_t np = (int64_t)tiles * 16;
  const bool part = splits > 1;
  const int es = !part && p.ybf16 ? 2 : 4;
  const int64_t ld = part ? np : p.ldy;
  char* out = part ? reinterpret_cast<char*>(parts + ((int64_t)split * p.M + m0) * np) : static_cast<char*>(p.y) + m0 * p.ldy * es;
  const int64_t cols = part ? np : p.N;
  // the resource ends with the last row's last channel: rows past M are dropped there
  const __amdgpu_buffer_rsrc_t yr = __builtin_amdgcn_make_buffer_rsrc(
      out + (int64_t)tile0 * 16 * es, (short)0, (int)(((rows - 1) * ld + cols - tile0 * 16) * es), 0x00020000);
  float xs[H][4];
  const __amdgpu_buffer_rsrc_t mr =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(p.xscale + m0), (short)0, rows * 4, 0x00020000);
#pragma unroll
  for (int t = 0; t < H; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      xs[t][e] = part ? 1.0f : __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(mr, (r0 + 16 * t + e) * 4, 0, 0));
  const int ldb = (int)ld * es;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int nc = (4 * wn + q) * 16 + c;
    if (tile0 * 16 + nc < cols) {
      const float pw = part ? 1.0f : p.powers[tile0 * 16 + nc];
#pragma unroll
      for (int t = 0; t < H; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y = fin[t][q][e] * pw * xs[t][e];
          const int yo = (r0 + 16 * t + e) * ldb + nc * es;
          if (es == 2) __builtin_amdgcn_raw_buffer_store_b16(to_bf16(y), yr, yo, 0, 0);
          else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y), yr, yo, 0, 0);
        }
    }
  }
}

// Y = xscale 2^e (the parts in split order); four channels per thread.
__global__ __launch_bounds__(256) void w4a8_join_kernel(const W4a8Args p, const float* __restrict__ parts, int splits) {
  const int64_t np = w4a8_tiles(p.N) * 16, quads = np / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.M * quads) return;
  const int64_t m = i / quads, n = 4 * (i - m * quads);
  const float* src = parts + m * np + n;
  f32x4 s = *reinterpret_cast<const f32x4*>(src);
  for (int k = 1; k < splits; ++k) s += *reinterpret_cast<const f32x4*>(src + (int64_t)k * p.M * np);
  const float xs = p.xscale[m];
  const f32x4 pw = *reinterpret_cast<const f32x4*>(p.powers + n);
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < p.N) {
      const float y = s[e] * pw[e] * xs;
      if (p.ybf16) static_cast<uint16_t*>(p.y)[m * p.ldy + n + e] = to_bf16(y);
      else static_cast<float*>(p.y)[m * p.ldy + n + e] = y;
    }
}

template <int KIND, int TM>
hipError_t launch_split(const W4a8Args& a, const Plan& pl, float* parts, hipStream_t st) {
  const int64_t mt = (a.M + 16 * TM - 1) / (16 * TM), nt = (a.N + kTileN - 1) / kTileN, blocks = mt * nt * pl.splits;
  w4a8_split_kernel<KIND, TM><<<(unsigned)((blocks + 7) / 8 * 8), 512, 0, st>>>(a, parts, (int)mt, (int)nt, pl.splits,
                                                                              pl.per_split);
  if (pl.splits > 1) {
    const int64_t quads = a.M * w4a8_tiles(a.N) * 4;
    w4a8_join_kernel<<<(unsigned)((quads + 255) / 256), 256, 0, st>>>(a, parts, pl.splits);
  }
  return hipGetLastError();
}

template <int KIND, int TM>
hipError_t launch_tile(const W4a8Args& a, uint32_t* sums, hipStream_t st) {
  const int64_t G = a.K / kGroup, Gp = padded_groups(a.K), pieces = a.M * Gp * 8;
  const int64_t mt = (a.M + 16 * TM - 1) / (16 * TM), nt = (a.N + kTileN - 1) / kTileN;
  w4a8_sums_kernel<KIND != kInt8><<<blocks_of((pieces + 255) / 256, 256), 256, 0, st>>>(
      static_cast<const uint8_t*>(a.x), a.M, a.ldx, G, Gp, sums);
  w4a8_tile_kernel<KIND, TM><<<(unsigned)((mt * nt + 7) / 8 * 8), 256, 0, st>>>(a, sums, Gp, (int)mt, (int)nt);
  return hipGetLastError();
}

template <int KIND>
hipError_t launch_kind(const W4a8Args& a, const Plan& pl, void* ws, hipStream_t st) {
  if (pl.path == kStream) return launch_stream<KIND>(a, pl, st);
  if (pl.path == kSplit) {
    float* parts = static_cast<float*>(ws);
    return pl.tm == 2 ? launch_split<KIND, 2>(a, pl, parts, st) : launch_split<KIND, 4>(a, pl, parts, st);
  }
  uint32_t* sums = static_cast<uint32_t*>(ws);
  if constexpr (KIND != kE4m3Wide) {  // the converted operands leave no registers for eight token tiles
    if (pl.tm == 8) return launch_tile<KIND, 8>(a, sums, st);
  }
  return launch_tile<KIND, 4>(a, sums, st);
}

}  // namespace

hipError_t launch_w4a8_weight(const int32_t* qweight, const uint16_t* scales, const uint16_t* zeros, int64_t N,
                              int64_t K, uint32_t* codes, uint32_t* steps, float* powers, hipStream_t st) {
  const int64_t rows = w4a8_tiles(N) * 16, words = rows * (K / 8);
  w4a8_codes_kernel<<<blocks_of((words + 255) / 256, 256), 256, 0, st>>>(reinterpret_cast<const uint32_t*>(qweight), N, K,
                                                                     words, codes);
  w4a8_steps_kernel<<<(unsigned)w4a8_tiles(N), 256, 0, st>>>(scales, zeros, N, K / kGroup, steps, powers);
  return hipGetLastError();
}

size_t w4a8_workspace(int64_t M, int64_t K, int64_t N) {
  const Plan pl = w4a8_plan(M, K, N);
  if (pl.path == kTile) return (size_t)(M * padded_groups(K) * 4);
  return pl.splits > 1 ? (size_t)(pl.splits * M * w4a8_tiles(N) * 16 * 4) : 0;
}

hipError_t launch_w4a8(const W4a8Args& a, void* ws, hipStream_t st) {
  const Plan pl = w4a8_plan(a.M, a.K, a.N);
  if (!a.e4m3) return launch_kind<kInt8>(a, pl, ws, st);
  return matrix_sums(a.sums, a.ybf16, a.M) ? launch_kind<kE4m3Fast>(a, pl, ws, st)
                                           : launch_kind<kE4m3Wide>(a, pl, ws, st);
}

}  // namespace awq
