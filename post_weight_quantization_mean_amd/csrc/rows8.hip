// The producers of a quantized layer's input: RMS norm with the residual's addition, and the gated
// activation, each written in fp32, bf16, or 8 bits with a scale per row.
//
//   norm  h = x + r;  y_k = h_k gamma_k / sqrt(mean h^2 + eps)
//   act   y_k = act(g_k) u_k / s_k
//   8-bit scale = max(max_k |y_k|, 2^-100) / Q,  code_k = rne(y_k / scale)
//
// 1 / rms is one number per row, so max |y| = max |h gamma| / rms: the sum of squares and the
// maximum come out of the same pass over the row, and the code is rne(h gamma * Q / max |h gamma|).
// The row stays in registers between that pass and the store, so every operand crosses memory once;
// the kernels are bound by those bytes.
//
// Maxima are taken over the bits of |v| as unsigned integers: the same order as the floats', with NaN
// above infinity, so that a NaN reaches the row's scale (fmaxf would drop it).
#include <type_traits>

#include "a8_internal.h"
#include "rows8_plan.h"

namespace awq {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

constexpr int kOpNorm = 0, kOpAct = 1;
constexpr float kFloorMax = 0x1p-100f;  // least row maximum a scale is made from
constexpr float kLog2e = 1.44269504088896341f, kLog2eLo = 1.92596299112661746887e-8f;
constexpr float kLn2 = 0.69314718055994531f;

template <int T>
constexpr int64_t esize() { return T == kF32 ? 4 : T == kBf16 ? 2 : 1; }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // round to nearest even
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

// The same types for rows that start anywhere: the hardware takes such accesses, at a few extra cycles where
// one crosses a cache line.
typedef unsigned u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef unsigned u32x4_any __attribute__((ext_vector_type(4), aligned(1)));

// eight consecutive elements as loaded, and as fp32
template <int T>
struct Raw8 {
  u32x4 q[T == kF32 ? 2 : 1];
};
// ALIGNED: the elements start at a multiple of 16 bytes, otherwise anywhere.
template <int T, bool ALIGNED>
__device__ __forceinline__ Raw8<T> load8(const void* p, int64_t i) {
  using V = typename std::conditional<ALIGNED, u32x4, u32x4_any>::type;
  Raw8<T> r;
  const V* s = reinterpret_cast<const V*>(static_cast<const char*>(p) + i * esize<T>());
  r.q[0] = s[0];
  if constexpr (T == kF32) r.q[1] = s[1];
  return r;
}
template <int T>
__device__ __forceinline__ float elem8(const Raw8<T>& r, int t) {  // t known at compile time
  if constexpr (T == kF32) return __uint_as_float(r.q[t / 4][t % 4]);
  const uint32_t w = r.q[0][t / 2];
  return __uint_as_float(t & 1 ? w & 0xffff0000u : w << 16);
}
template <bool ALIGNED>
__device__ __forceinline__ void store8_f32(void* p, int64_t i, const float* v) {
  using V = typename std::conditional<ALIGNED, u32x4, u32x4_any>::type;
  V* d = reinterpret_cast<V*>(static_cast<float*>(p) + i);
#pragma unroll
  for (int h = 0; h < 2; ++h)
    d[h] = (u32x4){__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]), __float_as_uint(v[4 * h + 2]),
                   __float_as_uint(v[4 * h + 3])};
}
template <bool ALIGNED>
__device__ __forceinline__ void store8_bf16(void* p, int64_t i, const float* v) {
  using V = typename std::conditional<ALIGNED, u32x4, u32x4_any>::type;
  *reinterpret_cast<V*>(static_cast<uint16_t*>(p) + i) =
      (u32x4){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}
template <bool ALIGNED>
__device__ __forceinline__ void store8_codes(void* p, int64_t i, const u32x2 w) {
  using V = typename std::conditional<ALIGNED, u32x2, u32x2_any>::type;
  *reinterpret_cast<V*>(static_cast<uint8_t*>(p) + i) = w;
}
template <int XT>
__device__ __forceinline__ float elem1(const void* p, int64_t i) {
  if constexpr (XT == kF32) return static_cast<const float*>(p)[i];
  else return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}
__device__ __forceinline__ void store1(void* p, int64_t i, float v, int type) {
  if (type == kF32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = (uint16_t)pack_bf16(v, v);
}

// four codes rne(v c) in one word.  int8: v c + 1.5 2^23 leaves the rounded integer, two's complement,
// in the low byte (one fused multiply-add, one rounding); |v c| <= Q (1 + 2^-21), so nothing clips.
// e4m3: the conversion rounds to nearest even, and a value up to 464 goes to 448.
__device__ __forceinline__ uint32_t codes4(const float* v, float c, bool e4m3) {
  if (e4m3) {
    uint32_t w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * c, v[1] * c, 0, false);
    return __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * c, v[3] * c, w, true);
  }
  uint32_t b[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) b[t] = __float_as_uint(fmaf(v[t], c, 12582912.0f));
  const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
  return lo | hi;
}

// SiLU below kSiluFar, where 1 + exp(-x) is exp(-x) to fp32 and its reciprocal leaves the normal numbers (x < -87.3)
// before x exp(x) does (-91.8): x times 2^64 exp(x), times 2^-64.
constexpr float kSiluFar = -79.0f;
__device__ __forceinline__ float silu_far(float x, bool fine) {
  const float t = x * kLog2e;
  float e = __builtin_amdgcn_exp2f(t + 64.0f);  // (the sum is exact where the result is not 0)
  if (fine && t > -256.0f) {
    const float lo = fmaf(x, kLog2e, -t) + x * kLog2eLo;
    e = fmaf(e, lo * kLn2, e);
  }
  return x * e * 0x1p-64f;
}

// act(x), for SiLU above kSiluFar.  SiLU by the hardware exponential and reciprocal (1 ulp each); for an fp32 result
// (fine) the exponent's rounding, |x| 2^-24 relative in exp(-x), is put back by its first-order term.
__device__ __forceinline__ float activate_near(float x, int act, bool fine) {
  if (act == kActSilu) {
    const float t = -x * kLog2e;
    float e = __builtin_amdgcn_exp2f(t);
    if (fine && fabsf(t) < 126.0f) {
      const float lo = fmaf(-x, kLog2e, -t) - x * kLog2eLo;
      e = fmaf(e, lo * kLn2, e);
    }
    return x * __builtin_amdgcn_rcpf(1.0f + e);
  }
  if (act == kActGelu) {
    // erfc(z) = exp(-z^2) p(1 / (1 + 0.43 z)) for z = |x| / sqrt 2: p of degree 8 fitted to exp(z^2) erfc(z) with
    // relative error 2^-23.4 up to z = 10.5 (above it the product underflows), halved here
    const float a = fabsf(x), t = __builtin_amdgcn_rcpf(fmaf(a, 0.30405592918395996f, 1.0f));
    float p = 0.03716862201690674f;
    p = fmaf(p, t, -0.15669101476669312f);
    p = fmaf(p, t, 0.19490274786949158f);
    p = fmaf(p, t, -0.0462779626250267f);
    p = fmaf(p, t, 0.12572525441646576f);
    p = fmaf(p, t, 0.10152062773704529f);
    p = fmaf(p, t, 0.12242478877305984f);
    p = fmaf(p, t, 0.12122516334056854f);
    p = fmaf(p, t, 1.818873215597705e-06f);
    const float e = p * __builtin_amdgcn_exp2f(a * a * (-0.5f * kLog2e));  // erfc(z) / 2
    // e is 0 long before 64: +Inf, cut to it beside e (as integers: one instruction), stays itself; -Inf times 0 is
    // NaN, as in the definition
    const int xi = __float_as_int(x), cut = __float_as_int(64.0f);
    return x < 0.0f ? x * e : fmaf(-__int_as_float(xi < cut ? xi : cut), e, x);
  }
  return x;
}

__device__ __forceinline__ float activate(float x, int act, bool fine) {
  return act == kActSilu && x < kSiluFar ? silu_far(x, fine) : activate_near(x, act, fine);
}
// Whether a lane of this wave holds an element below kSiluFar (or a negative NaN) in a unit: the elements' bits as
// unsigned integers are largest for the most negative ones.  Half an instruction an element, before the unit's
// activations, which then take one path for the whole wave (silu gate, 4096 x 14336 bf16 -> e4m3: 50.5 us).
template <int T>
__device__ __forceinline__ bool any_far(const Raw8<T>& x) {
  constexpr uint32_t kFar = 0xc29e0000u;  // the bits of kSiluFar, and their high half those of its bf16
  if constexpr (T == kF32) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t w = x.q[e / 4][e % 4];
      top = w > top ? w : top;
    }
    return __builtin_amdgcn_ballot_w64(top > kFar) != 0;
  } else {
    u16x2 top = {0, 0};
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      const uint32_t w = x.q[0][d];  // (a bit cast of the vector's element itself reads element 0)
      top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w));
    }
    return __builtin_amdgcn_ballot_w64(top[0] > (kFar >> 16) || top[1] > (kFar >> 16)) != 0;
  }
}

// The elements are unpacked behind this point, not once ahead of all the cases that read them: that would hold every
// operand of a row in fp32 at once (silu gate, 4096 x 14336: 71 registers, 65 us; 46 and 50.5 with it).
template <int T>
__device__ __forceinline__ void here(Raw8<T>& r) {
  asm volatile("" : "+v"(r.q[0]));
  if constexpr (T == kF32) asm volatile("" : "+v"(r.q[1]));
}

// ---- reductions -------------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t wave_umax(uint32_t x) {
  x = umax(x, dpp_u<kDppXor1>(x));
  x = umax(x, dpp_u<kDppXor2>(x));
  x = umax(x, dpp_u<kDppHalfMirror>(x));
  x = umax(x, dpp_u<kDppMirror>(x));
  const uint32_t a = __builtin_amdgcn_readlane(x, 0), b = __builtin_amdgcn_readlane(x, 16);
  const uint32_t c = __builtin_amdgcn_readlane(x, 32), d = __builtin_amdgcn_readlane(x, 48);
  return umax(umax(a, b), umax(c, d));
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// (sum, max) over the W waves of a row, the same in every thread: a wave's own by lane exchange, the
// waves' through LDS in wave order.  red: [2][W] pairs; the halves alternate by row, so one barrier a
// row is enough (a wave writes a half again only after the barrier of the row between).
template <int W>
__device__ __forceinline__ void row_reduce(float& sum, uint32_t& top, float2 (*red)[W], int parity, int wave,
                                           int lane) {
  sum = wave_sum(sum);
  top = wave_umax(top);
  if constexpr (W > 1) {
    if (lane == 0) red[parity][wave] = make_float2(sum, __uint_as_float(top));
    __syncthreads();
    float s = 0.0f;
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 v = red[parity][w];
      s += v.x;
      m = umax(m, __float_as_uint(v.y));
    }
    sum = s;
    top = m;
  }
}

// What the row's numbers give: the factor of the stored values (1 / rms, or 1), and for codes the
// factor that takes v to its code, and the scale.  A row that is not finite gets NaN in all of them.
// Where a small eps takes the codes' factor past fp32's range (max |v| below 2^-119, a row of zeros among
// them), a power of two of it, pre, is multiplied to v first; otherwise pre is 1.
struct RowFactors {
  float mul, code, scale, pre;
};
template <int OP>
__device__ __forceinline__ RowFactors row_factors(const RowArgs& a, float sum, uint32_t top) {
  RowFactors f;
  f.mul = 1.0f;
  const float inf = __builtin_inff(), nan = __builtin_nanf("");
  if (OP == kOpNorm) f.mul = sum < inf ? 1.0f / sqrtf(sum / (float)a.K + a.eps) : nan;
  const float q = a.y_type == kI8 ? 127.0f : 448.0f;
  const float m = __uint_as_float(top) * f.mul;  // max |y|; NaN stays
  const float mf = m < inf ? fmaxf(m, kFloorMax) : nan;
  f.scale = mf / q;
  f.code = q / mf;
  f.pre = 1.0f;
  if (OP == kOpNorm) {
    // Q / max |v|: 1 / rms cancels, and with it its roundings (but where the floor is above max |y|)
    const float t = __uint_as_float(top);
    if (m < kFloorMax) f.code = f.mul * (q / kFloorMax);
    else if (m < inf) f.code = q / t;
    if (f.code == inf) {
      f.pre = 0x1p64f;
      f.code = m < kFloorMax ? f.mul * 0x1p-64f * (q / kFloorMax) : q / (t * 0x1p64f);
    }
  }
  return f;
}

// ---- a row in registers -------------------------------------------------------------------------
// W waves per row (W = 1: four rows per block), U units of eight elements per lane.  ALIGNED: every row of
// every operand starts at a multiple of 16 bytes (8-bit outputs: 8) and K is a multiple of 8; otherwise the
// first K % 8 threads of a row take one of its last elements each.
template <int OP, int XT, int BT, int W, int U, bool ALIGNED>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void rows_kernel(const RowArgs a) {
  constexpr int T = 64 * W, RPB = W == 1 ? 4 : 1;
  __shared__ float2 red[2][W];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = W == 1 ? lane : threadIdx.x;
  const int units = (int)(a.K / 8);
  const bool tail = !ALIGNED && t < (int)(a.K % 8);
  const int kt = 8 * units + t;
  const int ytype = a.y_type, col_type = a.col_type;
  int parity = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + (W == 1 ? wave : 0); row < a.M; row += (int64_t)gridDim.x * RPB) {
    // units past the row's end load its first one again and count for nothing
    int k[U];
    Raw8<XT> x[U];
    Raw8<BT == kNoOperand ? kBf16 : BT> b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int unit = u * T + t;
      k[u] = unit < units ? 8 * unit : 0;
      if (!ALIGNED && units == 0) continue;
      x[u] = load8<XT, ALIGNED>(a.x, row * a.ldx + k[u]);
    }
    if constexpr (BT != kNoOperand) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (ALIGNED || units > 0) b[u] = load8<BT, ALIGNED>(a.b, row * a.ldb + k[u]);
    }
    float vt = 0.0f, ht = 0.0f;  // the tail element's value, and its h
    if (tail) {
      ht = elem1<XT>(a.x, row * a.ldx + kt);
      const float bt = BT != kNoOperand ? elem1<BT == kNoOperand ? kBf16 : BT>(a.b, row * a.ldb + kt) : 0.0f;
      const float ct = col_type == kF32 ? elem1<kF32>(a.col, kt) : col_type == kBf16 ? elem1<kBf16>(a.col, kt) : 1.0f;
      if (OP == kOpNorm) {
        if (BT != kNoOperand) ht += bt;
        vt = ht * ct;
        if (BT != kNoOperand && a.h != nullptr) store1(a.h, row * a.ldh + kt, ht, BT);
      } else {
        vt = activate(ht, a.act, ytype == kF32);
        if (BT != kNoOperand) vt *= bt;
        if (col_type == kF32) vt *= __builtin_amdgcn_rcpf(ct);
      }
    }
    float v[U][8], sum = ht * ht;
    uint32_t top = abs_bits(vt);
    if constexpr (OP == kOpNorm) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float sq = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[u][e] = elem8(x[u], e);
          if constexpr (BT != kNoOperand) v[u][e] += elem8(b[u], e);
          sq = fmaf(v[u][e], v[u][e], sq);
        }
        const bool in = u * T + t < units;
        sum += in ? sq : 0.0f;
        if constexpr (BT != kNoOperand) {
          if (in && a.h != nullptr) {
            if constexpr (BT == kF32) store8_f32<ALIGNED>(a.h, row * a.ldh + k[u], v[u]);
            else store8_bf16<ALIGNED>(a.h, row * a.ldh + k[u], v[u]);
          }
        }
      }
      if (!ALIGNED && units == 0) {
      } else if (col_type == kF32) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const Raw8<kF32> g = load8<kF32, ALIGNED>(a.col, k[u]);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[u][e] *= elem8(g, e);
        }
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const Raw8<kBf16> g = load8<kBf16, ALIGNED>(a.col, k[u]);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[u][e] *= elem8(g, e);
        }
      }
    } else {
      // the choice stands outside the eight elements' loop: one straight piece of code a case (GELU gate, 4096 x 11008:
      // 41 us; with the choice inside 49)
      const bool fine = ytype == kF32;
      if (ALIGNED || units > 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          auto each = [&](auto f) __attribute__((always_inline)) {
            here(x[u]);
            if constexpr (BT != kNoOperand) here(b[u]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              v[u][e] = f(elem8(x[u], e));
              if constexpr (BT != kNoOperand) v[u][e] *= elem8(b[u], e);
            }
          };
          if (a.act == kActSilu) {
            if (any_far<XT>(x[u])) each([&](float w) { return activate(w, kActSilu, fine); });
            else if (fine) each([](float w) { return activate_near(w, kActSilu, true); });
            else each([](float w) { return activate_near(w, kActSilu, false); });
          } else if (a.act == kActGelu) {
            each([](float w) { return activate_near(w, kActGelu, false); });
          } else {
            each([](float w) { return w; });
          }
        }
      }
      if (col_type == kF32 && (ALIGNED || units > 0)) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const Raw8<kF32> s = load8<kF32, ALIGNED>(a.col, k[u]);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[u][e] *= __builtin_amdgcn_rcpf(elem8(s, e));
        }
      }
    }
    if (OP == kOpNorm || ytype >= kI8) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = umax(m, abs_bits(v[u][e]));
        top = umax(top, u * T + t < units ? m : 0);
      }
      row_reduce<W>(sum, top, red, parity, wave, lane);
      parity ^= 1;
    }
    const RowFactors f = row_factors<OP>(a, sum, top);
    if (ytype >= kI8) {
      if (OP == kOpNorm && f.pre != 1.0f) {
        vt *= f.pre;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[u][e] *= f.pre;
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u * T + t < units)
          store8_codes<ALIGNED>(a.y, row * a.ldy + k[u],
                                (u32x2){codes4(v[u], f.code, ytype == kE4m3), codes4(v[u] + 4, f.code, ytype == kE4m3)});
      if (tail) {
        const float w[4] = {vt, vt, vt, vt};
        static_cast<uint8_t*>(a.y)[row * a.ldy + kt] = (uint8_t)codes4(w, f.code, ytype == kE4m3);
      }
      if (t == 0) a.scale[row] = f.scale;
    } else {
      if (tail) store1(a.y, row * a.ldy + kt, OP == kOpNorm ? vt * f.mul : vt, ytype);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (OP == kOpNorm) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[u][e] *= f.mul;
        }
        if (u * T + t < units) {
          if (ytype == kF32) store8_f32<ALIGNED>(a.y, row * a.ldy + k[u], v[u]);
          else store8_bf16<ALIGNED>(a.y, row * a.ldy + k[u], v[u]);
        }
      }
    }
  }
}

// ---- any row: two passes ------------------------------------------------------------------------
// Rows longer than the registers of a block (32768 elements): single elements, read again for the store (1000 rows of
// 65536, rmsnorm bf16 -> e4m3: 278 us; eight units a lane spill registers to memory and take 331).
template <int OP, int XT, int BT>
__global__ __launch_bounds__(1024) void rows_any_kernel(const RowArgs a) {
  constexpr int W = 16;
  __shared__ float2 red[2][W];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    float h = 0.0f;
    auto value = [&](int64_t k) {  // h gamma, or act(g) u / s; h itself in h
      h = elem1<XT>(a.x, row * a.ldx + k);
      if constexpr (OP == kOpNorm) {
        if constexpr (BT != kNoOperand) h += elem1<BT>(a.b, row * a.ldb + k);
        return h * (a.col_type == kF32 ? elem1<kF32>(a.col, k) : elem1<kBf16>(a.col, k));
      } else {
        float v = activate(h, a.act, a.y_type == kF32);
        if constexpr (BT != kNoOperand) v *= elem1<BT>(a.b, row * a.ldb + k);
        return a.col_type == kF32 ? v * __builtin_amdgcn_rcpf(static_cast<const float*>(a.col)[k]) : v;
      }
    };
    float sum = 0.0f;
    uint32_t top = 0;
    if (OP == kOpNorm || a.y_type >= kI8) {
      for (int64_t k = threadIdx.x; k < a.K; k += 64 * W) {
        const float v = value(k);
        sum = fmaf(h, h, sum);
        top = umax(top, abs_bits(v));
      }
      row_reduce<W>(sum, top, red, parity, wave, lane);
      parity ^= 1;
    }
    const RowFactors f = row_factors<OP>(a, sum, top);
    for (int64_t k = threadIdx.x; k < a.K; k += 64 * W) {
      const float v = value(k);
      if (OP == kOpNorm && BT != kNoOperand && a.h != nullptr) store1(a.h, row * a.ldh + k, h, BT);
      if (a.y_type >= kI8) {
        const float c = v * f.pre, w[4] = {c, c, c, c};
        static_cast<uint8_t*>(a.y)[row * a.ldy + k] = (uint8_t)codes4(w, f.code, a.y_type == kE4m3);
      } else {
        store1(a.y, row * a.ldy + k, OP == kOpNorm ? v * f.mul : v, a.y_type);
      }
    }
    if (threadIdx.x == 0 && a.y_type >= kI8) a.scale[row] = f.scale;
  }
}


template <int OP, int XT, int BT, bool ALIGNED>
void launch_rows_as(const RowArgs& a, hipStream_t st) {
#define AWQ_ROWS(WV, UV) \
  rows_kernel<OP, XT, BT, WV, UV, ALIGNED> \
      <<<blocks_of(WV == 1 ? (a.M - 1) / 4 + 1 : a.M, WV == 1 ? 256 : 64 * WV), WV == 1 ? 256 : 64 * WV, 0, st>>>(a)
  const RowLayout l = row_layout(a.M, a.K, ALIGNED);
  if (l.waves == 0) {
    rows_any_kernel<OP, XT, BT><<<blocks_of(a.M, 1024), 1024, 0, st>>>(a);
  } else if (l.waves == 1) {
    AWQ_ROWS(1, 2);
  } else if (l.waves == 4 && l.units == 2) {
    AWQ_ROWS(4, 2);
  } else if (l.waves == 4 && l.units == 4) {
    AWQ_ROWS(4, 4);
  } else if (l.waves == 16 && l.units == 1) {
    AWQ_ROWS(16, 1);
  } else if (l.waves == 16 && l.units == 2) {
    AWQ_ROWS(16, 2);
  } else if (l.waves == 16 && l.units == 3) {
    AWQ_ROWS(16, 3);
  } else if (l.waves == 16) {
    AWQ_ROWS(16, 4);
  } else if constexpr (ALIGNED) {
    if (l.waves == 4 && l.units == 1) AWQ_ROWS(4, 1);
    else if (l.waves == 4) AWQ_ROWS(4, 3);
    else AWQ_ROWS(8, 3);
  }
#undef AWQ_ROWS
}
template <int OP, int XT, int BT>
hipError_t launch_rows(const RowArgs& a, bool aligned, hipStream_t st) {
  if (aligned) launch_rows_as<OP, XT, BT, true>(a, st);
  else launch_rows_as<OP, XT, BT, false>(a, st);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const RowArgs& a, int x_type, int b_type, bool vec, hipStream_t st) {
  if (x_type == kF32) {
    if (b_type == kNoOperand) return launch_rows<kOpNorm, kF32, kNoOperand>(a, vec, st);
    if (b_type == kF32) return launch_rows<kOpNorm, kF32, kF32>(a, vec, st);
    return launch_rows<kOpNorm, kF32, kBf16>(a, vec, st);
  }
  if (b_type == kNoOperand) return launch_rows<kOpNorm, kBf16, kNoOperand>(a, vec, st);
  if (b_type == kF32) return launch_rows<kOpNorm, kBf16, kF32>(a, vec, st);
  return launch_rows<kOpNorm, kBf16, kBf16>(a, vec, st);
}

hipError_t launch_act_mul(const RowArgs& a, int x_type, bool vec, hipStream_t st) {
  if (x_type == kF32)
    return a.b != nullptr ? launch_rows<kOpAct, kF32, kF32>(a, vec, st)
                          : launch_rows<kOpAct, kF32, kNoOperand>(a, vec, st);
  return a.b != nullptr ? launch_rows<kOpAct, kBf16, kBf16>(a, vec, st)
                        : launch_rows<kOpAct, kBf16, kNoOperand>(a, vec, st);
}

}  // namespace awq
