// Mixture of experts over packed 4-bit weights, for the tokens of a decode batch or a short prompt:
//   Y[m] = sum_j w[m, j] D_e (act(G_e x[m]) * (U_e x[m])),  e = ids[m, j]
// Kernel 1 (up) forms act(gate) * up of every (token, expert) pair, kernel 2 (down) its product with D_e times w, kernel 3
// adds a token's pairs in order.  A block belongs to one expert and some of its channels and streams that part of the weight
// once for up to 32 of the expert's tokens; which tokens those are it finds itself, by a scan of the ids.
//
// A weight code becomes a bf16 operand exactly, as 16 + q (a nibble moved into the mantissa of 16.0: one instruction per
// code and no conversion); a group's products with q - z are sum x (16 + q) - (16 + z) sum x, the second sum a product
// with ones.  Both are fp32 sums of exact products, then multiplied with the group's step in fp32.  int8 activations take
// the integer products instead, whose sums are exact.
#include "moe_internal.h"
#include "x_operand.h"

namespace awq {
namespace {

#define AWQ_INLINE __attribute__((always_inline))

// ---- the router -----------------------------------------------------------------------------------
// A wave per token: lane l holds the logits of experts l, l + 64, ...  as integers of the same order.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t b = bits(v + 0.0f);  // -0 is 0
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  if (k == 0xffffffffu) return __builtin_nanf("");
  return flt(k >> 31 ? k & 0x7fffffffu : ~k);
}
constexpr uint32_t kMasked = 0x007fffffu;  // -Inf; below: no expert

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int i = 1; i < 64; i *= 2) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, i, 64);
    v = o > v ? o : v;
  }
  return v;
}

// The k choices of one token: lane j < k gets the j-th's expert and weight.
template <int V>
__device__ __forceinline__ void route_token(const void* row, bool lbf16, int E, int k, int score, bool renorm, int lane,
                                            int& id, float& weight) {
  uint32_t key[V];
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = lane + 64 * i;
    v[i] = e >= E   ? -__builtin_inff()
           : lbf16 ? flt((uint32_t) static_cast<const uint16_t*>(row)[e] << 16)
                   : static_cast<const float*>(row)[e];
    key[i] = e < E ? order_key(v[i]) : 0u;
  }
  uint32_t best = 0, top = 0;
  int at = 0;
  auto local = [&]() AWQ_INLINE {
    best = key[0], at = 0;
#pragma unroll
    for (int i = 1; i < V; ++i)
      if (key[i] > best) best = key[i], at = i;
  };
  local();
  id = -1;
  float mine = -__builtin_inff();
  for (int j = 0; j < k; ++j) {
    const uint32_t m = wave_max(best);
    if (j == 0) top = m;
    if (m <= kMasked) break;
    // the lowest index among the lanes that hold the largest: lane and place, the place counts first
    uint64_t has = __ballot(best == m);
    int owner = (int)__builtin_ctzll(has);
    int place = __builtin_amdgcn_readlane(at, owner);
    for (has &= has - 1; has != 0; has &= has - 1) {
      const int l = (int)__builtin_ctzll(has), pl = __builtin_amdgcn_readlane(at, l);
      if (pl < place) owner = l, place = pl;
    }
    if (lane == j) id = owner + 64 * place, mine = key_value(m);
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == at) key[i] = 0u;
      local();
    }
  }
  const float vmax = key_value(top);
  float s;
  if (score == kSoftmax) {
    s = id >= 0 ? expf(mine - vmax) : 0.0f;
    float sum = 0.0f;
    if (renorm) {
      sum = s;
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) sum += lane + 64 * i < E ? expf(v[i] - vmax) : 0.0f;
    }
    sum = wave_sum(sum);
    // a NaN or +Inf that was not among the chosen (or stands alone) makes the row NaN
    bool bad = vmax != vmax || vmax == __builtin_inff();
    weight = id < 0 ? 0.0f : bad ? __builtin_nanf("") : s / sum;
  } else {
    // scores below fp32's range keep their ratios: all are taken relative to the largest negative exponent
    const float c = renorm && vmax < 0.0f ? vmax : 0.0f;
    s = id < 0 ? 0.0f : mine >= 0.0f ? 1.0f / (1.0f + expf(-mine)) : expf(mine - c) / (1.0f + expf(mine));
    if (mine != mine) s = mine;
    const float sum = renorm ? wave_sum(s) : 1.0f;
    weight = id < 0 ? 0.0f : s / sum;
  }
}

template <int V>
__global__ __launch_bounds__(256) void moe_route_kernel(const RouteArgs p, bool lbf16) {
  const int lane = threadIdx.x & 63;
  const int64_t m = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (m >= p.M) return;
  const void* row = static_cast<const char*>(p.logits) + m * p.ld * (lbf16 ? 2 : 4);
  int id;
  float w;
  route_token<V>(row, lbf16, p.E, p.k, p.score, p.renorm, lane, id, w);
  if (lane < p.k) p.ids[m * p.k + lane] = id, p.weights[m * p.k + lane] = w;
}

// ---- operands of a group of 128 channels -------------------------------------------------------------
// The weight's layout gives lane l, of channel l % 16, the codes of k = 16 (l / 16) .. + 15 and 64 further on; step s of
// four takes eight of them, of both operands.
struct W16 {
  bf16x8 h[4];  // 16 + q
  __device__ __forceinline__ explicit W16(const u32x4 w) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint32_t lo = (w[s] << 3 & 0x78787878u) | 0x80808080u, hi = (w[s] >> 1 & 0x78787878u) | 0x80808080u;
      constexpr uint32_t k41 = 0x41414141u;  // the upper bytes of 16.0 .. 31.0 in bf16
      h[s] = __builtin_bit_cast(bf16x8, (u32x4){__builtin_amdgcn_perm(lo, k41, 0x00050004), __builtin_amdgcn_perm(lo, k41, 0x00070006),
                                                __builtin_amdgcn_perm(hi, k41, 0x00050004), __builtin_amdgcn_perm(hi, k41, 0x00070006)});
    }
  }
};
struct W8 {
  i32x4 b[2];
  __device__ __forceinline__ explicit W8(const u32x4 w) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      b[s / 2][2 * (s % 2)] = (int)(w[s] & 0x0f0f0f0fu);
      b[s / 2][2 * (s % 2) + 1] = (int)(w[s] >> 4 & 0x0f0f0f0fu);
    }
  }
};

template <int T>
__device__ __forceinline__ f32x4 dot(const bf16x8 (&x)[4][T], const bf16x8 (&w)[4]) {
  f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int t = T - 1; t >= 0; --t)
#pragma unroll
    for (int s = 0; s < 4; ++s) r = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[s][t], w[s], r, 0, 0, 0);
  return r;
}

// A group of one token per lane % 16.  kTerms: bf16 terms, as stored (planes) or made from the type.
constexpr int kPlanes2 = 4, kPlanes3 = 5;  // beside kF32 .. kE4m3
template <int XT>
struct Tokens {
  using Weight = W16;
  static constexpr float kZero = 16.0f;  // what the operand holds beyond q
  static constexpr int kTerms = XT == kF32 ? 3 : 1, kSize = XT == kF32 ? 4 : XT == kBf16 ? 2 : 1;
  X8<XT> x[4];
  __device__ __forceinline__ void load(const char* row, int64_t g, int64_t) {
    const char* p = row + g * kGroup * kSize;
    if constexpr (kSize == 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(p + 64 * i);
        x[2 * i].w[0] = v[0], x[2 * i].w[1] = v[1], x[2 * i + 1].w[0] = v[2], x[2 * i + 1].w[1] = v[3];
      }
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) x[s].load(p + (64 * (s / 2) + 8 * (s % 2)) * kSize);
    }
  }
  template <int CT>
  __device__ __forceinline__ void products(const Weight* w, f32x4 (&s)[CT], f32x4& sx) const {
    bf16x8 t[4][kTerms];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i].terms(t[i]);
    const u32x4 o = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    const bf16x8 one = __builtin_bit_cast(bf16x8, o), ones[4] = {one, one, one, one};
    sx = dot<kTerms>(t, ones);
#pragma unroll
    for (int q = 0; q < CT; ++q) s[q] = dot<kTerms>(t, w[q].h);
  }
};
template <>
struct Tokens<kI8> {
  using Weight = W8;
  static constexpr float kZero = 0.0f;
  static constexpr int kSize = 1;
  i32x4 x[2];
  __device__ __forceinline__ void load(const char* row, int64_t g, int64_t) {
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = *reinterpret_cast<const i32x4*>(row + g * kGroup + 64 * i);
  }
  // |sum| is below 2^18: its fp32 form is exact
  __device__ __forceinline__ static f32x4 dot8(const i32x4 (&x)[2], const i32x4 (&w)[2]) {
    i32x4 r = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) r = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[i], w[i], r, 0, 0, 0);
    return (f32x4){(float)r[0], (float)r[1], (float)r[2], (float)r[3]};
  }
  template <int CT>
  __device__ __forceinline__ void products(const Weight* w, f32x4 (&s)[CT], f32x4& sx) const {
    const i32x4 one = {0x01010101, 0x01010101, 0x01010101, 0x01010101}, ones[2] = {one, one};
    sx = dot8(x, ones);
#pragma unroll
    for (int q = 0; q < CT; ++q) s[q] = dot8(x, w[q].b);
  }
};
template <int T>
struct Planes {
  using Weight = W16;
  static constexpr float kZero = 16.0f;
  static constexpr int kSize = 2;
  u32x4 x[T][4];
  __device__ __forceinline__ void load(const char* row, int64_t g, int64_t plane) {  // plane: bytes
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        x[t][s] = *reinterpret_cast<const u32x4*>(row + t * plane + g * (2 * kGroup) + 128 * (s / 2) + 16 * (s % 2));
  }
  template <int CT>
  __device__ __forceinline__ void products(const Weight* w, f32x4 (&s)[CT], f32x4& sx) const {
    bf16x8 t[4][T];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < T; ++k) t[i][k] = __builtin_bit_cast(bf16x8, x[k][i]);
    const u32x4 o = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    const bf16x8 one = __builtin_bit_cast(bf16x8, o), ones[4] = {one, one, one, one};
    sx = dot<T>(t, ones);
#pragma unroll
    for (int q = 0; q < CT; ++q) s[q] = dot<T>(t, w[q].h);
  }
};
template <>
struct Tokens<kPlanes2> : Planes<2> {};
template <>
struct Tokens<kPlanes3> : Planes<3> {};

// ---- the pairs of an expert ---------------------------------------------------------------------------
// list: the pairs p < P with ids[p] = e, ascending; returns their number.  All of the block's 512 threads.
__device__ __forceinline__ int expert_pairs(const int32_t* ids, int P, int e, uint16_t* list, int* counts) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int total = 0;
  for (int p0 = 0; p0 < P; p0 += 512) {
    const int p = p0 + (int)threadIdx.x;
    const bool hit = p < P && ids[p] == e;
    const uint64_t mask = __ballot(hit);
    if (p0 > 0) __syncthreads();  // counts of the pass before are read
    if (lane == 0) counts[wave] = __popcll(mask);
    __syncthreads();
    int before = total;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const int c = counts[w];
      if (w < wave) before += c;
      total += c;
    }
    if (hit) list[before + __popcll(mask & ((1ull << lane) - 1))] = (uint16_t)p;
  }
  __syncthreads();
  return total;
}

// The block's expert and the list of its pairs: expert `slot` where slots are experts, else the expert of pair `slot`,
// which the first of its pairs takes for all.  False: nothing to do, for the whole block.
__device__ __forceinline__ bool block_expert(const MoeArgs& p, int slot, int P, bool by_pair, int e, uint16_t* list,
                                             int* counts, int& n) {
  if (e < 0 || e >= p.E) return false;
  n = expert_pairs(p.ids, P, e, list, counts);
  return n > 0 && (!by_pair || list[0] == slot);
}

// ---- the stream ---------------------------------------------------------------------------------------
// tot[t][q] of 16 TT tokens (row[t]: this lane's, at its channels) with two channel tiles, over this wave's groups: wave,
// wave + 8, ...; D groups are requested ahead.
template <typename X, int TT>
__device__ __forceinline__ void stream(const ExpertWeights& w, const int64_t (&tile)[2], int G, int wave, int lane,
                                       const char* const (&row)[TT], int64_t plane, f32x4 (&tot)[TT][2]) {
  constexpr int WV = 8, D = sizeof(X) * TT > 128 ? 1 : 2;
  const int c = lane & 15;
  const uint32_t* codes[2];
  const uint32_t* steps[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) codes[q] = w.codes + tile[q] * G * 256, steps[q] = w.steps + tile[q] * G * 16;
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int q = 0; q < 2; ++q) tot[t][q] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  struct Group {
    u32x4 w[2];
    uint32_t dz[2];
    X x[TT];
  } buf[D];
  auto fetch = [&](Group& b, int64_t g) AWQ_INLINE {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      b.w[q] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(codes[q] + g * 256) + (unsigned)lane);
      b.dz[q] = (steps[q] + g * 16)[(unsigned)c];
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) b.x[t].load(row[t], g, plane);
  };
  auto use = [&](const Group& b) AWQ_INLINE {
    const typename X::Weight op[2] = {typename X::Weight(b.w[0]), typename X::Weight(b.w[1])};
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      f32x4 s[2], sx;
      b.x[t].template products<2>(op, s, sx);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float d = half_lo(b.dz[q]), z = half_lo(b.dz[q] >> 16) + X::kZero;
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[t][q][i] = fmaf(d, fmaf(-z, sx[i], s[q][i]), tot[t][q][i]);
      }
    }
  };
  const int n = (G - wave + WV - 1) / WV;  // this wave's groups (none or fewer where G < wave)
#pragma unroll
  for (int i = 0; i < D; ++i)
    if (i < n) fetch(buf[i], wave + i * WV);
  for (int i0 = 0; i0 < n; i0 += D)
#pragma unroll
    for (int i = 0; i < D; ++i) {
      if (i0 + i < n) use(buf[i]);
      if (i0 + i + D < n) fetch(buf[i], wave + (int64_t)(i0 + i + D) * WV);
    }
}

__device__ __forceinline__ float activate(float g, int act) {
  if (act != 1) return 0.5f * g * erfcf(-g * 0.70710678f);
  const float e = expf(-fabsf(g));  // at most 1: no overflow far below zero
  return (g < 0.0f ? g * e : g) / (1.0f + e);
}

// ---- kernel 1: act(gate) * up ----------------------------------------------------------------------------
// A block: one expert, sixteen channels of I (a tile of gate rows and the tile of up rows beside it), its tokens 16 TT at a
// time.
template <int XT, int TT>
__global__ __launch_bounds__(512) void moe_up_kernel(const MoeArgs p, bool by_pair) {
  using X = Tokens<XT>;
  __shared__ float part[8][512];
  __shared__ uint16_t list[kMoePairs];
  __shared__ int counts[8];
  const int lane = threadIdx.x & 63, j = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slot = (int)blockIdx.y, P = p.M * p.k;
  const int e = by_pair ? __builtin_amdgcn_readfirstlane(p.ids[slot]) : slot;
  int n = 0;
  if (!block_expert(p, slot, P, by_pair, e, list, counts, n)) return;
  const int64_t first = (int64_t)e * (p.I / 8) + blockIdx.x;  // its gate tile
  const int64_t tile[2] = {first, first + p.I / 16};
  const int64_t plane = (int64_t)P * p.I;
  for (int t0 = 0; t0 < n; t0 += 16 * TT) {
    const char* row[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int i = t0 + 16 * t + c;
      row[t] = static_cast<const char*>(p.x) + ((int64_t)(list[i < n ? i : n - 1] / p.k) * p.ldx + 16 * j) * X::kSize;
    }
    f32x4 tot[TT][2];
    stream<X, TT>(p.up, tile, p.H / kGroup, wave, lane, row, 0, tot);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      __syncthreads();  // the sums before are read
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][q * 256 + (4 * j + i) * 16 + c] = tot[t][q][i];
      __syncthreads();
      const int o = (int)threadIdx.x, at = t0 + 16 * t + o / 16;
      if (o < 256 && at < n) {
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) g += part[w][o], u += part[w][256 + o];
        const int pair = list[at];
        g *= p.up.powers[tile[0] * 16 + o % 16];
        u *= p.up.powers[tile[1] * 16 + o % 16];
        if constexpr (XT == kI8 || XT == kE4m3) {
          const float s = p.xscale[pair / p.k];
          g *= s, u *= s;
        }
        float v = activate(g, p.act) * u;
        uint16_t* h = p.h + (int64_t)pair * p.I + (int64_t)blockIdx.x * 16 + o % 16;
        for (int s = 0; s < p.terms - 1; ++s) {  // all but the last cut, the last rounded
          h[s * plane] = (uint16_t)(bits(v) >> 16);
          v -= cut(v);
        }
        h[(p.terms - 1) * plane] = (uint16_t)pack_rne(v, v);
      }
    }
  }
}

// ---- kernel 2: w D (...) per pair ---------------------------------------------------------------------------
// A block: one expert, 32 channels of H.
template <int T, int TT>
__global__ __launch_bounds__(512) void moe_down_kernel(const MoeArgs p, bool by_pair) {
  using X = Tokens<T == 2 ? kPlanes2 : kPlanes3>;
  __shared__ float part[8][512];
  __shared__ uint16_t list[kMoePairs];
  __shared__ int counts[8];
  const int lane = threadIdx.x & 63, j = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slot = (int)blockIdx.y, P = p.M * p.k;
  const int e = by_pair ? __builtin_amdgcn_readfirstlane(p.ids[slot]) : slot;
  int n = 0;
  if (!block_expert(p, slot, P, by_pair, e, list, counts, n)) return;
  const int64_t first = (int64_t)e * (p.H / 16) + 2 * blockIdx.x;
  const int64_t tile[2] = {first, first + 1};
  const int64_t plane = (int64_t)P * p.I * 2;
  for (int t0 = 0; t0 < n; t0 += 16 * TT) {
    const char* row[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int i = t0 + 16 * t + c;
      row[t] = reinterpret_cast<const char*>(p.h + (int64_t)list[i < n ? i : n - 1] * p.I + 16 * j);
    }
    f32x4 tot[TT][2];
    stream<X, TT>(p.down, tile, p.I / kGroup, wave, lane, row, plane, tot);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      __syncthreads();
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][(4 * j + i) * 32 + 16 * q + c] = tot[t][q][i];
      __syncthreads();
      const int o = (int)threadIdx.x, at = t0 + 16 * t + o / 32;
      if (at < n) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += part[w][o];
        const int pair = list[at];
        p.o[(int64_t)pair * p.H + (int64_t)blockIdx.x * 32 + o % 32] = s * p.down.powers[first * 16 + o % 32] * p.weights[pair];
      }
    }
  }
}

// ---- kernel 3: a token's pairs in order -----------------------------------------------------------------------
__global__ __launch_bounds__(256) void moe_sum_kernel(const MoeArgs p) {
  const int m = (int)blockIdx.y, n = ((int)blockIdx.x * 256 + (int)threadIdx.x) * 4;
  if (n >= p.H) return;
  f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < p.k; ++j) {
    const int e = p.ids[m * p.k + j];
    if (e >= 0 && e < p.E) s += *reinterpret_cast<const f32x4*>(p.o + ((int64_t)m * p.k + j) * p.H + n);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (p.ybf16) static_cast<uint16_t*>(p.y)[m * p.ldy + n + i] = (uint16_t)pack_rne(s[i], s[i]);
    else static_cast<float*>(p.y)[m * p.ldy + n + i] = s[i];
  }
}

template <int XT>
hipError_t launch_experts(const MoeArgs& a, hipStream_t st) {
  const int P = a.M * a.k;
  const bool by_pair = P < a.E;
  const unsigned slots = (unsigned)(by_pair ? P : a.E);
  const bool wide = P > 8 * a.E;  // more than eight tokens an expert: 32 at a time
  const dim3 up((unsigned)(a.I / 16), slots), down((unsigned)(a.H / 32), slots);
  if (wide) moe_up_kernel<XT, 2><<<up, 512, 0, st>>>(a, by_pair);
  else moe_up_kernel<XT, 1><<<up, 512, 0, st>>>(a, by_pair);
  if (a.terms == 2) {
    if (wide) moe_down_kernel<2, 2><<<down, 512, 0, st>>>(a, by_pair);
    else moe_down_kernel<2, 1><<<down, 512, 0, st>>>(a, by_pair);
  } else {
    if (wide) moe_down_kernel<3, 2><<<down, 512, 0, st>>>(a, by_pair);
    else moe_down_kernel<3, 1><<<down, 512, 0, st>>>(a, by_pair);
  }
  moe_sum_kernel<<<dim3((unsigned)((a.H + 1023) / 1024), (unsigned)a.M), 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, int l_type, hipStream_t st) {
  const unsigned blocks = (unsigned)((a.M + 3) / 4);
  const bool b = l_type == kBf16;
  if (a.E <= 64) moe_route_kernel<1><<<blocks, 256, 0, st>>>(a, b);
  else if (a.E <= 128) moe_route_kernel<2><<<blocks, 256, 0, st>>>(a, b);
  else if (a.E <= 256) moe_route_kernel<4><<<blocks, 256, 0, st>>>(a, b);
  else if (a.E <= 512) moe_route_kernel<8><<<blocks, 256, 0, st>>>(a, b);
  else moe_route_kernel<16><<<blocks, 256, 0, st>>>(a, b);
  return hipGetLastError();
}

hipError_t launch_moe(const MoeArgs& a, int x_type, hipStream_t st) {
  switch (x_type) {
    case kF32: return launch_experts<kF32>(a, st);
    case kBf16: return launch_experts<kBf16>(a, st);
    case kI8: return launch_experts<kI8>(a, st);
    default: return launch_experts<kE4m3>(a, st);
  }
}

}  // namespace awq
