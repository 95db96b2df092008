// Mixture of experts over packed 4-bit weights, for the tokens of a decode batch or a short prompt:
//   Y[m] = sum_j w[m, j] D_e (act(G_e x[m]) * (U_e x[m])),  e = ids[m, j]
// The up kernel forms act(gate) * up of every (token, expert) pair, the down kernel its product with D_e times w, and a third
// kernel adds a token's pairs in order.  In the first two a block belongs to one expert and a run of its channels, keeps the
// expert's tokens as operands in registers and streams its part of the weight past them; experts with many tokens take
// them from LDS, 64 at a time.  Which tokens those are a block finds itself, by a scan of the ids.
//
// A weight code becomes a bf16 operand exactly, as 8 + q / 2 (a nibble moved into the mantissa of 8.0: one instruction per
// code and no conversion).  A group's sum x (q - z) / 2 is sum x (8 + q / 2) - (8 + z / 2) sum x in fp32 sums of exact
// products, then multiplied with the group's step in fp32.  The operands hold 2^-20 of these values and the channel's power of
// two the rest: 128 products with 8 + q / 2 reach 2^11 |x|, and the layout's steps are scaled to 2^10 and more, so that an x
// of 3e37 would take the sums out of fp32 where the result stays inside.  This way only the result's own magnitude does, in
// channels whose largest step is 2^-11 or more.  int8 activations take the integer products instead, whose sums are exact.
#include "moe_internal.h"
#include "moe_plan.h"
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

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
  return o > v ? o : v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<kDppMirror>(dpp_max<kDppHalfMirror>(dpp_max<kDppXor2>(dpp_max<kDppXor1>(v))));
  uint32_t m = 0;  // of the four rows of sixteen lanes
#pragma unroll
  for (int i = 0; i < 64; i += 16) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)v, i);
    m = o > m ? o : m;
  }
  return m;
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
constexpr float kSmall = 0x1p-20f;
struct W16 {
  bf16x8 h[4];  // 2^-20 (8 + q / 2)
  __device__ __forceinline__ explicit W16(const u32x4 w) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint32_t lo = w[s] << 3 & 0x78787878u, hi = w[s] >> 1 & 0x78787878u;
      constexpr uint32_t kUpper = 0x37373737u;  // the upper bytes of 2^-20 times 8.0 .. 15.5 in bf16
      h[s] = __builtin_bit_cast(
          bf16x8, (u32x4){__builtin_amdgcn_perm(lo, kUpper, 0x00050004), __builtin_amdgcn_perm(lo, kUpper, 0x00070006),
                          __builtin_amdgcn_perm(hi, kUpper, 0x00050004), __builtin_amdgcn_perm(hi, kUpper, 0x00070006)});
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

// ---- sums over a group ---------------------------------------------------------------------------------
// The activations of sixteen tokens (one per lane % 16) in a group, as operands: T bf16 terms, or int8 codes.
__device__ __forceinline__ bf16x8 constant8(uint32_t two) { return __builtin_bit_cast(bf16x8, (u32x4){two, two, two, two}); }

template <int T>
struct Terms {
  using Weight = W16;
  static constexpr float kUnit = 2.0f / kSmall;  // of sum()
  bf16x8 t[T][4];
  // 2^-20 sum x of the group, for the zero points
  __device__ __forceinline__ f32x4 ones() const {
    const bf16x8 one = constant8(pack_cut(kSmall, kSmall));
    f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = T - 1; k >= 0; --k)
#pragma unroll
      for (int s = 0; s < 4; ++s) r = __builtin_amdgcn_mfma_f32_16x16x32_bf16(t[k][s], one, r, 0, 0, 0);
    return r;
  }
  // 2^-20 sum x (q - z) / 2.  INNER: every 32 products with 8 + q / 2 are followed by 32 with -(8 + z / 2), so that no sum
  // grows past those 32 (a sum of 128 rounds at 12 sqrt(128) sigma for a result of 3 sqrt(128) sigma); z is a whole number.
  // For an fp32 result, whose error was up to 1.3e-6 of its norm without (20 tokens, 129 experts of 768 x 512); a bf16 result
  // rounds a thousand times that, and takes the half of the products.
  template <bool INNER>
  __device__ __forceinline__ f32x4 sum(const W16& w, float z, const f32x4 sx) const {
    f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (INNER) {
      const float m = fmaf(z, -0.5f * kSmall, -8.0f * kSmall);
      const bf16x8 mz = constant8(pack_cut(m, m));
#pragma unroll
      for (int k = T - 1; k >= 0; --k)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          r = __builtin_amdgcn_mfma_f32_16x16x32_bf16(t[k][s], w.h[s], r, 0, 0, 0);
          r = __builtin_amdgcn_mfma_f32_16x16x32_bf16(t[k][s], mz, r, 0, 0, 0);
        }
      return r;
    } else {
#pragma unroll
      for (int k = T - 1; k >= 0; --k)
#pragma unroll
        for (int s = 0; s < 4; ++s) r = __builtin_amdgcn_mfma_f32_16x16x32_bf16(t[k][s], w.h[s], r, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = fmaf(fmaf(z, -0.5f, -8.0f), sx[i], r[i]);
      return r;
    }
  }
};
struct Codes {
  using Weight = W8;
  static constexpr float kUnit = 1.0f;
  i32x4 b[2];
  // |sum| is below 2^18: its fp32 form is exact
  __device__ __forceinline__ static f32x4 dot(const i32x4 (&x)[2], const i32x4 (&w)[2]) {
    i32x4 r = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) r = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[i], w[i], r, 0, 0, 0);
    return (f32x4){(float)r[0], (float)r[1], (float)r[2], (float)r[3]};
  }
  __device__ __forceinline__ f32x4 ones() const {
    const i32x4 one = {0x01010101, 0x01010101, 0x01010101, 0x01010101}, o[2] = {one, one};
    return dot(b, o);
  }
  template <bool>
  __device__ __forceinline__ f32x4 sum(const W8& w, float z, const f32x4 sx) const {
    f32x4 r = dot(b, w.b);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = fmaf(-z, sx[i], r[i]);  // exact
    return r;
  }
};

// How a group of one token is read: from X, or from the planes that the up kernel left.
constexpr int kPlanes2 = 4, kPlanes3 = 5;  // beside kF32 .. kE4m3
// gather: piece(i) is where the group's i-th 16 bytes of the lane's token are, j = lane / 16 which of its channels;
// load: the same for a row in memory, from this lane's first channel on.
template <int XT>
struct Source {
  using Operand = Terms<XT == kF32 ? 3 : 1>;
  static constexpr int kSize = XT == kF32 ? 4 : XT == kBf16 ? 2 : 1, kPlanes = 1;
  template <typename Piece>
  static __device__ __forceinline__ void gather(Operand& o, Piece piece, int j, int) {
    X8<XT> x[4];
    if constexpr (kSize == 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(piece(j + 4 * i));
        x[2 * i].w[0] = v[0], x[2 * i].w[1] = v[1], x[2 * i + 1].w[0] = v[2], x[2 * i + 1].w[1] = v[3];
      }
    } else {
      constexpr int kEach = kSize / 2;  // pieces of eight channels
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(piece(kEach * (2 * j + 8 * (s / 2) + s % 2) + i));
#pragma unroll
          for (int d = 0; d < 4; ++d) x[s].w[4 * i + d] = v[d];
        }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      bf16x8 t[X8<XT>::kTerms];
      x[s].terms(t);
#pragma unroll
      for (int k = 0; k < X8<XT>::kTerms; ++k) o.t[k][s] = t[k];
    }
  }
  static __device__ __forceinline__ void load(Operand& o, const char* row, int64_t g, int64_t) {
    const char* p = row + g * kGroup * kSize;
    gather(o, [&](int i) AWQ_INLINE { return p + 16 * i; }, 0, 0);
  }
};
template <>
struct Source<kI8> {
  using Operand = Codes;
  static constexpr int kSize = 1, kPlanes = 1;
  template <typename Piece>
  static __device__ __forceinline__ void gather(Operand& o, Piece piece, int j, int) {
#pragma unroll
    for (int i = 0; i < 2; ++i) o.b[i] = *reinterpret_cast<const i32x4*>(piece(j + 4 * i));
  }
  static __device__ __forceinline__ void load(Operand& o, const char* row, int64_t g, int64_t) {
    const char* p = row + g * kGroup;
    gather(o, [&](int i) AWQ_INLINE { return p + 16 * i; }, 0, 0);
  }
};
template <int T>
struct Planes {
  using Operand = Terms<T>;
  static constexpr int kSize = 2, kPlanes = T;
  template <typename Piece>
  static __device__ __forceinline__ void gather(Operand& o, Piece piece, int j, int64_t plane) {  // plane: bytes
#pragma unroll
    for (int k = 0; k < T; ++k)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        o.t[k][s] = __builtin_bit_cast(
            bf16x8, *reinterpret_cast<const u32x4*>(piece(2 * j + 8 * (s / 2) + s % 2) + k * plane));
  }
  static __device__ __forceinline__ void load(Operand& o, const char* row, int64_t g, int64_t plane) {
    const char* p = row + g * (2 * kGroup);
    gather(o, [&](int i) AWQ_INLINE { return p + 16 * i; }, 0, plane);
  }
};
template <>
struct Source<kPlanes2> : Planes<2> {};
template <>
struct Source<kPlanes3> : Planes<3> {};

// ---- the pairs of an expert ---------------------------------------------------------------------------
// list: the pairs p < P with ids[p] = e, ascending; returns their number.  All of the block's WV waves; the ids are all
// requested at once (251 tokens, 8 of 64 experts: 3 us of the layer less than one turn after the other).
template <int WV>
__device__ __forceinline__ int expert_pairs(const int32_t* ids, int P, int e, uint16_t* list, int (*counts)[WV]) {
  constexpr int TURNS = kMoePairs / (64 * WV);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint64_t mask[TURNS];
  int id[TURNS];
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    const int p = 64 * WV * i + (int)threadIdx.x;
    id[i] = p < P ? ids[p] : -1;
  }
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    mask[i] = __ballot(id[i] == e);
    if (lane == 0) counts[i][wave] = __popcll(mask[i]);
  }
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    if (i > 0 && 64 * WV * i >= P) break;
    int before = total;
#pragma unroll
    for (int w = 0; w < WV; ++w) {
      const int c = counts[i][w];
      if (w < wave) before += c;
      total += c;
    }
    if (id[i] == e) list[before + __popcll(mask[i] & ((1ull << lane) - 1))] = (uint16_t)(64 * WV * i + (int)threadIdx.x);
  }
  __syncthreads();
  return total;
}

// Waves per SIMD that a kernel is built for, by its tokens' operands: four (two blocks of eight waves on a CU) up to 128 bytes
// of them, else two.  It bounds the registers and sizes the grid; what a kernel then needs may be less (fp32 X, one group a
// wave: 124 registers) or just above what lets a second block in (down in three terms, one group a wave: 130).
constexpr int waves_per_simd(size_t operands) { return operands <= 128 ? 4 : 2; }

// The expert of a slot: experts, where there are at least as many pairs as experts, else the expert of the pair of that
// number, which the first of its pairs takes for all.
__device__ __forceinline__ int slot_expert(const MoeArgs& p, const int32_t* ids, int slot) {
  const int e = p.by_pair ? __builtin_amdgcn_readfirstlane(ids[slot]) : slot;
  return e >= 0 && e < p.E ? e : -1;
}

// ---- an expert's tokens past a run of channel tiles -------------------------------------------------------
// The block's WV waves share the groups, NG each at a time, and take an expert's tokens sixteen at a time.  A step is a pair
// of channel tiles in WV NG groups; every group's codes are requested a step ahead, into the registers that it just freed.
// Where one step covers all groups the tokens' operands stay in registers while the weight passes; otherwise they are read
// again for every WV NG groups of PC pairs.  The waves' sums meet in LDS, in wave order, and out(list position, pair of
// tiles, channel, sum of the one tile, of the other) takes them.
struct Tiles {
  int64_t first, other;  // the run's first tile, and how much further the second of a pair is
  int step, count;       // from pair to pair; pairs
};

template <int SRC, int NG, int WV, int PC, bool INNER>
struct ExpertPass {
  using S = Source<SRC>;
  using Op = typename S::Operand;
  struct Group {
    u32x4 w[2];
    uint32_t dz[2];
  } buf[NG];
  ExpertWeights w;
  Tiles tiles;
  int G, wave, lane;

  __device__ __forceinline__ void fetch(int i, int pair, int g0) {
    const int g = g0 + wave + i * WV;
    if (g >= G) return;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int64_t at = (tiles.first + (int64_t)pair * tiles.step + q * tiles.other) * G + g;
      buf[i].w[q] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w.codes + at * 256) + (unsigned)lane);
      buf[i].dz[q] = (w.steps + at * 16)[(unsigned)(lane & 15)];
    }
  }
  __device__ __forceinline__ void begin() {
#pragma unroll
    for (int i = 0; i < NG; ++i) fetch(i, 0, 0);
  }

  // all of the expert's n tokens; row(list position) is a token's first channel for this lane
  template <typename Row, typename Out>
  __device__ __forceinline__ void run(int n, int64_t plane, float (*part)[WV][512], Row row, Out out) {
    const int c = lane & 15, j = lane >> 4;
    int turn = 0;
    for (int t0 = 0; t0 < n; t0 += 16) {
      const char* r = row(t0 + c < n ? t0 + c : n - 1);
      Op x[NG];
      f32x4 sx[NG];
      for (int p0 = 0; p0 < tiles.count; p0 += PC) {
        const int pairs = tiles.count - p0 < PC ? tiles.count - p0 : PC;
        f32x4 tot[PC][2];
#pragma unroll
        for (int u = 0; u < PC; ++u)
#pragma unroll
          for (int q = 0; q < 2; ++q) tot[u][q] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        for (int g0 = 0; g0 < G; g0 += WV * NG) {
          if (p0 == 0 || G > WV * NG) {
#pragma unroll
            for (int i = 0; i < NG; ++i) {
              const int g = g0 + wave + i * WV;
              if (g < G) S::load(x[i], r, g, plane);
            }
            if constexpr (!INNER) {
#pragma unroll
              for (int i = 0; i < NG; ++i)
                if (g0 + wave + i * WV < G) sx[i] = x[i].ones();
            }
          }
#pragma unroll
          for (int u = 0; u < PC; ++u) {
            if (u > 0 && u >= pairs) break;
            // the step after this one: the next pair, the next groups, the next pairs, the next tokens
            int npair = p0 + u + 1, ng0 = g0;
            bool more = true;
            if (u + 1 >= pairs) {
              npair = p0, ng0 = g0 + WV * NG;
              if (ng0 >= G) {
                npair = p0 + PC, ng0 = 0;
                if (npair >= tiles.count) npair = 0, more = t0 + 16 < n;
              }
            }
#pragma unroll
            for (int i = 0; i < NG; ++i) {
              if (g0 + wave + i * WV >= G) {  // none of this wave's here: only what comes next
                if (more) fetch(i, npair, ng0);
                continue;
              }
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const typename Op::Weight wq(buf[i].w[q]);
                const float d = half_lo(buf[i].dz[q]), z = half_lo(buf[i].dz[q] >> 16);
                const f32x4 v = x[i].template sum<INNER>(wq, z, sx[i]);
#pragma unroll
                for (int k = 0; k < 4; ++k) tot[u][q][k] = fmaf(d, v[k], tot[u][q][k]);
              }
              if (more) fetch(i, npair, ng0);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < PC; ++u) {
          if (u > 0 && u >= pairs) break;
          const int64_t first = (tiles.first + (int64_t)(p0 + u) * tiles.step) * 16 + (threadIdx.x & 15);
          const float power0 = Op::kUnit * w.powers[first], power1 = Op::kUnit * w.powers[first + 16 * tiles.other];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (t0 + 4 * j + k < n) {
              part[turn][wave][(4 * j + k) * 16 + c] = tot[u][0][k];
              part[turn][wave][256 + (4 * j + k) * 16 + c] = tot[u][1][k];
            }
          }
          __syncthreads();  // and the buffer of two turns ago has been read
          const int o = (int)threadIdx.x, at = t0 + o / 16;
          if (o < 256 && at < n) {
            float a = 0.0f, b = 0.0f;
#pragma unroll
            for (int v = 0; v < WV; ++v) a += part[turn][v][o], b += part[turn][v][256 + o];
            out(at, p0 + u, o % 16, a * power0, b * power1);
          }
          turn ^= 1;
        }
      }
    }
  }
};

__device__ __forceinline__ float activate(float g, int act) {
  if (act != 1) return 0.5f * g * erfcf(-g * 0.70710678f);
  const float e = expf(-fabsf(g));  // at most 1: no overflow far below zero
  return (g < 0.0f ? g * e : g) / (1.0f + e);
}

// h of a pair and channel as bf16 terms: all but the last cut, the last rounded.
__device__ __forceinline__ void store_h(const MoeArgs& p, int64_t plane, int pair, int ch, float v) {
  uint16_t* h = p.h + (int64_t)pair * p.I + ch;
  for (int s = 0; s < p.terms - 1; ++s) {
    h[s * plane] = (uint16_t)(bits(v) >> 16);
    v -= cut(v);
  }
  h[(p.terms - 1) * plane] = (uint16_t)pack_rne(v, v);
}

// act(gate) * up.  A block: a slot, `per` tiles of sixteen channels of I.
// ROUTE: from the router's logits, for a token a wave; every block makes the routing for itself, and one writes it for the
// kernels behind (4 tokens, 8 of 128 experts: the layer takes 30.9 us, 32.0 with the router in a kernel of its own).
template <int XT, int NG, int WV, bool INNER, bool ROUTE>
__global__ __launch_bounds__(64 * WV, waves_per_simd(sizeof(typename Source<XT>::Operand) * NG)) void moe_up_kernel(
    const MoeArgs p, const RouteArgs r, bool lbf16, int per) {
  __shared__ float part[2][WV][512];
  __shared__ uint16_t list[kMoePairs];
  __shared__ int counts[kMoePairs / (64 * WV)][WV];
  const int lane = threadIdx.x & 63, j = lane >> 4;
  __shared__ int32_t routed[ROUTE ? WV * kMaxChosen : 1];
  const int slot = (int)blockIdx.y, P = p.M * p.k, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t* ids = p.ids;
  if constexpr (ROUTE) {
    if (wave < p.M) {
      int id;
      float w;
      route_token<kRouteHere / 64>(static_cast<const char*>(r.logits) + wave * r.ld * (lbf16 ? 2 : 4), lbf16, r.E, r.k, r.score,
                                   r.renorm, lane, id, w);
      if (lane < r.k) {
        routed[wave * r.k + lane] = id;
        if (blockIdx.x == 0 && slot == 0) r.ids[wave * r.k + lane] = id, r.weights[wave * r.k + lane] = w;
      }
    }
    __syncthreads();
    ids = routed;
  }
  const int e = slot_expert(p, ids, slot);
  if (e < 0) return;
  const int tile0 = (int)blockIdx.x * per, left = p.I / 16 - tile0;
  ExpertPass<XT, NG, WV, 1, INNER> pass;
  pass.w = p.up;
  pass.tiles = Tiles{(int64_t)e * (p.I / 8) + tile0, p.I / 16, 1, left < per ? left : per};
  pass.G = p.H / kGroup, pass.lane = lane, pass.wave = wave;
  pass.begin();
  const int n = expert_pairs<WV>(ids, P, e, list, counts);
  if (n == 0 || (p.by_pair && list[0] != slot)) return;
  const int64_t plane = (int64_t)P * p.I;
  pass.run(
      n, 0, part,
      [&](int i) AWQ_INLINE {
        return static_cast<const char*>(p.x) + ((int64_t)(list[i] / p.k) * p.ldx + 16 * j) * Source<XT>::kSize;
      },
      [&](int at, int pair, int ch, float g, float u) AWQ_INLINE {
        const int q = list[at];
        if constexpr (XT == kI8 || XT == kE4m3) {
          const float s = p.xscale[q / p.k];
          g *= s, u *= s;
        }
        store_h(p, plane, q, (tile0 + pair) * 16 + ch, activate(g, p.act) * u);
      });
}

// w D (...) of every pair.  A block: a slot, `per` pairs of tiles of sixteen channels of H.
template <int T, int NG, int WV, int PC>
__global__ __launch_bounds__(64 * WV, waves_per_simd(sizeof(Terms<T>) * NG)) void moe_down_kernel(const MoeArgs p, int per) {
  __shared__ float part[2][WV][512];
  __shared__ uint16_t list[kMoePairs];
  __shared__ int counts[kMoePairs / (64 * WV)][WV];
  const int lane = threadIdx.x & 63, j = lane >> 4;
  const int slot = (int)blockIdx.y, P = p.M * p.k, e = slot_expert(p, p.ids, slot);
  if (e < 0) return;
  const int pair0 = (int)blockIdx.x * per, left = p.H / 32 - pair0;
  ExpertPass<T == 2 ? kPlanes2 : kPlanes3, NG, WV, PC, T == 3> pass;
  pass.w = p.down;
  pass.tiles = Tiles{(int64_t)e * (p.H / 16) + 2 * pair0, 1, 2, left < per ? left : per};
  pass.G = p.I / kGroup, pass.lane = lane, pass.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  pass.begin();
  const int n = expert_pairs<WV>(p.ids, P, e, list, counts);
  if (n == 0 || (p.by_pair && list[0] != slot)) return;
  pass.run(
      n, (int64_t)P * p.I * 2, part,
      [&](int i) AWQ_INLINE { return reinterpret_cast<const char*>(p.h + (int64_t)list[i] * p.I + 16 * j); },
      [&](int at, int pair, int ch, float a, float b) AWQ_INLINE {
        const int q = list[at];
        float* o = p.o + (int64_t)q * p.H + (pair0 + pair) * 32 + ch;
        o[0] = a * p.weights[q];
        o[16] = b * p.weights[q];
      });
}

// ---- many tokens an expert: tiles ---------------------------------------------------------------------------
// A block of eight waves: an expert's tokens 16 TM at a time with 256 channels of the weight (up: 128 gate rows and the up
// rows beside them), all groups one after the other.  A wave has all the tokens and two channel tiles, whose codes come
// straight into registers a group or two ahead; the tokens come into LDS, two groups in turn, requested two groups ahead.
// Nothing is summed across waves, and a code is unpacked once for 16 TM tokens.
// Rows in LDS hold their 16-byte pieces at piece ^ swizzle(row): the reads of sixteen rows' same piece use every bank once.
template <int SRC, int TM>
struct TileStage {
  using S = Source<SRC>;
  static constexpr int kPlanes = S::kPlanes, kRow = kGroup * S::kSize, kPieces = kRow / 16;  // of a row of a plane
  static constexpr int kPer = (16 * TM * kPieces + 511) / 512;  // pieces of a plane per thread
  static constexpr int kPlane = 16 * TM * kRow, kBytes = kPlanes * kPlane;
  static __device__ __forceinline__ int place(int row, int piece) {
    return row * kRow + 16 * (piece ^ (kPieces == 8 ? row >> 1 & 7 : row & 15));
  }
  const char* from[kPer];  // null: nothing for this thread
  u32x4 v[kPlanes][kPer];
  // row(r) is where row r < rows of the tile starts in memory
  template <typename Row>
  __device__ __forceinline__ void point(int rows, Row row) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int q = (int)threadIdx.x + 512 * i;
      from[i] = q / kPieces < rows ? row(q / kPieces) + 16 * (q % kPieces) : nullptr;
    }
  }
  __device__ __forceinline__ void load(int g, int64_t plane) {
#pragma unroll
    for (int k = 0; k < kPlanes; ++k)
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (from[i] != nullptr) v[k][i] = *reinterpret_cast<const u32x4*>(from[i] + (int64_t)g * kRow + k * plane);
  }
  __device__ __forceinline__ void store(char* stage) const {
#pragma unroll
    for (int k = 0; k < kPlanes; ++k)
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int q = (int)threadIdx.x + 512 * i;
        if (from[i] != nullptr) *reinterpret_cast<u32x4*>(stage + k * kPlane + place(q / kPieces, q % kPieces)) = v[k][i];
      }
  }
  // the operand of the sixteen tokens from row 16 t on
  static __device__ __forceinline__ void read(typename S::Operand& o, const char* stage, int t, int c, int j) {
    const int row = 16 * t + c;
    auto piece = [&](int p) AWQ_INLINE { return stage + place(row, p); };
    S::gather(o, piece, j, kPlane);
  }
};

template <int SRC, int TM, bool INNER>
struct TilePass {
  using Stage = TileStage<SRC, TM>;
  using Op = typename Source<SRC>::Operand;
  // tot[t][q] of tiles tile[q] over all groups; used: the token tiles that hold any token.  All eight waves.
  static __device__ __forceinline__ void run(const ExpertWeights& w, const int64_t (&tile)[2], int G, Stage& st, int64_t plane,
                                             char* lds, int used, int lane, f32x4 (&tot)[TM][2]) {
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
      for (int q = 0; q < 2; ++q) tot[t][q] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    if (used <= 1) groups<1>(w, tile, G, st, plane, lds, lane, tot);
    else if (TM == 2 || used == 2) groups<2>(w, tile, G, st, plane, lds, lane, tot);
    else if (used == 3) groups<(TM < 3 ? TM : 3)>(w, tile, G, st, plane, lds, lane, tot);
    else groups<TM>(w, tile, G, st, plane, lds, lane, tot);
  }
  // Codes are requested two groups ahead where a group is few products, one ahead where these hide the way to memory.  us, one
  // ahead / two / as here: 16 experts of 4096 x 4096, 16 tokens each, 163 / 134 / 135; 8 of 4096 x 14336, 32 tokens each,
  // 384 / 365 / 343; 64 of 2048 x 1024, 31 tokens each, 107 / 108 / 106.
  template <int USED>
  static __device__ __forceinline__ void groups(const ExpertWeights& w, const int64_t (&tile)[2], int G, Stage& st,
                                                int64_t plane, char* lds, int lane, f32x4 (&tot)[TM][2]) {
    const int c = lane & 15, j = lane >> 4;
    constexpr int kAhead = TM == 4 && USED <= 2 ? 2 : 1;
    u32x4 codes[kAhead][2];
    uint32_t dz[kAhead][2];
    auto fetch = [&](auto parity, int g) AWQ_INLINE {
      constexpr int C = decltype(parity)::value % kAhead;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        codes[C][q] = *(reinterpret_cast<const u32x4*>(w.codes + (tile[q] * G + g) * 256) + (unsigned)lane);
        dz[C][q] = (w.steps + (tile[q] * G + g) * 16)[(unsigned)c];
      }
    };
    constexpr std::integral_constant<int, 0> even;
    constexpr std::integral_constant<int, 1> odd;
    fetch(even, 0);
    st.load(0, plane);
    __syncthreads();  // the stages have been read
    st.store(lds);
    if (G > 1) {
      if constexpr (kAhead == 2) fetch(odd, 1);
      st.load(1, plane);
    }
    __syncthreads();
    auto group = [&](auto parity, int g) AWQ_INLINE {
      constexpr int P = decltype(parity)::value, C = P % kAhead;
      const char* now = lds + P * Stage::kBytes;
      const typename Op::Weight op[2] = {typename Op::Weight(codes[C][0]), typename Op::Weight(codes[C][1])};
      float d[2], z[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) d[q] = half_lo(dz[C][q]), z[q] = half_lo(dz[C][q] >> 16);
      if (g + 1 < G) {
        if constexpr (kAhead == 1) fetch(parity, g + 1);
        st.store(lds + (1 - P) * Stage::kBytes);
      }
      if (g + 2 < G) {
        if constexpr (kAhead == 2) fetch(parity, g + 2);
        st.load(g + 2, plane);
      }
#pragma unroll
      for (int t = 0; t < USED; ++t) {
        Op x;
        Stage::read(x, now, t, c, j);
        f32x4 sx = {0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (!INNER) sx = x.ones();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const f32x4 v = x.template sum<INNER>(op[q], z[q], sx);
#pragma unroll
          for (int k = 0; k < 4; ++k) tot[t][q][k] = fmaf(d[q], v[k], tot[t][q][k]);
        }
      }
      __syncthreads();
    };
#pragma unroll 1
    for (int g = 0; g < G; g += 2) {
      group(even, g);
      if (g + 1 < G) group(odd, g + 1);
    }
  }
};

template <int XT, int TM, bool INNER>
__global__ __launch_bounds__(512) void moe_up_tile_kernel(const MoeArgs p) {
  using Stage = TileStage<XT, TM>;
  __shared__ __attribute__((aligned(16))) char lds[2 * Stage::kBytes];
  __shared__ uint16_t list[kMoePairs];
  __shared__ int counts[kMoePairs / 512][8];
  const int lane = threadIdx.x & 63, j = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = (int)blockIdx.y, P = p.M * p.k;
  const int n = expert_pairs<8>(p.ids, P, e, list, counts);
  const int tile0 = (int)blockIdx.x * 8 + wave;  // of I
  const int64_t first = (int64_t)e * (p.I / 8) + tile0, plane = (int64_t)P * p.I;
  const int64_t tile[2] = {first, first + p.I / 16};
  for (int t0 = (int)blockIdx.z * 16 * TM; t0 < n; t0 += 16 * TM * (int)gridDim.z) {
    Stage st;
    st.point(n - t0 < 16 * TM ? (n - t0 + 15) / 16 * 16 : 16 * TM, [&](int r) AWQ_INLINE {
      return static_cast<const char*>(p.x) + (int64_t)(list[t0 + r < n ? t0 + r : n - 1] / p.k) * p.ldx * Source<XT>::kSize;
    });
    f32x4 tot[TM][2];
    TilePass<XT, TM, INNER>::run(p.up, tile, p.H / kGroup, st, 0, lds, (n - t0 + 15) / 16, lane, tot);
    constexpr float kUnit = Source<XT>::Operand::kUnit;
    const float pg = kUnit * p.up.powers[tile[0] * 16 + c], pu = kUnit * p.up.powers[tile[1] * 16 + c];
#pragma unroll
    for (int t = 0; t < TM; ++t) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int at = t0 + 16 * t + 4 * j + k;
        if (at < n) {
          const int pair = list[at];
          float a = tot[t][0][k] * pg, b = tot[t][1][k] * pu;
          if constexpr (XT == kI8 || XT == kE4m3) a *= p.xscale[pair / p.k], b *= p.xscale[pair / p.k];
          store_h(p, plane, pair, tile0 * 16 + c, activate(a, p.act) * b);
        }
      }
    }
  }
}

template <int T, int TM>
__global__ __launch_bounds__(512) void moe_down_tile_kernel(const MoeArgs p) {
  constexpr int SRC = T == 2 ? kPlanes2 : kPlanes3;
  using Stage = TileStage<SRC, TM>;
  __shared__ __attribute__((aligned(16))) char lds[2 * Stage::kBytes];
  __shared__ uint16_t list[kMoePairs];
  __shared__ int counts[kMoePairs / 512][8];
  const int lane = threadIdx.x & 63, j = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e = (int)blockIdx.y, P = p.M * p.k;
  const int n = expert_pairs<8>(p.ids, P, e, list, counts);
  const int tiles = p.H / 16, tile0 = (int)blockIdx.x * 16 + 2 * wave;  // a wave has both or, past the end, none
  const int64_t first = (int64_t)e * tiles + (tile0 < tiles ? tile0 : 0);
  const int64_t tile[2] = {first, first + 1};
  for (int t0 = (int)blockIdx.z * 16 * TM; t0 < n; t0 += 16 * TM * (int)gridDim.z) {
    Stage st;
    st.point(n - t0 < 16 * TM ? (n - t0 + 15) / 16 * 16 : 16 * TM, [&](int r) AWQ_INLINE {
      return reinterpret_cast<const char*>(p.h + (int64_t)list[t0 + r < n ? t0 + r : n - 1] * p.I);
    });
    f32x4 tot[TM][2];
    TilePass<SRC, TM, T == 3>::run(p.down, tile, p.I / kGroup, st, (int64_t)P * p.I * 2, lds, (n - t0 + 15) / 16, lane, tot);
    if (tile0 >= tiles) continue;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float power = Terms<T>::kUnit * p.down.powers[tile[q] * 16 + c];
#pragma unroll
      for (int t = 0; t < TM; ++t) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = t0 + 16 * t + 4 * j + k;
          if (at < n) {
            const int pair = list[at];
            p.o[(int64_t)pair * p.H + (tile0 + q) * 16 + c] = tot[t][q][k] * power * p.weights[pair];
          }
        }
      }
    }
  }
}

// ---- sums in order -----------------------------------------------------------------------------------------
// Y from a token's pairs.
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

template <int XT, int NG, int WV, bool INNER>
void up_with(const MoeArgs& a, const RouteArgs* r, int l_type, unsigned slots, hipStream_t st) {
  const int per = units_per_block((int)slots, a.I / 16, WV, waves_per_simd(sizeof(typename Source<XT>::Operand) * NG));
  const dim3 grid((unsigned)((a.I / 16 + per - 1) / per), slots);
  if (r != nullptr) moe_up_kernel<XT, NG, WV, INNER, true><<<grid, 64 * WV, 0, st>>>(a, *r, l_type == kBf16, per);
  else moe_up_kernel<XT, NG, WV, INNER, false><<<grid, 64 * WV, 0, st>>>(a, RouteArgs{}, false, per);
}
template <int XT, bool INNER>
void launch_up(const MoeArgs& a, const RouteArgs* r, int l_type, unsigned slots, hipStream_t st) {
  const int G = a.H / kGroup;
  if (G <= 8) up_with<XT, 1, 8, INNER>(a, r, l_type, slots, st);
  else if (G <= 16) up_with<XT, 2, 8, INNER>(a, r, l_type, slots, st);
  else up_with<XT, XT == kF32 ? 1 : 2, 16, INNER>(a, r, l_type, slots, st);
}

template <int T, int NG, int WV, int PC>
void down_with(const MoeArgs& a, unsigned slots, hipStream_t st) {
  const int per = units_per_block((int)slots, a.H / 32, WV, waves_per_simd(sizeof(Terms<T>) * NG));
  moe_down_kernel<T, NG, WV, PC><<<dim3((unsigned)((a.H / 32 + per - 1) / per), slots), 64 * WV, 0, st>>>(a, per);
}
template <int T>
void launch_down(const MoeArgs& a, unsigned slots, hipStream_t st) {
  if (a.I / kGroup <= 8) down_with<T, 1, 8, 1>(a, slots, st);
  else if (a.I / kGroup <= 16) down_with<T, 1, 16, 1>(a, slots, st);
  else down_with<T, 1, 16, 2>(a, slots, st);
}

template <int XT, int TM, bool INNER>
void up_tiles(const MoeArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)(a.I / 128), (unsigned)a.E, tile_depth(a.M, a.k, a.E, 16 * TM));
  moe_up_tile_kernel<XT, TM, INNER><<<grid, 512, 0, st>>>(a);
}
template <int T, int TM>
void down_tiles(const MoeArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)((a.H + 255) / 256), (unsigned)a.E, tile_depth(a.M, a.k, a.E, 16 * TM));
  moe_down_tile_kernel<T, TM><<<grid, 512, 0, st>>>(a);
}

template <int XT, bool INNER>
void launch_products(const MoeArgs& a, const RouteArgs* r, int l_type, hipStream_t st) {
  const unsigned slots = (unsigned)(a.by_pair ? a.M * a.k : a.E);
  if (in_tiles(a.M, a.k, a.E)) up_tiles<XT, XT == kF32 ? 2 : 4, INNER>(a, st);
  else launch_up<XT, INNER>(a, r, l_type, slots, st);
}
template <int T>
void launch_sums(const MoeArgs& a, hipStream_t st) {
  const unsigned slots = (unsigned)(a.by_pair ? a.M * a.k : a.E);
  if (in_tiles(a.M, a.k, a.E)) down_tiles<T, T == 2 ? 4 : 2>(a, st);
  else launch_down<T>(a, slots, st);
  moe_sum_kernel<<<dim3((unsigned)((a.H + 1023) / 1024), (unsigned)a.M), 256, 0, st>>>(a);
}

template <int XT>
hipError_t launch_experts(MoeArgs a, const RouteArgs* r, int l_type, hipStream_t st) {
  a.by_pair = a.M * a.k < a.E;
  if (a.terms == 2) {
    launch_products<XT, false>(a, r, l_type, st);
    launch_sums<2>(a, st);
  } else {
    launch_products<XT, XT != kI8>(a, r, l_type, st);
    launch_sums<3>(a, st);
  }
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

// Up to eight tokens (a wave of the smallest block each) that do not run in tiles, and few enough experts.
bool moe_routes(int64_t M, int k, int E) { return M <= 8 && E <= kRouteHere && !in_tiles(M, k, E); }

hipError_t launch_moe(const MoeArgs& a, const RouteArgs* r, int l_type, int x_type, hipStream_t st) {
  switch (x_type) {
    case kF32: return launch_experts<kF32>(a, r, l_type, st);
    case kBf16: return launch_experts<kBf16>(a, r, l_type, st);
    case kI8: return launch_experts<kI8>(a, r, l_type, st);
    default: return launch_experts<kE4m3>(a, r, l_type, st);
  }
}

}  // namespace awq
