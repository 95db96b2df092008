// Low-rank adapters of many requests beside a shared projection:
//   Y[m] = base[m] + s_a B_a (A_a x[m]),  a = ids[m]
// in two kernels, t = s_a A_a x and Y = base + B_a t, on the bf16 matrix cores.  Tokens are taken sixteen at a time, as
// they stand: a tile's distinct adapters are found with a few ballots, each is multiplied with all sixteen rows, and
// only the rows that are its own are kept.  Nothing is sorted, and the rows of other adapters cost no memory traffic.
#include "lora_internal.h"
#include "x_operand.h"

namespace awq {
namespace {

#define AWQ_INLINE __attribute__((always_inline))

constexpr int kNone = -1;    // the row keeps its base
constexpr int kAbsent = -2;  // no row

// The adapter of the tile's row c = lane % 16.
__device__ __forceinline__ int row_adapter(const LoraArgs& p, int64_t m0, int c) {
  if (m0 + c >= p.M) return kAbsent;
  const int id = p.ids[m0 + c];
  return id >= 0 && id < p.n ? id : kNone;
}

// Calls f(adapter, rows as a mask) for the distinct adapters of the tile (kNone among them) whose place among the
// distinct ones is `part` modulo `parts`; uniform over the wave.
template <typename F>
__device__ __forceinline__ void each_adapter(int id, int part, int parts, F f) {
  uint32_t left = (uint32_t)__ballot(id != kAbsent) & 0xffffu;
  for (int at = 0; left != 0; ++at) {
    const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    const uint32_t same = (uint32_t)__ballot(id == a) & 0xffffu;
    left &= ~same;
    if (at % parts == part) f(a, same);
  }
}

__device__ __forceinline__ int adapter_rank(const LoraArgs& p, int a) {
  if (p.ranks == nullptr) return p.R;
  const int r = p.ranks[a];
  return r < 0 ? 0 : r < p.R ? r : p.R;
}

// t[split][m][r] = scale (xscale sum_k x[m, k] A[r, k]) over the split's share of K.  A block: sixteen tokens, RT tiles of
// sixteen ranks, its eight waves taking steps of 64 channels in turn, U at a time.  The tokens of the first U steps are
// requested before the adapter is known and stay in registers for all of the tile's adapters: with as many splits as
// lora_splits makes, that is often all of K.
template <int XT, int RT>
__global__ __launch_bounds__(512) void lora_down_kernel(const LoraArgs p, int parts, int rank_blocks) {
  constexpr int WV = 8, U = XT == kF32 ? (RT == 1 ? 2 : 1) : 4 / RT;
  __shared__ float sums[WV][RT * 256];
  const int lane = threadIdx.x & 63, j = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)blockIdx.x * 16;
  const int part = (int)blockIdx.y / rank_blocks, r0 = ((int)blockIdx.y % rank_blocks) * RT * 16;
  const int split = (int)blockIdx.z;
  const int id = row_adapter(p, m0, c);
  const int xs = XT == kF32 ? 4 : XT == kBf16 ? 2 : 1;
  const char* xrow = static_cast<const char*>(p.x) + ((m0 + c < p.M ? m0 + c : p.M - 1) * p.ldx + 16 * j) * xs;
  const int64_t steps = (p.K + 63) / 64, s0 = (int64_t)split * WV + wave, stride = (int64_t)WV * p.splits;
  // a step's 64 channels: lane / 16 has sixteen of them, in two operands
  X8<XT> x[U][2];
  auto load_x = [&](int64_t s) AWQ_INLINE {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t k = 64 * (s + u * stride) + 8 * h;
        if (k + 16 * j < p.K) x[u][h].load(xrow + k * xs);
        else x[u][h].clear();
      }
  };
  load_x(s0);
  each_adapter(id, part, parts, [&](int a, uint32_t rows) AWQ_INLINE {
    if (a == kNone) return;
    const int rank = adapter_rank(p, a);
    if (r0 >= rank) return;
    const uint16_t* arow[RT];
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      const int r = r0 + 16 * q + c < rank ? r0 + 16 * q + c : rank - 1;  // past the rank: its last row again, not kept
      arow[q] = p.a + ((int64_t)a * p.R + r) * p.K + 16 * j;
    }
    f32x4 acc[RT];
#pragma unroll
    for (int q = 0; q < RT; ++q) acc[q] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t s = s0; s < steps; s += U * stride) {
      if (s0 + U * stride < steps) load_x(s);
      X8<kBf16> w[U][2][RT];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t k = 64 * (s + u * stride) + 8 * h;
#pragma unroll
          for (int q = 0; q < RT; ++q) {
            if (k + 16 * j < p.K) w[u][h][q].load(reinterpret_cast<const char*>(arow[q] + k));
            else w[u][h][q].clear();
          }
        }
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          bf16x8 xt[X8<XT>::kTerms];
          x[u][h].terms(xt);
#pragma unroll
          for (int q = 0; q < RT; ++q) {
            bf16x8 wt[1];
            w[u][h][q].terms(wt);
#pragma unroll
            for (int t = X8<XT>::kTerms - 1; t >= 0; --t)
              acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xt[t], wt[0], acc[q], 0, 0, 0);
          }
        }
      }
    }
    __syncthreads();  // the last adapter's sums are read
#pragma unroll
    for (int q = 0; q < RT; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) sums[wave][(4 * j + i) * (RT * 16) + 16 * q + c] = acc[q][i];
    __syncthreads();
    const float sa = p.scale != nullptr ? p.scale[a] : 1.0f;
    for (int o = threadIdx.x; o < RT * 256; o += 64 * WV) {
      const int row = o / (RT * 16), r = r0 + o % (RT * 16);
      if (!(rows >> row & 1u) || r >= rank) continue;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < WV; ++w) v += sums[w][o];
      if constexpr (XT == kI8 || XT == kE4m3) v *= p.xscale[m0 + row];
      p.t[((int64_t)split * p.M + m0 + row) * p.R + r] = sa * v;
    }
  });
}

// t of this lane's token (if it is `mine`) and eight ranks from r8 on, of which `have` count, as operand terms.  The splits'
// parts are requested two at a time and added in order.
template <int T>
__device__ __forceinline__ void load_t(const LoraArgs& p, int64_t m, int r8, int have, bool mine, bf16x8 (&t)[T]) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  if (mine && have > 0) {
    const float* from = p.t + m * p.R + r8;
    for (int s0 = 0; s0 < p.splits; s0 += 2) {
      f32x4 x[2][2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const f32x4* tp = reinterpret_cast<const f32x4*>(from + (int64_t)(s0 + s < p.splits ? s0 + s : s0) * p.M * p.R);
        x[s][0] = tp[0], x[s][1] = tp[1];
      }
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s0 + s < p.splits)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += x[s][i / 4][i % 4];
    }
    if (have < 8)  // beyond the rank: zeros, whatever is stored there
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= have) v[i] = 0.0f;
  }
  split_terms<T>(v, t);
}

// Sixteen consecutive values of a row of base or Y, `have` of which are there.  (In units of 16 bytes, 64 apart, so that a
// token's four lanes read 64 bytes in a row, the prompt's kernel took 68 us against 64.)
template <bool YB, bool VEC>
struct Sixteen {
  static constexpr int kSize = YB ? 2 : 4, kWords = 4 * kSize;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const char* p, int have) {
    if (VEC && have >= 16) {
#pragma unroll
      for (int i = 0; i < kSize; ++i) {
        const u32x4 v = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
        for (int d = 0; d < 4; ++d) w[4 * i + d] = v[d];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if constexpr (YB) {
          const uint32_t v = i < have ? reinterpret_cast<const uint16_t*>(p)[i] : 0u;
          w[i / 2] = i % 2 ? w[i / 2] | v << 16 : v;
        } else {
          w[i] = i < have ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
        }
      }
    }
  }
  __device__ __forceinline__ void add(const f32x4 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float a = v[i / 4][i % 4], b = v[i / 4][i % 4 + 1];
      if constexpr (YB) w[i / 2] = pack_rne(flt(w[i / 2] << 16) + a, flt(w[i / 2] & 0xffff0000u) + b);
      else w[i] = bits(flt(w[i]) + a), w[i + 1] = bits(flt(w[i + 1]) + b);
    }
  }
  __device__ __forceinline__ void store(char* p, int have) const {
    if (VEC && have >= 16) {
#pragma unroll
      for (int i = 0; i < kSize; ++i)
        reinterpret_cast<u32x4*>(p)[i] = (u32x4){w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i < have) {
          if constexpr (YB) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(i % 2 ? w[i / 2] >> 16 : w[i / 2]);
          else reinterpret_cast<uint32_t*>(p)[i] = w[i];
        }
      }
    }
  }
};

// acc[q][i] += B t for the 64 channels from n0 on, over an adapter's ranks.  The channels are the left operand's rows, the
// tokens the right operand's columns: row r of tile q is channel 16 (r / 4) + 4 q + r % 4 of the 64, so that lane 16 j + c
// has channels 16 j + 4 q + i of token c.  t of the first 32 HELD ranks is held in registers.
template <int T, int HELD>
__device__ __forceinline__ void add_products(const LoraArgs& p, int a, int rank, int64_t n0, int64_t m, bool mine, int c, int j,
                                             const bf16x8 (&held)[HELD][T], f32x4 (&acc)[4]) {
  const int last = p.N - n0 < 64 ? (int)(p.N - n0) - 1 : 63;  // past the last channel: the last again, not stored
  const char* from = reinterpret_cast<const char*>(p.b + ((int64_t)a * p.N + n0) * p.R);
  int at[4];  // bytes from there: below 2^16
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int ch = 16 * (c / 4) + 4 * q + c % 4;
    at[q] = ((ch < last ? ch : last) * p.R + 8 * j) * 2;
  }
  auto ranks = [&](int r, const bf16x8 (&t)[T]) AWQ_INLINE {
    const int have = rank - r - 8 * j;  // of this lane's eight ranks
    X8<kBf16> w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (have > 0) w[q].load(from + 2 * r + at[q]);
      else w[q].clear();
    }
    if (rank & 7) {  // beyond the rank: zeros, whatever is stored there
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[q].w[i] &= 2 * i + 1 < have ? 0xffffffffu : 2 * i < have ? 0x0000ffffu : 0u;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      bf16x8 wt[1];
      w[q].terms(wt);
#pragma unroll
      for (int i = T - 1; i >= 0; --i) acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wt[0], t[i], acc[q], 0, 0, 0);
    }
  };
#pragma unroll
  for (int h = 0; h < HELD; ++h)
    if (32 * h < rank) ranks(32 * h, held[h]);
  for (int r = 32 * HELD; r < rank; r += 32) {
    bf16x8 t[T];
    load_t<T>(p, m, r + 8 * j, rank - r - 8 * j, mine, t);
    ranks(r, t);
  }
}

// Y = base + B t for sixteen tokens and 64 channels a wave; a tile's adapters go to `parts` blocks.
template <int T, bool YB, bool VEC, int HELD>
__global__ __launch_bounds__(256) void lora_up_kernel(const LoraArgs p, int parts) {
  const int lane = threadIdx.x & 63, j = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t across = (p.N + 255) / 256;
  const int64_t m0 = (int64_t)blockIdx.x / across * 16, n0 = ((int64_t)blockIdx.x % across * 4 + wave) * 64;
  if (n0 >= p.N) return;
  const int64_t m = m0 + c < p.M ? m0 + c : p.M - 1;
  using Values = Sixteen<YB, VEC>;
  const char* brow = static_cast<const char*>(p.base) + (m * p.ldb + n0 + 16 * j) * Values::kSize;
  char* yrow = static_cast<char*>(p.y) + (m * p.ldy + n0 + 16 * j) * Values::kSize;
  const int64_t there = p.N - n0 - 16 * j;  // channels from this lane's first on
  const int have = there < 64 ? (int)there : 64;
  const int id = row_adapter(p, m0, c);
  const bool copies = p.base != p.y;
  each_adapter(id, (int)blockIdx.y, parts, [&](int a, uint32_t rows) AWQ_INLINE {
    if (a == kNone && !copies) return;
    const bool mine = rows >> c & 1u;
    Values v;
    if (mine) v.load(brow, have);
    if (a != kNone) {
      const int rank = adapter_rank(p, a);
      bf16x8 held[HELD][T];
#pragma unroll
      for (int h = 0; h < HELD; ++h) load_t<T>(p, m, 32 * h + 8 * j, rank - 32 * h - 8 * j, mine, held[h]);
      f32x4 acc[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[q] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
      add_products<T, HELD>(p, a, rank, n0, m, mine, c, j, held, acc);
      if (mine) v.add(acc);
    }
    if (mine) v.store(yrow, have);
  });
}

// The same for prompts: sixteen tokens and 512 or 1024 channels a block, whose eight waves lay their products out in LDS, so
// that base and Y go by in whole runs of a row.  All of base is requested before anything else.  N is a multiple of a unit of
// 16 bytes, the rows start at multiples of them.  Two runs of 64 channels a wave where the registers leave two blocks on a
// CU.  us, both kernels, one run / two: 4096 x 4096 -> 14336 bf16, rank 16, 75 / 70; 777 x 5120 -> 11008 fp32, rank 32,
// 36 / 39; without LDS, each lane with its sixteen channels, 89 and 40.
constexpr int up_runs(bool bf16, int held) { return bf16 && held == 1 ? 2 : 1; }

template <int T, bool YB, int HELD>
__global__ __launch_bounds__(512) void lora_up_rows_kernel(const LoraArgs p) {
  constexpr int RUNS = up_runs(YB, HELD), C = 512 * RUNS;         // channels of a block
  constexpr int kSize = YB ? 2 : 4, kUnit = 16 / kSize;           // channels of 16 bytes
  constexpr int kTurns = 16 * C / kUnit / 512;                    // units of a thread
  static_assert(C / kUnit % 64 == 0, "a wave's units are one row's");
  constexpr int kRow = C + 4;                                     // sixteen rows' same 16 bytes: all banks
  __shared__ __attribute__((aligned(16))) float sums[16 * kRow];
  const int lane = threadIdx.x & 63, j = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t across = (p.N + C - 1) / C;
  const int64_t m0 = (int64_t)blockIdx.x / across * 16, b0 = (int64_t)blockIdx.x % across * C, n0 = b0 + 64 * RUNS * wave;
  u32x4 v[kTurns];
  auto place = [&](int i, int& row, int& ch) AWQ_INLINE {
    const int u = (int)threadIdx.x + 512 * i;
    row = u / (C / kUnit), ch = u % (C / kUnit) * kUnit;
    return m0 + row < p.M && b0 + ch < p.N;
  };
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    int row, ch;
    if (place(i, row, ch))
      v[i] = *reinterpret_cast<const u32x4*>(static_cast<const char*>(p.base) + ((m0 + row) * p.ldb + b0 + ch) * kSize);
  }
  const int64_t m = m0 + c < p.M ? m0 + c : p.M - 1;
  const int id = row_adapter(p, m0, c);
  if (n0 < p.N) {
    each_adapter(id, 0, 1, [&](int a, uint32_t rows) AWQ_INLINE {
      if (a == kNone) return;
      const bool mine = rows >> c & 1u;
      const int rank = adapter_rank(p, a);
      bf16x8 held[HELD][T];
#pragma unroll
      for (int h = 0; h < HELD; ++h) load_t<T>(p, m, 32 * h + 8 * j, rank - 32 * h - 8 * j, mine, held[h]);
#pragma unroll 1
      for (int k = 0; k < RUNS; ++k) {
        if (n0 + 64 * k >= p.N) break;
        f32x4 acc[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
        add_products<T, HELD>(p, a, rank, n0 + 64 * k, m, mine, c, j, held, acc);
        if (mine)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(sums + c * kRow + 64 * (RUNS * wave + k) + 16 * j + 4 * q) = acc[q];
      }
    });
  }
  __syncthreads();
  const bool copies = p.base != p.y;
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    int row, ch;
    const bool there = place(i, row, ch);
    const int a = __builtin_amdgcn_readlane(id, __builtin_amdgcn_readfirstlane(row));  // a wave's 64 units are one row's
    if (!there || (a == kNone && !copies)) continue;
    if (a != kNone) {
      const float* s = sums + row * kRow + ch;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        if constexpr (YB) v[i][d] = pack_rne(flt(v[i][d] << 16) + s[2 * d], flt(v[i][d] & 0xffff0000u) + s[2 * d + 1]);
        else v[i][d] = bits(flt(v[i][d]) + s[d]);
      }
    }
    *reinterpret_cast<u32x4*>(static_cast<char*>(p.y) + ((m0 + row) * p.ldy + b0 + ch) * kSize) = v[i];
  }
}

// Up to this many tokens a tile's distinct adapters go to blocks of their own (a decode batch: up to sixteen requests in a
// tile); beyond, one block takes them in turn (prompts: one or two requests in a tile).
constexpr int64_t kParallelTokens = 256;
int parts_of(int64_t M) { return M > kParallelTokens ? 1 : M < 16 ? (int)M : 16; }

template <int XT>
hipError_t launch_down(const LoraArgs& a, hipStream_t st) {
  const int parts = parts_of(a.M), tiles = (a.R + 15) / 16;
  const int rt = a.M > kParallelTokens ? (tiles >= 4 ? 4 : tiles >= 2 ? 2 : 1) : 1;
  const int rb = (tiles + rt - 1) / rt;
  const dim3 grid((unsigned)((a.M + 15) / 16), (unsigned)(parts * rb), (unsigned)a.splits);
  if (rt == 4) lora_down_kernel<XT, 4><<<grid, 512, 0, st>>>(a, parts, rb);
  else if (rt == 2) lora_down_kernel<XT, 2><<<grid, 512, 0, st>>>(a, parts, rb);
  else lora_down_kernel<XT, 1><<<grid, 512, 0, st>>>(a, parts, rb);
  return hipGetLastError();
}

template <int T, bool YB>
hipError_t launch_up(const LoraArgs& a, hipStream_t st) {
  const int64_t tiles = (a.M + 15) / 16;
  if (a.M > kParallelTokens && a.vec && a.N % (YB ? 8 : 4) == 0) {
    const int held = a.R <= 32 ? 1 : 2, C = 512 * up_runs(YB, held);
    const unsigned grid = (unsigned)((a.N + C - 1) / C * tiles);
    if (held == 1) lora_up_rows_kernel<T, YB, 1><<<grid, 512, 0, st>>>(a);
    else lora_up_rows_kernel<T, YB, 2><<<grid, 512, 0, st>>>(a);
    return hipGetLastError();
  }
  const int parts = parts_of(a.M);
  const dim3 grid((unsigned)((a.N + 255) / 256 * tiles), (unsigned)parts);
  if (!a.vec) lora_up_kernel<T, YB, false, 1><<<grid, 256, 0, st>>>(a, parts);
  else if (a.R <= 32) lora_up_kernel<T, YB, true, 1><<<grid, 256, 0, st>>>(a, parts);
  else lora_up_kernel<T, YB, true, 2><<<grid, 256, 0, st>>>(a, parts);
  return hipGetLastError();
}

}  // namespace

// Blocks that share K: about 512 in all, each with at least 512 channels for its eight waves; for many tokens at most
// four, because every wave of the second kernel reads all of them.
int lora_splits(int64_t M, int64_t K, int64_t R) {
  const int64_t tiles = (M + 15) / 16, ranks = (R + 15) / 16;
  const int64_t blocks = M > kParallelTokens ? tiles * ((ranks + 3) / 4) : tiles * (M < 16 ? M : 16) * ranks;
  int64_t s = (512 + blocks - 1) / blocks, most = M > kParallelTokens ? 4 : 16;
  if (most > K / 512) most = K / 512;
  if (s > most) s = most;
  return s < 1 ? 1 : (int)s;
}

hipError_t launch_lora(const LoraArgs& a, int x_type, hipStream_t st) {
  hipError_t e = x_type == kF32    ? launch_down<kF32>(a, st)
                 : x_type == kBf16 ? launch_down<kBf16>(a, st)
                 : x_type == kI8   ? launch_down<kI8>(a, st)
                                   : launch_down<kE4m3>(a, st);
  if (e != hipSuccess) return e;
  return a.ybf16 ? launch_up<2, true>(a, st) : launch_up<3, false>(a, st);
}

}  // namespace awq
