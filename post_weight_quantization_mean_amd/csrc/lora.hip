// Low-rank adapters of many requests beside a shared projection:
//   Y[m] = base[m] + s_a B_a (A_a x[m]),  a = ids[m]
// in two kernels, t = s_a A_a x and Y = base + B_a t, on the bf16 matrix cores.  Tokens are taken sixteen at a time, as
// they stand: a tile's distinct adapters are found with a few ballots, each is multiplied with all sixteen rows, and
// only the rows that are its own are kept.  Nothing is sorted, and the rows of other adapters cost no memory traffic.
#include "lora_internal.h"
#include "x_operand.h"

namespace awq {
namespace {

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
// sixteen ranks, its eight waves taking steps of 32 channels in turn.
template <int XT, int RT>
__global__ __launch_bounds__(512) void lora_down_kernel(const LoraArgs p, int parts, int rank_blocks) {
  constexpr int WV = 8, U = XT == kF32 ? 2 : 4;
  __shared__ float sums[WV][RT * 256];
  const int lane = threadIdx.x & 63, j = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)blockIdx.x * 16;
  const int part = (int)blockIdx.y / rank_blocks, r0 = ((int)blockIdx.y % rank_blocks) * RT * 16;
  const int split = (int)blockIdx.z;
  const int id = row_adapter(p, m0, c);
  const int xs = XT == kF32 ? 4 : XT == kBf16 ? 2 : 1;
  const char* xrow = static_cast<const char*>(p.x) + ((m0 + c < p.M ? m0 + c : p.M - 1) * p.ldx + 8 * j) * xs;
  const int64_t steps = (p.K + 31) / 32;
  each_adapter(id, part, parts, [&](int a, uint32_t rows) {
    if (a == kNone) return;
    const int rank = adapter_rank(p, a);
    if (r0 >= rank) return;
    const uint16_t* arow[RT];
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      const int r = r0 + 16 * q + c < rank ? r0 + 16 * q + c : rank - 1;  // past the rank: its last row again, not kept
      arow[q] = p.a + ((int64_t)a * p.R + r) * p.K + 8 * j;
    }
    f32x4 acc[RT];
#pragma unroll
    for (int q = 0; q < RT; ++q) acc[q] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t s = (int64_t)split * WV + wave; s < steps; s += (int64_t)U * WV * p.splits) {
      X8<XT> x[U];
      X8<kBf16> w[U][RT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t k = 32 * (s + (int64_t)u * WV * p.splits);
        if (k + 8 * j < p.K) {
          x[u].load(xrow + k * xs);
#pragma unroll
          for (int q = 0; q < RT; ++q) w[u][q].load(reinterpret_cast<const char*>(arow[q] + k));
        } else {
          x[u].clear();
#pragma unroll
          for (int q = 0; q < RT; ++q) w[u][q].clear();
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        bf16x8 xt[X8<XT>::kTerms];
        x[u].terms(xt);
#pragma unroll
        for (int q = 0; q < RT; ++q) {
          bf16x8 wt[1];
          w[u][q].terms(wt);
#pragma unroll
          for (int t = X8<XT>::kTerms - 1; t >= 0; --t)
            acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xt[t], wt[0], acc[q], 0, 0, 0);
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

// Y = base + B t for sixteen tokens and 64 channels a wave.  The channels are the left operand's rows: row r of tile q is
// channel 16 (r / 4) + 4 q + r % 4 of the 64, so that a lane holds sixteen consecutive channels of its token.
template <int T, bool YB, bool VEC>
__global__ __launch_bounds__(256) void lora_up_kernel(const LoraArgs p, int parts) {
  const int lane = threadIdx.x & 63, j = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t chunks = (p.N + 255) / 256;
  const int64_t m0 = (int64_t)blockIdx.x / chunks * 16, n0 = ((int64_t)blockIdx.x % chunks * 4 + wave) * 64;
  if (n0 >= p.N) return;
  const int id = row_adapter(p, m0, c);
  const int64_t m = m0 + c < p.M ? m0 + c : p.M - 1;
  const int64_t n = n0 + 16 * j;  // this lane's first channel
  constexpr int YS = YB ? 2 : 4;
  const char* brow = static_cast<const char*>(p.base) + (m * p.ldb + n) * YS;
  char* yrow = static_cast<char*>(p.y) + (m * p.ldy + n) * YS;
  const bool copies = p.base != p.y;
  each_adapter(id, (int)blockIdx.y, parts, [&](int a, uint32_t rows) {
    if (a == kNone && !copies) return;
    const bool mine = rows >> c & 1u;
    const int count = n >= p.N ? 0 : p.N - n < 16 ? (int)(p.N - n) : 16;
    uint32_t raw[4 * YS];  // the sixteen values of base
    if (VEC && count == 16) {
      if (mine) {
#pragma unroll
        for (int i = 0; i < YS; ++i) {
          const u32x4 v = reinterpret_cast<const u32x4*>(brow)[i];
#pragma unroll
          for (int d = 0; d < 4; ++d) raw[4 * i + d] = v[d];
        }
      }
    } else if (mine) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if constexpr (YB) {
          const uint32_t v = i < count ? reinterpret_cast<const uint16_t*>(brow)[i] : 0u;
          raw[i / 2] = i % 2 ? raw[i / 2] | v << 16 : v;
        } else {
          raw[i] = i < count ? reinterpret_cast<const uint32_t*>(brow)[i] : 0u;
        }
      }
    }
    f32x4 acc[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    const int rank = a == kNone ? 0 : adapter_rank(p, a);
    for (int r = 0; r < rank; r += 32) {
      const int r8 = r + 8 * j, have = rank - r8;  // this lane's eight ranks, and how many of them there are
      float tv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) tv[i] = 0.0f;
      X8<kBf16> w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q].clear();
      if (have > 0) {
        if (mine) {
          for (int s = 0; s < p.splits; ++s) {
            const f32x4* tp = reinterpret_cast<const f32x4*>(p.t + ((int64_t)s * p.M + m) * p.R + r8);
            const f32x4 lo = tp[0], hi = tp[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) tv[i] += lo[i], tv[4 + i] += hi[i];
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int64_t ch = n0 + 16 * (c / 4) + 4 * q + c % 4;
          w[q].load(reinterpret_cast<const char*>(p.b + ((int64_t)a * p.N + (ch < p.N ? ch : p.N - 1)) * p.R + r8));
        }
        if (have < 8) {  // beyond the rank: zeros, whatever is stored there
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (i >= have) tv[i] = 0.0f;
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[q].w[i] &= 2 * i + 1 < have ? 0xffffffffu : 2 * i < have ? 0x0000ffffu : 0u;
        }
      }
      bf16x8 tt[T];
      split_terms<T>(tv, tt);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        bf16x8 wt[1];
        w[q].terms(wt);
#pragma unroll
        for (int t = T - 1; t >= 0; --t)
          acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wt[0], tt[t], acc[q], 0, 0, 0);
      }
    }
    if (!mine) return;
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float b = YB ? flt(i % 2 ? raw[i / 2] & 0xffff0000u : raw[i / 2] << 16) : flt(raw[i]);
      v[i] = a == kNone ? b : b + acc[i / 4][i % 4];
    }
    if constexpr (YB) {
#pragma unroll
      for (int i = 0; i < 8; ++i) raw[i] = pack_rne(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) raw[i] = bits(v[i]);
    }
    if (VEC && count == 16) {
#pragma unroll
      for (int i = 0; i < YS; ++i)
        reinterpret_cast<u32x4*>(yrow)[i] = (u32x4){raw[4 * i], raw[4 * i + 1], raw[4 * i + 2], raw[4 * i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i < count) {
          if constexpr (YB) reinterpret_cast<uint16_t*>(yrow)[i] = (uint16_t)(i % 2 ? raw[i / 2] >> 16 : raw[i / 2]);
          else reinterpret_cast<uint32_t*>(yrow)[i] = raw[i];
        }
      }
    }
  });
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
  const int parts = parts_of(a.M);
  const dim3 grid((unsigned)((a.N + 255) / 256 * ((a.M + 15) / 16)), (unsigned)parts);
  if (a.vec) lora_up_kernel<T, YB, true><<<grid, 256, 0, st>>>(a, parts);
  else lora_up_kernel<T, YB, false><<<grid, 256, 0, st>>>(a, parts);
  return hipGetLastError();
}

}  // namespace

// Blocks that share K, so that few tokens still fill the card: each has at least 512 channels for its eight waves.
int lora_splits(int64_t M, int64_t K, int64_t R) {
  const int64_t blocks = (M + 15) / 16 * (M < 16 ? M : 16) * ((R + 15) / 16);
  int64_t s = 32 / blocks;
  if (s > K / 512) s = K / 512;
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
