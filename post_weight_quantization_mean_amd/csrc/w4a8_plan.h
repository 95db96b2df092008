// How a W4A8 product runs, by its sizes alone (so that the workspace's size can be told before).  Host code without
// HIP: which kernel a size takes can be asked from a plain C++ program.
#pragma once

#include <cstdint>

namespace awq {

constexpr int kW4a8Group = 128;  // channels of a group
constexpr int kTileN = 256;      // channels of a tile (split, tile)
constexpr int64_t w4a8_tiles(int64_t N) { return (N + 15) / 16; }
constexpr int64_t padded_groups(int64_t K) { return (K / kW4a8Group + 7) / 8 * 8; }

constexpr int kStream = 0, kSplit = 1, kTile = 2;
struct Plan {
  int path;
  int tm;                 // token tiles of 16 per block
  int splits, per_split;  // split: blocks and groups per tile
  int ct, waves;          // stream: channel tiles of 16 and waves per block
};

// How a product of e4m3 codes is summed: true, by the matrix unit (14 bits of the largest of sixteen products),
// false, in fp32.  Left to the kernel, bf16 results of more than 256 tokens take the matrix unit's sums, because there
// the matrix rate counts, which fp32 sums halve; a rule on the tokens, not on the plan's path, so that a re-fitted cost
// changes no result.  us, matrix unit / fp32: 4096 x 4096 -> 28672 435 / 845, 1024 x 11008 -> 4096 60 / 104, 512 x 4096
// -> 4096 17 / 26; up to 256 tokens, 1 x 4096 -> 28672 12.7 / 16.5, 16 x 14336 -> 4096 10.7 / 11.3, 64 x 4096 -> 4096
// 7.0 / 7.3, 101 x 4096 -> 6144 13.0 / 14.6, 256 x 14336 -> 4096 32 / 42, 128 x 4096 -> 17000 29 / 44.
constexpr int kSumsDefault = 0, kSumsF32 = 1, kSumsMatrix = 2;
constexpr bool matrix_sums(int sums, bool ybf16, int64_t M) {
  return sums == kSumsMatrix || (sums == kSumsDefault && ybf16 && M > 256);
}

// Blocks of 32 tokens and ct channel tiles: the fewest channels that leave at most one block of eight waves per CU
// (more channels read X less often, fewer blocks leave CUs idle); then blocks of four waves, several per CU.
// K = 4096, us: 192 blocks of 2 tiles 7.5, 256 of 3 8.4, 256 of 4 8.9; 512 of 3 in four waves 13.3 (384 of 4 14.6,
// 768 of 2 in eight 15.9); 448 of 4 in four waves 16.5 (in eight 17.9; 896 of 2 21.3).  Beyond 512 blocks the split
// path is as fast or faster (64 x 4096 -> 28672: 30.4 / 26.0; 129 x 8192 -> 8192: 38.2 / 33.9).
struct StreamShape {
  int ct, waves;
  float us;  // estimated
};
inline StreamShape stream_shape(int64_t M, int64_t G, int64_t tiles) {
  const int64_t rows = (M + 31) / 32;
  auto blocks = [&](int ct) { return (tiles + ct - 1) / ct * rows; };
  const float g = (float)G;
  if (blocks(2) <= 256) return {2, 8, 3.2f + (0.053f + 0.0025f * (float)(M < 32 ? M : 32)) * g};
  if (blocks(3) <= 256) return {3, 8, 3.2f + 0.163f * g};
  if (blocks(4) <= 256) return {4, 8, 3.2f + 0.175f * g};
  if (blocks(3) <= 512) return {3, 4, 3.2f + 0.316f * g};
  const float b = (float)blocks(4);
  return {4, 4, 3.2f + 0.356f * g * (b <= 384.0f ? 1.0f : b <= 512.0f ? b / 384.0f : b / 307.0f)};
}

// The costs are microseconds fitted to measurements (K = 4096 and 14336, N = 4096 to 28672, 17 to 640 tokens, weights
// from memory), for the ratio of two paths rather than for themselves: a tile's 0.95 a group is int8's at K = 4096; at
// K = 11008 int8 takes 0.84, and e4m3 with a bf16 result 0.70 at either, where the streams' estimates are high as much.
// Stream against tile at their crossovers, us (int8; e4m3 -> bf16): 65 x 4096 -> 16641 26 / 32; 26 / 31 (stream taken),
// 96 x 4096 -> 17000 30 / 32; 29 / 28 (stream), 65 x 11008 -> 17000 69 / 75; 68 / 65 (stream), 129 x 4096 -> 12288
// 27 / 31; 27 / 26 (tile), 128 x 4096 -> 17000 39 / 33; 38 / 29 (tile), 192 x 4096 -> 12288 37 / 31; 38 / 26 (tile).
inline Plan w4a8_plan(int64_t M, int64_t K, int64_t N) {
  const int64_t G = K / kW4a8Group, nt = (N + kTileN - 1) / kTileN;
  const int64_t tiles16 = w4a8_tiles(N);
  // up to 16 tokens: two channel tiles per block halve the reads of X where that still leaves more blocks than CUs
  // (16 tokens x 4096 -> 28672: 15.0 us against 20.4; 5 x 14336 -> 4096: 10.6 against 8.8)
  if (M <= 16) return tiles16 >= 320 ? Plan{kStream, 1, 1, (int)G, 2, 8} : Plan{kStream, 1, 1, (int)G, 1, 16};
  Plan pl{kStream, 1, 1, (int)G, 0, 0};
  const int64_t t64 = (M + 63) / 64 * nt, t128 = (M + 127) / 128 * nt;
  float best;
  if (t64 > 128) {
    // Tiles.  128-token tiles do a token's work in 0.77 of the time but leave whole rounds of 512 blocks (two per
    // CU) emptier: they run where the last round is five sixths full or there are many (K = 4096, e4m3, us,
    // 64- against 128-token tiles: 448 of the latter 73 / 68, 384 66 / 68, 560 98 / 103, 896 135 / 132).
    pl.path = kTile;
    pl.tm = t128 >= 1024 || t128 * 6 >= (t128 + 511) / 512 * 512 * 5 ? 8 : 4;
    best = 3.0f + 0.95f * (float)G * (t64 <= 256 ? 1.0f : 1.4f * (float)t64 / 512.0f);
  } else {
    // Few tiles: split.  Per two groups of a block 1.18 (32-token tiles) or 1.86 (64); with more than one split the
    // second kernel, and the parts written and read at 4 TB/s.  (101 x 4096 -> 6144: 18.4 us with 32-token tiles and
    // two splits, 21.6 with 64 and five; 256 x 14336 -> 4096: 40.0 and two, 34.4 and four.  At more than 128
    // 64-token tiles a split is one block per tile and loses to the tile kernel's two per CU: 41 / 33 at 224.)
    pl.path = kSplit;
    pl.tm = 0;
    best = 0.0f;
    for (int tm = 2; tm <= (M <= 32 ? 2 : 4); tm += 2) {
      const int64_t tiles = (M + 16 * tm - 1) / (16 * tm) * nt;
      int64_t most = 256 / tiles;
      if (most > G / 2) most = G / 2;
      if (most < 1) most = 1;
      for (int64_t want = most; want >= 1; want /= 2) {
        const int64_t per = (G + want - 1) / want, splits = (G + per - 1) / per;
        float us = 5.0f + (float)((per + 1) / 2) * (tm == 2 ? 1.18f : 1.86f);
        if (splits > 1) us += 2.5f + (float)(splits * M * N) * 2e-6f;
        if (pl.tm == 0 || us < best) {
          best = us;
          pl.tm = tm;
          pl.per_split = (int)per;
          pl.splits = (int)splits;
        }
      }
    }
  }
  if (M <= 256) {
    const StreamShape s = stream_shape(M, G, tiles16);
    if (s.us < best) return Plan{kStream, 2, 1, (int)G, s.ct, s.waves};
  }
  return pl;
}

}  // namespace awq
