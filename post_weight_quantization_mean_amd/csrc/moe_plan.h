// How the experts' products run, by their sizes alone.  Host code without HIP: it can be asked from a plain C++ program.
#pragma once

#include <cstdint>

namespace awq {

// Ten tokens an expert and more run in tiles of 64 (32), fewer stream past sixteen at a time: from there on, with experts
// chosen evenly, some expert has more than sixteen.  us, stream / tiles: 64 experts of 2048 x 1024, 8 tokens each 58 / 71, 10
// 87 / 76, 12 99 / 82, 16 103 / 85, 31 157 / 103; 16 of 4096 x 4096, 8 104 / 119, 12 142 / 121; 8 of 4096 x 14336, 8 167 /
// 237, 12 229 / 268, 16 297 / 297; in fp32 (X and Y) 64 of 2048 x 2048, 8 149 / 174, 10 258 / 208; 16 of 4096 x 4096, 8 217 /
// 167, 10 290 / 191, 16 381 / 265; 16 of 1280 x 896, too few tiles for the card, 9 28 / 35, 12 29 / 35.
// All M k pairs count, also those whose expert is on another device, which the host cannot tell: with an eighth of the
// experts here tiles begin at one or two tokens for each of them (8 of 64 experts of 2048 x 1024, k 8: 8 tokens stream in 21,
// 10 take 28 in tiles).  Nor does the rule ask whether the tiles fill the card: few small experts would stream faster also
// beyond (4 of 2048 x 1024, 10 tokens each 15 / 30, 32 each 27 / 45; 8 of 2048 x 1408, 16 each 32 / 42).
inline bool in_tiles(int64_t M, int k, int E) { return M * k >= 10 * E; }

// Blocks for an expert's token tiles: half as many again as it has on average, at most eight; they take more in turn.
inline unsigned tile_depth(int M, int k, int E, int tokens) {
  const int depth = M * k * 3 / (2 * E * tokens) + 1;
  return (unsigned)(depth < 8 ? depth : 8);
}

// Units of a block's run in the stream kernels: blocks of `waves` waves for one round of the card's 256 CUs, a CU taking four
// times per_simd waves (a kernel's waves on a SIMD), and one block at least: sixteen waves are a CU's own also where the
// kernel is built for two a SIMD.  (37 fp32 tokens, 16 experts of 1280 x 896: 26.8 us, 31.4 in two rounds; 4 tokens, 8 of 128
// experts, 30.9, with twice the blocks 37.3; 2 fp32 tokens, 4 of 16 experts of 4096 x 4096, 85, with half the blocks 146.)
inline int units_per_block(int slots, int units, int waves, int per_simd) {
  const int on_cu = 4 * per_simd / waves, total = 256 * (on_cu > 1 ? on_cu : 1), blocks = (total + slots - 1) / slots;
  const int per = (units + blocks - 1) / blocks;
  return per < 1 ? 1 : per;
}

}  // namespace awq
