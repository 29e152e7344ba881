// Which kernel and tile shape a block-scaled product takes (host only: a CPU
// test compiles this file alone and checks that the GPU tests reach every
// shape).
#pragma once
#include <algorithm>
#include <cstdint>

#include "linear_plan.h"

namespace moe {

constexpr int kStreamTiles = 128;  // tiles a workgroup of k_block_stream holds
// Shapes beside kShapes[2 ..], which k_block_tile takes.
constexpr int kBig = 0;     // k_block_big
constexpr int kStream = 5;  // k_block_stream

// Whether k_block_small takes the dense call.
inline bool block_small_wins(int T, int R, bool gated, int K, bool exact) { return small_wins(T, R, gated, K, exact); }

// 256 x 256 tiles where they fill the chip, else the shapes of the linear
// product from 128 x 128 on, K split where that helps.  128 x 128 tiles that
// pass two a CU are walked without a pause.  us, 256 x 256, walked, 128 x 128:
// 4096 x 4096 x 7168 102, 121, 126; 4096 x 7168 x 2048 64, 66, 72; 1024 x 4096
// x 2048 29, 15.6, 16.4.  fp32 outputs (exact): k_block_tile alone.
inline TilePlan plan_block_tiles(int T, int N, bool gated, int K, bool exact) {
  const int R = gated ? 2 * N : N, steps = K / 128;
  const int64_t big = (int64_t)((T + 255) / 256) * (gated ? (N + 127) / 128 : (N + 255) / 256);
  if (!exact && big >= 192) return TilePlan{kBig, 1, steps};
  TilePlan pl = plan_tiles(T, R, K, exact);
  pl.shape = std::max(pl.shape, 2);
  const int64_t tiles = (int64_t)((T + 127) / 128) * (gated ? (N + 63) / 64 : (N + 127) / 128);
  if (!exact && steps >= 2 && tiles > 2 * kCus && tiles <= (int64_t)2 * kCus * kStreamTiles) return TilePlan{kStream, 1, steps};
  return pl;
}

// Most row blocks of bm rows that T rows of E experts can make.
inline int64_t most_row_blocks(int T, int E, int bm) {
  const int64_t used = T < E ? T : E;
  return used + (T - used) / bm;
}

// Grouped: k_block_small while the experts have a row or two each.  us against
// the better of the tiles, 128 experts of 2 x 768 x 2048: 64 rows 22.0 to 22.8,
// 128 33.4 to 37.6, 512 61.2 to 62.2; of 2048 x 768: 128 23.3 to 22.3, 512
// 44.1 to 40.3; 32 experts of 2 x 1024 x 7168: 32 rows 49 to 62.
inline bool grouped_small_wins(int T, int E) { return T <= 2 * E; }

// Else tiles walked without a pause: where the experts start and end is known
// on the device alone, and each tile's look for its own place, its first loads
// and its epilogue would stand still a CU's half.  us, 4096 tokens by 8 of 128
// experts: 2 x 768 x 2048 180 against 207 with a workgroup a tile, 2048 x 768
// 112 against 149; 512 tokens, 2 x 768 x 2048 93 against 97 (64 x 128 tiles).
// Up to 8 rows an expert 64 x 128 tiles, which are more: 128 tokens 77 against
// 82, 32 tokens 55 against 58, 64 tokens by 8 of 32 experts 24 against 28.
// most: the most row blocks of 128 there can be.
inline TilePlan plan_grouped_tiles(int T, int E, int N, bool gated, int K, bool exact, int64_t most) {
  const int steps = K / 128;
  const int64_t tiles = most * (gated ? (N + 63) / 64 : (N + 127) / 128);
  if (!exact && T > 8 * E && steps >= 2 && tiles <= (int64_t)2 * kCus * kStreamTiles) return TilePlan{kStream, 1, steps};
  return TilePlan{T / E >= 48 ? 2 : 3, 1, steps};
}

// Waves of a grouped k_block_small workgroup: there are workgroups enough, and the small ones end and start
// soonest.  us with 4, 8, 16 waves: 128 rows of 128 experts of 2 x 768 x 2048 33.4, 42.0, 53.1; 8 of 32 of 2 x
// 1024 x 7168 27.1, 25.6, 25.0; 32 of 128 of 2 x 1024 x 4096 35.8, 34.4, 41.0.
inline int grouped_small_waves(int K) { return K / 128 >= 32 ? 8 : 4; }

// Threads of the grid that a grouped call launches; a grid holds fewer than
// 2^32.  fits: the call's strides fit the tiles.
inline int64_t grouped_threads(int T, int E, int N, bool gated, int K, bool exact, bool fits) {
  if (!fits || grouped_small_wins(T, E))
    return most_row_blocks(T, E, 16) * ((N + 15) / 16) * 64 * grouped_small_waves(K);
  const TilePlan pl = plan_grouped_tiles(T, E, N, gated, K, exact, most_row_blocks(T, E, 128));
  if (pl.shape == kStream) return (int64_t)2 * kCus * 256;
  const int bo = kShapes[pl.shape].bn / (gated ? 2 : 1);
  return (most_row_blocks(T, E, kShapes[pl.shape].bm) * ((N + bo - 1) / bo) + 7) / 8 * 8 * 256;
}

}  // namespace moe
