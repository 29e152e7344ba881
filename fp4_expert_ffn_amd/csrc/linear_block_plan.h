// Which kernel and tile shape a block-scaled product takes (host only: a CPU
// test compiles this file alone and checks that the GPU tests reach every
// shape).
#pragma once
#include <algorithm>
#include <cstdint>

#include "linear_plan.h"

namespace moe {

// Whether k_block_small takes the dense call.
inline bool block_small_wins(int T, int R, bool gated, int K, bool exact) { return small_wins(T, R, gated, K, exact); }

// Tiles of 256 x 256 where they fill the chip, else of 128 x 128, two a CU
// (4096 x 4096 x 7168: 100 against 121 us; 4096 x 7168 x 2048 67 against 72; 1024 x 4096 x 2048 29
// against 16).
inline TilePlan plan_block_tiles(int T, int R, int K, bool exact) {
  const long long big = (long long)((T + 255) / 256) * ((R + 255) / 256);
  if (!exact && big >= 192) return TilePlan{0, 1, K / 128};
  TilePlan pl = plan_tiles(T, R, K, exact);
  if (pl.shape < 2) pl.shape = 2;
  return pl;
}

// Grouped: rows a workgroup by the mean number of an expert's rows.
inline bool grouped_small_wins(int T, int E) { return T <= 16 * E; }

inline TilePlan plan_grouped_tiles(int T, int E, int K, bool exact) {
  const int mean = T / E, steps = K / 128;
  const int shape = mean >= 32 ? 2 : 3;
  return TilePlan{shape, 1, steps};
}

}  // namespace moe
