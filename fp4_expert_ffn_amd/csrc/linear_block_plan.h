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

inline TilePlan plan_block_tiles(int T, int R, int K, bool exact) { return plan_tiles(T, R, K, exact); }

// Grouped: rows a workgroup by the mean number of an expert's rows.
inline bool grouped_small_wins(int T, int E) { return T <= 16 * E; }

inline TilePlan plan_grouped_tiles(int T, int E, int K, bool exact) {
  const int mean = T / E, steps = K / 128;
  const int shape = mean >= 512 && !exact ? 0 : (mean >= 96 ? 1 : 3);
  return TilePlan{shape, 1, steps};
}

}  // namespace moe
