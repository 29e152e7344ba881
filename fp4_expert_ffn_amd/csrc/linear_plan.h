// Which kernel and tile shape a linear product takes (host only: a CPU test
// compiles this file alone and checks that the GPU tests reach every shape).
#pragma once
#include <algorithm>
#include <cstdint>

namespace moe {

constexpr int kSmallMaxT = 16;  // longer batches: the tile kernel

// us of a call by what a CU loads: 2 + a workgroup's KB (weights 0.032, x
// 0.02) for each workgroup in turn; rows: weight rows a workgroup.
inline float few_cost(int T, int N, int kb, int cols, int rows) {
  const int turns = (N + cols * 256 - 1) / (cols * 256);
  return 2.f + (float)kb * 1e-3f * ((float)rows * 0.032f + (float)T * 0.02f) * (float)turns;
}

inline bool eight_columns(int T, int N, int kb) { return few_cost(T, N, kb, 8, 16) < few_cost(T, N, kb, 16, 32); }

// Whether k_linear_small takes the call.  It is bound by what one CU can load
// (every workgroup reads its whole weight rows and all of x), the tile kernel
// with its split K by launches and HBM: about 7.3 us + bytes at 8 TB/s.  Both
// estimates are fit to 1 to 17 tokens of 256 to 7168 rows of 2 to 14 KB.  One
// token, bf16: 4096 x 4096 8.3 against 11.8 us; 16 tokens: 7168 x 2048 10.4
// against 10.6, 7168 x 7168 27.3 against 20.1.  Decoded E4M3 (fp32 outputs)
// costs the tiles more: 2048 x 2048 4.0 against 12.9, 7168 x 7168 15.8 against
// 15.7.
inline bool small_wins(int T, int R, bool gated, int kb, bool exact) {
  if (T > kSmallMaxT) return false;
  if (exact) return true;
  const float few = gated ? std::min(few_cost(T, R / 2, kb, 8, 16), few_cost(T, R / 2, kb, 16, 32))
                          : few_cost(T, R, kb, 16, 16);
  return few <= 7.3f + (float)R * (float)kb * 1.25e-7f;
}

// The tile shapes and what a call of one costs, in us: a step of a tile on a
// CU, and the rest of a call (launch, first loads, epilogue).  Measured with
// one or two tiles a CU over 16 to 112 steps (bf16, FP8 and MXFP8 alike: a
// step is 128 bytes of a row in each).
struct TileShape {
  int bm, bn;
  float step, rest;
};
constexpr TileShape kShapes[] = {{256, 256, 1.25f, 10.f}, {128, 256, 0.73f, 6.f}, {128, 128, 0.47f, 5.f},
                                 {64, 128, 0.32f, 4.5f},  {64, 64, 0.25f, 4.f}};
constexpr int kCus = 256;

struct TilePlan {
  int shape, splits, per;
};

// The shape and the split of K with the least estimated time: tiles in
// rounds of one a CU; a split costs the join's launch and the sums' way
// through memory.
inline TilePlan plan_tiles(int T, int R, int kb, bool exact) {
  const int steps = (kb + 127) / 128;
  TilePlan best{4, 1, steps};
  float least = 1e30f;
  for (int i = exact ? 1 : 0; i < 5; ++i) {
    const TileShape& h = kShapes[i];
    const int64_t tiles = (int64_t)((T + h.bm - 1) / h.bm) * ((R + h.bn - 1) / h.bn);
    for (int sp = 1; sp <= (i == 0 ? 1 : 16) && (sp == 1 || steps >= 4 * sp); ++sp) {
      const int per = (steps + sp - 1) / sp;
      if ((steps + per - 1) / per != sp) continue;  // an empty run
      const float rounds = (float)((tiles * sp + kCus - 1) / kCus);
      const float t = rounds * (per * h.step + (rounds > 1.f ? 0.5f * h.rest : 0.f)) + h.rest +
                      (sp > 1 ? 3.5f + (float)sp * T * R * 8e-6f / 4.f : 0.f);
      if (t < least) {
        least = t;
        best = TilePlan{i, sp, per};
      }
    }
  }
  return best;
}

}  // namespace moe
