// The FP8 product with a scale per block of 128 for batches: the linear
// product's tiles (linear_tile.h) with the scales of each 128-column step in
// the ring, dense and over the row tiles of routed experts.  fp32 outputs, K
// split and small grids; longer batches: linear_block_big.hip and
// linear_block_stream.hip.
#include <algorithm>

#include "linear_block.h"
#include "linear_block_plan.h"
#include "linear_tile.h"

namespace moe {

bool block_tile_fits(const BlockParams& B) {
  // 32-bit offsets inside a tile's rows (grouped: over all of x) and over the weights' scales
  constexpr int64_t lim = 1 << 24;
  return B.L.ldx < lim && B.L.ldw < lim && B.L.ldr < lim && B.L.ldo < lim && (int64_t)B.nb * B.steps < (1 << 28);
}

namespace {

template <bool GATED, bool EXACT, bool GROUPED, int WM, int WN, int TM, int TN, int S>
void launch_one(const BlockParams& B, const TilePlan& pl, float* part, hipStream_t s) {
  constexpr int BM = WM * TM * 16, BO = WN * TN * 16 / (GATED ? 2 : 1);
  const LinParams& P = B.L;
  LinTiles G;
  G.mt = GROUPED ? 0 : (P.T + BM - 1) / BM;
  G.nt = (P.N + BO - 1) / BO;
  const int es = P.out_f32 ? 4 : 2;
  G.vec_out = ((uintptr_t)P.out & 15) == 0 && (P.ldo * es) % 16 == 0;
  G.vec_res = ((uintptr_t)P.res & 15) == 0 && P.ldr % 8 == 0;
  G.splits = pl.splits;
  G.per = pl.per;
  G.part = part;
  const long long mt = GROUPED ? most_row_blocks(P.T, B.E, BM) : G.mt;
  const long long grid = (mt * G.nt * G.splits + 7) / 8 * 8;
  launch(k_block_tile<GATED, EXACT, GROUPED, WM, WN, TM, TN, S>, dim3((unsigned)grid), dim3(64 * WM * WN), 0, s, B, G);
  if (!GROUPED && G.splits > 1)
    launch(k_linear_join<MOE_Q_NONE, GATED>, dim3((unsigned)(((int64_t)P.T * P.N + 255) / 256)), dim3(256), 0, s, P,
           part, G.splits);
}

template <bool GATED, bool EXACT, bool GROUPED>
void launch_shape(const BlockParams& B, const TilePlan& pl, float* part, hipStream_t s) {
  if constexpr (!GROUPED) {
    if (pl.shape == 4) return launch_one<GATED, EXACT, GROUPED, 2, 1, 2, 4, 3>(B, pl, part, s);
  }
  if (pl.shape == 2) launch_one<GATED, EXACT, GROUPED, 2, 2, 4, 4, 2>(B, pl, part, s);
  else launch_one<GATED, EXACT, GROUPED, 2, 2, 2, 4, 3>(B, pl, part, s);
}

template <bool GATED, bool GROUPED>
void launch_out(const BlockParams& B, const TilePlan& pl, float* part, hipStream_t s) {
  if (B.L.out_f32) launch_shape<GATED, true, GROUPED>(B, pl, part, s);
  else launch_shape<GATED, false, GROUPED>(B, pl, part, s);
}

}  // namespace

void launch_block_tile(const BlockParams& B, const TilePlan& pl, void* workspace, hipStream_t s) {
  float* part = static_cast<float*>(workspace);
  if (pl.shape == kBig) return launch_block_big(B, s);
  if (pl.shape == kStream) return launch_block_stream(B, s);
  if (B.offsets) B.L.gated ? launch_out<true, true>(B, pl, part, s) : launch_out<false, true>(B, pl, part, s);
  else B.L.gated ? launch_out<true, false>(B, pl, part, s) : launch_out<false, false>(B, pl, part, s);
}

}  // namespace moe
