// The linear product for batches: output tiles of BM tokens x BN weight rows
// (gfx950).
//
// K advances 128 bytes of every operand row a step.  A step's operands go
// from global memory straight to LDS (global_load_lds_dwordx4, one wave-wide
// load moves 8 rows x 128 bytes) into a ring of S stages; the 16-byte pieces
// of a row are permuted by bits 3:1 of the row so that a fragment's 16 rows
// fall into different banks.
//
// Bound: the matrix cores, at the rate the L2 fills the ring.  4096 tokens,
// against the time of a large library product at its 1.40 (bf16) and 3.09
// (FP8) PFLOP/s: 2048 x 2048 bf16 36 us (24.5; the library's own product of
// this size, without the epilogue, 34.1), 7168 x 2048 FP8 75 us (39; 62.6), 2
// x 2048 x 7168 MXFP8 with SwiGLU 92 us (78); cards and runs differ by 2 %,
// bf16 by 5.  Counters there: matrix cores busy 0.31, 0.29 and 0.53 of the
// cycles, texture unit 0.33, 0.40 and 0.44, LDS conflicts under 1 %; the L2s
// fetch 2.4, 1.9 and 3.0 times the bytes of x, w and residual.  The FP8 case
// is 448 tiles on 256 CUs, a second round three quarters full; 128-row tiles
// round better and load more bytes a product: 91 us.
//
// EXACT (fp32 outputs of E4M3): the FP8 instructions cut small products, so
// the codes are decoded to bf16: four matrix instructions and the decoding in
// the place of one (4096 x 7168 x 7168: 375 us against 174).
#include <algorithm>

#include "linear.h"
#include "linear_plan.h"
#include "linear_tile.h"

namespace moe {

bool linear_tile_fits(const LinParams& P) {
  // 32-bit offsets inside a tile's rows
  constexpr int64_t lim = 1 << 24;
  return P.ldx < lim && P.ldw < lim && P.ldr < lim && P.ldo < lim;
}

namespace {

template <int QM, bool GATED, bool EXACT, int WM, int WN, int TM, int TN, int S>
void launch_one(const LinParams& P, const TilePlan& pl, float* part, hipStream_t s) {
  constexpr int BM = WM * TM * 16, BO = WN * TN * 16 / (GATED ? 2 : 1);
  LinTiles G;
  G.mt = (P.T + BM - 1) / BM;
  G.nt = (P.N + BO - 1) / BO;
  const int es = P.out_f32 ? 4 : 2;
  G.vec_out = ((uintptr_t)P.out & 15) == 0 && (P.ldo * es) % 16 == 0;
  G.vec_res = ((uintptr_t)P.res & 15) == 0 && P.ldr % 8 == 0;
  G.splits = pl.splits;
  G.per = pl.per;
  G.part = part;
  const long long grid = ((long long)G.mt * G.nt * G.splits + 7) / 8 * 8;
  launch(k_linear_tile<QM, GATED, EXACT, WM, WN, TM, TN, S>, dim3((unsigned)grid), dim3(64 * WM * WN), 0, s, P, G);
  if (G.splits > 1)
    launch(k_linear_join<QM, GATED>, dim3((unsigned)(((int64_t)P.T * P.N + 255) / 256)), dim3(256), 0, s, P, part,
           G.splits);
}

template <int QM, bool GATED, bool EXACT>
void launch_shape(const LinParams& P, float* part, hipStream_t s) {
  const TilePlan pl = plan_tiles(P.T, P.R, P.kb, EXACT);
  if constexpr (!EXACT) {
    if (pl.shape == 0) return launch_one<QM, GATED, EXACT, 2, 4, 8, 4, 2>(P, pl, part, s);
  }
  if (pl.shape == 1) launch_one<QM, GATED, EXACT, 2, 4, 4, 4, 3>(P, pl, part, s);
  else if (pl.shape == 2) launch_one<QM, GATED, EXACT, 2, 2, 4, 4, 2>(P, pl, part, s);
  else if (pl.shape == 3) launch_one<QM, GATED, EXACT, 2, 2, 2, 4, 3>(P, pl, part, s);
  else launch_one<QM, GATED, EXACT, 2, 1, 2, 4, 3>(P, pl, part, s);
}

template <int QM, bool EXACT>
void launch_gate(const LinParams& P, float* part, hipStream_t s) {
  if (P.gated) launch_shape<QM, true, EXACT>(P, part, s);
  else launch_shape<QM, false, EXACT>(P, part, s);
}

}  // namespace

size_t linear_tile_workspace(int T, int R, int kb, bool exact) {
  const TilePlan pl = plan_tiles(T, R, kb, exact);
  return pl.splits > 1 ? (size_t)pl.splits * T * R * sizeof(float) : 0;
}

void launch_linear_tile(const LinParams& P, int qm, void* workspace, hipStream_t s) {
  float* part = static_cast<float*>(workspace);
  if (qm == MOE_Q_NONE) launch_gate<MOE_Q_NONE, false>(P, part, s);
  else if (qm == MOE_Q_FP8 && P.out_f32) launch_gate<MOE_Q_FP8, true>(P, part, s);
  else if (qm == MOE_Q_FP8) launch_gate<MOE_Q_FP8, false>(P, part, s);
  else if (P.out_f32) launch_gate<MOE_Q_MXFP8, true>(P, part, s);
  else launch_gate<MOE_Q_MXFP8, false>(P, part, s);
}

}  // namespace moe
