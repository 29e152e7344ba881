// The product of E4M3 rows with a scale per 128 columns and weights with a
// scale per 128 x 128 block (gfx950), dense and grouped over routed experts:
//
//   y[t,n] = sum_b xs[b][t] ws[n / 128][b] sum_{c in block b} x[t,c] w[n,c]
//
// with the linear product's epilogue.  A block of 128 columns is one FP8
// matrix step from a zero accumulator; its sums are added to the running ones
// in fp32, times the product of the two scales.
#include <algorithm>

#include "linear_block.h"
#include "linear_block_plan.h"

namespace {

using namespace moe;

// Few rows: a stream of the weights, as k_linear_small.  One workgroup: NC
// columns (gated: their gate and up rows) x 16 rows of one expert (of the
// batch); its NWV waves take runs of kU K-steps in turn and load a run at
// once: long runs where a wave has one, short ones, and so more waves a CU,
// where there are many workgroups (16 tokens by 8 of 128 experts, 2048 x 768,
// 21.8 us against 32.7 with runs of 4) or where two fragments of weights a step
// leave no registers beside 16 waves.
// Bound: HBM, or where few workgroups fill the call one memory latency.  1 x
// (2 x 2048) x 7168 6.8 us, 4.3 TB/s; 8 experts of it 42, 5.6 TB/s; 16 x 7168
// x 2048 6.2.
constexpr int small_run(bool grouped, int fragments) { return grouped || fragments == 2 ? 2 : 4; }

template <bool GATED, bool EXACT, bool GROUPED, int NC, int NWV>
__global__ __launch_bounds__(64 * NWV) void k_block_small(BlockParams B, int n_tiles) {
  static_assert(NC == 16 || (NC == 8 && GATED), "whole fragments");
  constexpr int NB = GATED && NC == 16 ? 2 : 1, kU = small_run(GROUPED, NB);
  __shared__ __align__(16) float part[NWV][NB][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n0 = (int)(blockIdx.x % n_tiles) * NC;
  LinParams P = B.L;
  int t0 = (int)(blockIdx.x / n_tiles) * 16, end = P.T;
  if constexpr (GROUPED) {
    const RowBlock rb = find_row_block<16>(B, (int)(blockIdx.x / n_tiles));
    if (rb.e < 0) return;  // whole workgroups leave
    t0 = rb.t0;
    end = rb.end;
    if (t0 >= end) return;
    to_slot(B, rb.e, P);
  }
  const int r = lane & 15, g = lane >> 4;
  // rows past the end re-read the last one
  int t = min(t0 + r, end - 1);
  if constexpr (GROUPED) t = x_row(B, t);
  const int n = min(n0 + r % NC, P.N - 1) + (r >= NC ? P.N : 0);
  const uint8_t* xp = P.x + (int64_t)t * P.ldx + g * 16;
  const uint8_t* wp[NB];
  wp[0] = P.w + (int64_t)n * P.ldw + g * 16;
  if constexpr (NB == 2) wp[1] = P.w + (int64_t)(P.N + n) * P.ldw + g * 16;
  // scales: the lane's token; the column block of its rows of each fragment
  // (a lane of 32 .. 63 holds up rows where a fragment holds both)
  const float* xs = static_cast<const float*>(P.xs) + t;
  const float* ws[NB];
  ws[0] = static_cast<const float*>(P.ws) + (int64_t)((n0 >> 7) + (NC == 8 && g >= 2 ? B.nb : 0)) * B.steps;
  if constexpr (NB == 2) ws[1] = ws[0] + (int64_t)B.nb * B.steps;
  lf32x4_t acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = lf32x4_t{0.f, 0.f, 0.f, 0.f};
  auto load = [&](const uint8_t* p, int s) {
    Frag f;
    f.a = *reinterpret_cast<const uint4*>(p + s * 128);
    f.b = *reinterpret_cast<const uint4*>(p + s * 128 + 64);
    return f;
  };
  for (int s0 = wave * kU; s0 < B.steps; s0 += NWV * kU) {
    Frag fx[kU], fw[kU][NB];
    float sx[kU], sw[kU][NB];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int s = min(s0 + u, B.steps - 1);  // past the end: the last step again, times 0
      fx[u] = load(xp, s);
      sx[u] = xs[(int64_t)s * B.X];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        fw[u][b] = load(wp[b], s);
        sw[u][b] = ws[b][s];
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // or the compiler waits for each step's loads before the next's
#pragma unroll
    for (int u = 0; u < kU; ++u) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        lf32x4_t p = lf32x4_t{0.f, 0.f, 0.f, 0.f};
        if constexpr (EXACT) p = mma_decoded<false>(fw[u][b], fx[u], p, 0, 0, g);
        else p = mma_fp8<0, 0>(fw[u][b], fx[u], p, 127, 127);
        const float f = s0 + u < B.steps ? sx[u] * sw[u][b] : 0.f;
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[b][v] = fmaf(p[v], f, acc[b][v]);
      }
    }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) *reinterpret_cast<lf32x4_t*>(&part[wave][b][lane * 4]) = acc[b];
  // thread o: row o / NC, column o % NC; what its epilogue reads is loaded ahead of the barrier
  static_assert(64 * NWV >= 256, "an output a thread at most");
  const int tl = tid / NC, cl = tid % NC, to = t0 + tl, c = n0 + cl;
  const bool mine = tl < 16 && to < end && c < P.N;
  Epilogue<MOE_Q_NONE, GATED> e;
  if (mine) e.load(P, to, c);
  __syncthreads();
  if (!mine) return;
  const int at = (tl + 16 * (cl >> 2)) * 4 + (cl & 3);
  float a = 0.f, u = 0.f;
#pragma unroll
  for (int i = 0; i < NWV; ++i) {
    a += part[i][0][at];
    if (GATED) u += NB == 2 ? part[i][NB - 1][at] : part[i][0][at + 16 * (NC / 4) * 4];  // up: rows NC .. of the fragment
  }
  put(P, to, c, e.finish(P, a, u));
}

template <bool GATED, bool EXACT, bool GROUPED, int NC, int NWV>
void launch_small_waves(const BlockParams& B, hipStream_t s) {
  const int nt = (B.L.N + NC - 1) / NC;
  const int64_t rb = GROUPED ? most_row_blocks(B.L.T, B.E, 16) : (B.L.T + 15) / 16;
  launch(k_block_small<GATED, EXACT, GROUPED, NC, NWV>, dim3((unsigned)(nt * rb)), dim3(64 * NWV), 0, s, B, nt);
}

// Waves of a workgroup.  Dense: as many as have a run of 2 to 4 each.
template <bool GATED, bool EXACT, bool GROUPED, int NC>
void launch_small_cols(const BlockParams& B, hipStream_t s) {
  if constexpr (GROUPED) {
    if (grouped_small_waves(B.L.K) == 8) launch_small_waves<GATED, EXACT, GROUPED, NC, 8>(B, s);
    else launch_small_waves<GATED, EXACT, GROUPED, NC, 4>(B, s);
  } else {
    if (B.steps > 32) launch_small_waves<GATED, EXACT, GROUPED, NC, 16>(B, s);
    else if (B.steps > 16) launch_small_waves<GATED, EXACT, GROUPED, NC, 8>(B, s);
    else launch_small_waves<GATED, EXACT, GROUPED, NC, 4>(B, s);
  }
}

template <bool GATED, bool GROUPED, bool EXACT>
void launch_small_rows(const BlockParams& B, hipStream_t s) {
  if constexpr (GATED && !GROUPED) {
    // 8 gate and 8 up rows a workgroup by the linear product's rule: 2 x 2048 x
    // 7168, one token, 6.9 us against 9.6.  Grouped it gained nothing (2 experts
    // of 2 x 1024 x 4096 13.0 against 11.9).
    if (eight_columns(std::min(B.L.T, 16), B.L.N, B.L.kb)) return launch_small_cols<GATED, EXACT, GROUPED, 8>(B, s);
  }
  launch_small_cols<GATED, EXACT, GROUPED, 16>(B, s);
}

template <bool GATED, bool GROUPED>
void launch_small_out(const BlockParams& B, hipStream_t s) {
  if (B.L.out_f32) launch_small_rows<GATED, GROUPED, true>(B, s);
  else launch_small_rows<GATED, GROUPED, false>(B, s);
}

template <bool GROUPED>
void launch_small(const BlockParams& B, hipStream_t s) {
  if (B.L.gated) launch_small_out<true, GROUPED>(B, s);
  else launch_small_out<false, GROUPED>(B, s);
}

}  // namespace

namespace moe {

size_t linear_block_workspace(int T, int N, int K, bool gated, bool out_f32) {
  const int R = gated ? 2 * N : N;
  if (block_small_wins(T, R, gated, K, out_f32)) return 0;
  const TilePlan pl = plan_block_tiles(T, N, gated, K, out_f32);
  return pl.splits > 1 ? (size_t)pl.splits * T * R * sizeof(float) : 0;
}

void launch_linear_block(const BlockParams& B, void* workspace, hipStream_t s) {
  const LinParams& P = B.L;
  const bool fits = block_tile_fits(B);
  if (B.offsets) {
    if (!fits || grouped_small_wins(P.T, B.E)) launch_small<true>(B, s);
    else launch_block_tile(B, plan_grouped_tiles(P.T, B.E, P.N, P.gated, P.K, P.out_f32, most_row_blocks(P.T, B.E, 128)),
                           nullptr, s);
  } else {
    if (!fits || block_small_wins(P.T, P.R, P.gated, P.K, P.out_f32)) launch_small<false>(B, s);
    else launch_block_tile(B, plan_block_tiles(P.T, P.N, P.gated, P.K, P.out_f32), workspace, s);
  }
}

}  // namespace moe

extern "C" moe_status moe_linear_grouped(const moe_grouped_args* g, moe_stream_t stream) {
  MOE_CHECK_ARG(g, "moe_linear_grouped: null pointer");
  const moe_linear_args* a = &g->lin;
  MOE_CHECK_ARG(a->qmode == MOE_Q_FP8_BLOCK, "moe_linear_grouped: bad qmode %d", a->qmode);
  MOE_CHECK_ARG(a->fn >= MOE_FN_NONE && a->fn <= MOE_FN_RELU, "moe_linear_grouped: bad fn %d", a->fn);
  MOE_CHECK_ARG(a->T >= 0 && a->N >= 1 && a->K >= 1 && a->T < (1 << 24) && a->N < (1 << 24) && a->K < (1 << 24) &&
                    g->x_rows >= 0 && g->x_rows < (1 << 24),
                "moe_linear_grouped: bad sizes T=%d N=%d K=%d x_rows=%d", a->T, a->N, a->K, g->x_rows);
  MOE_CHECK_ARG(a->K % 128 == 0, "moe_linear_grouped: K=%d must be a multiple of 128", a->K);
  MOE_CHECK_ARG(g->E >= 1 && g->E <= 1024, "moe_linear_grouped: bad E=%d (1 to 1024)", g->E);
  MOE_CHECK_ARG(!a->residual, "moe_linear_grouped: no residual");
  MOE_CHECK_ARG(!g->rows || g->rows_div >= 1, "moe_linear_grouped: rows_div=%d must be at least 1", g->rows_div);
  MOE_CHECK_ARG(g->rows || g->x_rows >= a->T, "moe_linear_grouped: x_rows=%d, at least T=%d without rows", g->x_rows,
                a->T);
  MOE_CHECK_ARG(a->T == 0 || g->x_rows >= 1, "moe_linear_grouped: x_rows=%d with T=%d", g->x_rows, a->T);
  const int64_t ldx = a->ldx ? a->ldx : a->K, ldw = a->ldw ? a->ldw : a->K, ldo = a->ldo ? a->ldo : a->N;
  MOE_CHECK_ARG(ldx >= a->K && ldw >= a->K && ldx % 16 == 0 && ldw % 16 == 0,
                "moe_linear_grouped: row strides of x (%lld) and w (%lld) must be at least K=%d, in 16-byte pieces",
                (long long)ldx, (long long)ldw, a->K);
  MOE_CHECK_ARG(ldo >= a->N, "moe_linear_grouped: row stride of out (%lld) must be at least N=%d", (long long)ldo, a->N);
  MOE_CHECK_ARG(g->x_rows * ldx < (1LL << 32) && ldw < (1 << 24) && ldo < (1 << 24),
                "moe_linear_grouped: x of %d rows of %lld bytes (below 2^32 together), strides of w and out below 2^24",
                g->x_rows, (long long)ldx);
  const int R = a->gated ? 2 * a->N : a->N, steps = a->K / 128, nb = (a->N + 127) / 128;
  const int64_t wst = g->w_stride ? g->w_stride : R * ldw;
  const int64_t sst = g->w_scale_stride ? g->w_scale_stride : (int64_t)(a->gated ? 2 : 1) * nb * steps * 4;
  MOE_CHECK_ARG(wst % 16 == 0 && wst >= 0 && sst % 4 == 0 && sst >= 0,
                "moe_linear_grouped: slot strides of w (%lld) and w_scale (%lld) in pieces of 16 and 4 bytes",
                (long long)wst, (long long)sst);
  if (a->T == 0) return MOE_OK;
  MOE_CHECK_ARG(a->x && a->w && a->out && a->x_scale && a->w_scale && g->offsets, "moe_linear_grouped: null pointer");
  MOE_CHECK_ARG((((uintptr_t)a->x | (uintptr_t)a->w) & 15) == 0,
                "moe_linear_grouped: x and w must lie on 16-byte boundaries");
  MOE_CHECK_ARG((((uintptr_t)a->bias | (uintptr_t)a->x_scale | (uintptr_t)a->w_scale | (uintptr_t)g->offsets |
                  (uintptr_t)g->rows | (uintptr_t)g->slot_of_expert) & 3) == 0 &&
                    ((uintptr_t)a->out & (a->out_f32 ? 3 : 1)) == 0,
                "moe_linear_grouped: misaligned out, bias, scales, offsets, rows or slots");
  const BlockParams B{{a->T, a->N, a->K, R, a->K, static_cast<const uint8_t*>(a->x), static_cast<const uint8_t*>(a->w),
                       ldx, ldw, a->x_scale, a->w_scale, a->bias, nullptr, a->out, 0, ldo, a->fn, a->gated, a->out_f32},
                      g->x_rows, steps, nb, g->E, g->rows_div, g->offsets, g->rows, g->slot_of_expert, wst, sst / 4};
  MOE_CHECK_ARG(grouped_threads(a->T, g->E, a->N, a->gated, a->K, a->out_f32, block_tile_fits(B)) < (1LL << 32),
                "moe_linear_grouped: T=%d rows of N=%d are more than a grid holds", a->T, a->N);
  launch_linear_block(B, nullptr, reinterpret_cast<hipStream_t>(stream));
  MOE_LAUNCHED();
  return MOE_OK;
}
