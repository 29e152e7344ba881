// The linear product with its epilogue (gfx950): out = fn(x W^T + bias)
// [* up] + residual, for bf16 and E4M3 operands, fp32 accumulation.
//
// Every operand row is read in K-steps of 128 bytes: 128 E4M3 codes or 64
// bf16 values.
// The weights are the instruction's first operand: lane l of the result
// holds token l % 16 and columns 4 (l / 16) + v.
#include <algorithm>

#include "linear.h"
#include "linear_plan.h"

namespace {

using namespace moe;

// Few tokens: a stream of the weights.  One workgroup: NC columns (gated:
// their gate and up rows) x 16 tokens; its NWV waves take runs of kU K-steps
// in turn and load a run at once (gated, 16 columns: 16 KiB of weights a wave
// in flight), so that a row of up to NWV * kU steps costs one memory latency;
// the waves' sums are joined in LDS in wave order.  NC = 8 (gated): the gate
// and up rows of 8 columns are the rows of one fragment, twice the workgroups
// where 16 columns leave CUs idle (one token, 2048 + 2048 FP8 rows of 7168:
// 9.1 -> 6.6 us; 3584 + 3584 rows fill the chip with 16 columns).  Bound:
// what a CU can load (few workgroups), else the memory behind the L2s.  That
// call reads 4.5 TB/s where its 29 MB stay in the last-level cache from call
// to call, and takes 7.4 us, 4.0 TB/s, where 22 sets of weights take turns.
constexpr int kU = 4;

template <int QM, bool GATED, bool EXACT, int NC, int NWV>
__global__ __launch_bounds__(64 * NWV) void k_linear_small(LinParams P, int n_tiles) {
  static_assert(NC == 16 || (NC == 8 && GATED), "whole fragments");
  constexpr int NB = GATED && NC == 16 ? 2 : 1;
  constexpr bool MX = QM == MOE_Q_MXFP8;
  __shared__ float part[NWV][NB][256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n0 = (int)(blockIdx.x % n_tiles) * NC, t0 = (int)(blockIdx.x / n_tiles) * 16;
  const int r = lane & 15, g = lane >> 4;
  // rows past the end re-read the last one
  const int t = min(t0 + r, P.T - 1), n = min(n0 + r % NC, P.N - 1) + (r >= NC ? P.N : 0);
  const uint8_t* xp = P.x + (int64_t)t * P.ldx;
  const uint8_t* wp[NB];
  wp[0] = P.w + (int64_t)n * P.ldw;
  if constexpr (NB == 2) wp[1] = P.w + (int64_t)(P.N + n) * P.ldw;
  lf32x4_t acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = lf32x4_t{0.f, 0.f, 0.f, 0.f};
  const int steps = (P.kb + 127) / 128;
  // Lane l reads the 16-byte pieces l / 16 and 4 + l / 16 of a step: the FP8
  // instruction's order of K, of which lane l scales columns 32 (l / 16) .. + 31.
  // Past the row's end a valid piece is loaded (and zeroed below).
  auto load = [&](const uint8_t* p, int s) {
    Frag f;
    const int o = s * 128 + g * 16;
    f.a = *reinterpret_cast<const uint4*>(p + min(o, P.kb - 16));
    f.b = *reinterpret_cast<const uint4*>(p + min(o + 64, P.kb - 16));
    return f;
  };
  auto cut = [&](Frag& f, int s) {
    const int o = s * 128 + g * 16;
    const uint32_t ma = o < P.kb ? ~0u : 0u, mb = o + 64 < P.kb ? ~0u : 0u;
    f.a = make_uint4(f.a.x & ma, f.a.y & ma, f.a.z & ma, f.a.w & ma);
    f.b = make_uint4(f.b.x & mb, f.b.y & mb, f.b.z & mb, f.b.w & mb);
  };
  for (int s0 = wave * kU; s0 < steps; s0 += NWV * kU) {
    Frag fx[kU], fw[kU][NB];
    uint32_t sx[kU], sw[kU][NB];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int s = min(s0 + u, steps - 1);
      fx[u] = load(xp, s);
#pragma unroll
      for (int b = 0; b < NB; ++b) fw[u][b] = load(wp[b], s);
      if constexpr (MX) {
        // the row's four block scales
        sx[u] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(P.xs) + ((int64_t)s * P.T + t) * 4);
#pragma unroll
        for (int b = 0; b < NB; ++b)
          sw[u][b] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(P.ws) +
                                                        ((int64_t)s * P.R + b * P.N + n) * 4);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (s0 + u < steps) {
        if (!MX && s0 + u == steps - 1) {
          cut(fx[u], s0 + u);
#pragma unroll
          for (int b = 0; b < NB; ++b) cut(fw[u][b], s0 + u);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if constexpr (QM == MOE_Q_NONE) acc[b] = mma_bf16_step(fw[u][b], fx[u], acc[b]);
          else if constexpr (EXACT) acc[b] = mma_decoded<MX>(fw[u][b], fx[u], acc[b], MX ? sw[u][b] : 0, MX ? sx[u] : 0, g);
          else acc[b] = mma_fp8<0, 0>(fw[u][b], fx[u], acc[b], MX ? (int)(sw[u][b] >> (8 * g)) : 127,
                                      MX ? (int)(sx[u] >> (8 * g)) : 127);
        }
      }
    }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) *reinterpret_cast<lf32x4_t*>(&part[wave][b][lane * 4]) = acc[b];
  // thread o: token o / NC, column o % NC; what its epilogue reads is loaded ahead of the barrier
  static_assert(64 * NWV >= 256, "an output a thread at most");
  const int tl = tid / NC, cl = tid % NC, to = t0 + tl, c = n0 + cl;
  const bool mine = tl < 16 && to < P.T && c < P.N;
  Epilogue<QM, GATED> e;
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

template <int QM, bool GATED, bool EXACT, int NC>
void launch_small_waves(const LinParams& P, hipStream_t s) {
  const int nt = (P.N + NC - 1) / NC, tt = (P.T + 15) / 16;
  const dim3 g((unsigned)((long long)nt * tt));
  const int steps = (P.kb + 127) / 128;
  if (steps > 8 * kU) launch(k_linear_small<QM, GATED, EXACT, NC, 16>, g, dim3(1024), 0, s, P, nt);
  else if (steps > 4 * kU) launch(k_linear_small<QM, GATED, EXACT, NC, 8>, g, dim3(512), 0, s, P, nt);
  else launch(k_linear_small<QM, GATED, EXACT, NC, 4>, g, dim3(256), 0, s, P, nt);
}

template <int QM, bool GATED, bool EXACT>
void launch_small_cols(const LinParams& P, hipStream_t s) {
  if constexpr (GATED) {
    if (eight_columns(std::min(P.T, 16), P.N, P.kb)) return launch_small_waves<QM, GATED, EXACT, 8>(P, s);
  }
  launch_small_waves<QM, GATED, EXACT, 16>(P, s);
}

template <int QM, bool GATED>
void launch_small_gate(const LinParams& P, hipStream_t s) {
  if (QM != MOE_Q_NONE && P.out_f32) launch_small_cols<QM, GATED, QM != MOE_Q_NONE>(P, s);
  else launch_small_cols<QM, GATED, false>(P, s);
}

template <int QM>
void launch_small(const LinParams& P, hipStream_t s) {
  if (P.gated) launch_small_gate<QM, true>(P, s);
  else launch_small_gate<QM, false>(P, s);
}

}  // namespace

extern "C" size_t moe_linear_workspace_size(const moe_linear_args* a) {
  if (!a || a->T < 1 || a->N < 1 || a->K < 1 || a->T >= (1 << 24) || a->N >= (1 << 24) || a->K >= (1 << 24))
    return 0;
  const int kb = a->K * (a->qmode == MOE_Q_NONE ? 2 : 1);
  const int R = a->gated ? 2 * a->N : a->N;
  const bool exact = a->qmode != MOE_Q_NONE && a->out_f32;
  return small_wins(a->T, R, a->gated, kb, exact) ? 0 : linear_tile_workspace(a->T, R, kb, exact);
}

extern "C" moe_status moe_linear(const moe_linear_args* a, moe_stream_t stream) {
  MOE_CHECK_ARG(a, "moe_linear: null pointer");
  MOE_CHECK_ARG(a->qmode >= MOE_Q_NONE && a->qmode <= MOE_Q_MXFP8, "moe_linear: bad qmode %d", a->qmode);
  MOE_CHECK_ARG(a->fn >= MOE_FN_NONE && a->fn <= MOE_FN_RELU, "moe_linear: bad fn %d", a->fn);
  MOE_CHECK_ARG(a->T >= 0 && a->N >= 1 && a->K >= 1 && a->T < (1 << 24) && a->N < (1 << 24) && a->K < (1 << 24),
                "moe_linear: bad sizes T=%d N=%d K=%d", a->T, a->N, a->K);
  const int es = a->qmode == MOE_Q_NONE ? 2 : 1;
  const int kq = a->qmode == MOE_Q_NONE ? 8 : (a->qmode == MOE_Q_FP8 ? 16 : 128);
  MOE_CHECK_ARG(a->K % kq == 0, "moe_linear: K=%d must be a multiple of %d", a->K, kq);
  const int64_t ldx = a->ldx ? a->ldx : a->K, ldw = a->ldw ? a->ldw : a->K;
  const int64_t ldr = a->ldr ? a->ldr : a->N, ldo = a->ldo ? a->ldo : a->N;
  MOE_CHECK_ARG(ldx >= a->K && ldw >= a->K && (ldx * es) % 16 == 0 && (ldw * es) % 16 == 0,
                "moe_linear: row strides of x (%lld) and w (%lld) must be at least K=%d, in 16-byte pieces",
                (long long)ldx, (long long)ldw, a->K);
  MOE_CHECK_ARG(ldr >= a->N && ldo >= a->N, "moe_linear: row strides of residual (%lld) and out (%lld) must be at least N=%d",
                (long long)ldr, (long long)ldo, a->N);
  if (a->T == 0) return MOE_OK;
  MOE_CHECK_ARG(a->x && a->w && a->out && (a->qmode == MOE_Q_NONE || (a->x_scale && a->w_scale)),
                "moe_linear: null pointer");
  MOE_CHECK_ARG((((uintptr_t)a->x | (uintptr_t)a->w) & 15) == 0, "moe_linear: x and w must lie on 16-byte boundaries");
  auto off = [](const void* p, unsigned n) { return ((uintptr_t)p & (n - 1)) != 0; };
  MOE_CHECK_ARG(!off(a->out, a->out_f32 ? 4 : 2) && !off(a->bias, 4) && !off(a->residual, 2) && !off(a->x_scale, 4) &&
                    !off(a->w_scale, 4),
                "moe_linear: misaligned out, bias, residual or scales");
  LinParams P{};
  P.T = a->T;
  P.N = a->N;
  P.K = a->K;
  P.R = a->gated ? 2 * a->N : a->N;
  P.kb = a->K * es;
  P.x = static_cast<const uint8_t*>(a->x);
  P.w = static_cast<const uint8_t*>(a->w);
  P.ldx = ldx * es;
  P.ldw = ldw * es;
  P.xs = a->x_scale;
  P.ws = a->w_scale;
  P.bias = a->bias;
  P.res = a->residual;
  P.out = a->out;
  P.ldr = ldr;
  P.ldo = ldo;
  P.fn = a->fn;
  P.gated = a->gated;
  P.out_f32 = a->out_f32;
  const bool tile =
      !small_wins(P.T, P.R, P.gated, P.kb, a->qmode != MOE_Q_NONE && P.out_f32) && linear_tile_fits(P);
  const size_t need = tile ? moe_linear_workspace_size(a) : 0;
  if (need > 0) {
    if (!a->workspace || a->workspace_bytes < need)
      return set_error(MOE_ENOMEM, "moe_linear: workspace %zu bytes, needs %zu", a->workspace ? a->workspace_bytes : 0,
                       need);
    MOE_CHECK_ARG(!off(a->workspace, 16), "moe_linear: workspace must lie on a 16-byte boundary");
  }
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (tile) launch_linear_tile(P, a->qmode, a->workspace, s);
  else if (a->qmode == MOE_Q_NONE) launch_small<MOE_Q_NONE>(P, s);
  else if (a->qmode == MOE_Q_FP8) launch_small<MOE_Q_FP8>(P, s);
  else launch_small<MOE_Q_MXFP8>(P, s);
  MOE_LAUNCHED();
  return MOE_OK;
}
