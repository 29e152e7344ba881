// The linear product with its epilogue (gfx950): out = fn(x W^T + bias)
// [* up] + residual, for bf16 operands (v_mfma_f32_16x16x32_bf16) and E4M3
// operands (decoded to bf16), fp32 accumulation.
//
// Every operand row is read in K-steps of 128 bytes: 128 E4M3 codes or 64
// bf16 values.
// The weights are the instruction's first operand: lane l of the result
// holds token l % 16 and columns 4 (l / 16) + v.
#include <algorithm>

#include "linear.h"

namespace {

using namespace moe;

// One workgroup: 16 columns (gated: their gate and up rows) x 16 tokens, the
// K-steps dealt to its 4 waves, their sums joined in LDS in wave order.
constexpr int kSmallWaves = 4;

template <int QM, bool GATED>
__global__ __launch_bounds__(64 * kSmallWaves) void k_linear_small(LinParams P, int n_tiles) {
  constexpr int NB = GATED ? 2 : 1;
  __shared__ lf32x4_t part[kSmallWaves][NB][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n0 = (int)(blockIdx.x % n_tiles) * 16, t0 = (int)(blockIdx.x / n_tiles) * 16;
  const int r = lane & 15, g = lane >> 4;
  const int t = min(t0 + r, P.T - 1), n = min(n0 + r, P.N - 1);  // rows past the end re-read the last one
  const uint8_t* xp = P.x + (int64_t)t * P.ldx;
  const uint8_t* wp[NB];
  wp[0] = P.w + (int64_t)n * P.ldw;
  if (GATED) wp[1] = P.w + (int64_t)(P.N + n) * P.ldw;
  lf32x4_t acc[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b] = lf32x4_t{0.f, 0.f, 0.f, 0.f};
  const int steps = (P.kb + 127) / 128;
  // Lane l reads bytes 32 (l / 16) .. + 31 of a step: the same permutation of
  // K in both operands, and for MXFP8 one scale block.  Bytes past the row's
  // end: a valid piece is loaded and zeroed.
  auto load = [&](const uint8_t* p, int s) {
    Frag f;
    const int o = s * 128 + g * 32;
    const uint4 a = *reinterpret_cast<const uint4*>(p + min(o, P.kb - 16));
    const uint4 b = *reinterpret_cast<const uint4*>(p + min(o + 16, P.kb - 16));
    const uint32_t ma = o < P.kb ? ~0u : 0u, mb = o + 16 < P.kb ? ~0u : 0u;
    f.a = make_uint4(a.x & ma, a.y & ma, a.z & ma, a.w & ma);
    f.b = make_uint4(b.x & mb, b.y & mb, b.z & mb, b.w & mb);
    return f;
  };
  for (int s = wave; s < steps; s += kSmallWaves) {
    const Frag xf = load(xp, s);
    float fx = 1.f, fw[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) fw[b] = 1.f;
    if constexpr (QM == MOE_Q_MXFP8) {
      fx = e8m0_to_f32(static_cast<const uint8_t*>(P.xs)[((int64_t)s * P.T + t) * 4 + g]);
#pragma unroll
      for (int b = 0; b < NB; ++b)
        fw[b] = e8m0_to_f32(static_cast<const uint8_t*>(P.ws)[((int64_t)s * P.R + b * P.N + n) * 4 + g]);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[b] = mma_exact<QM>(load(wp[b], s), xf, acc[b], fw[b], fx);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) part[wave][b][lane] = acc[b];
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int i = 1; i < kSmallWaves; ++i) acc[b] += part[i][b][lane];
  }
  if (t0 + r >= P.T) return;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const int c = n0 + 4 * g + v;
    if (c < P.N) put(P, t, c, finish<QM, GATED>(P, t, c, acc[0][v], GATED ? acc[NB - 1][v] : 0.f));
  }
}

template <int QM>
void launch_small(const LinParams& P, hipStream_t s) {
  const int nt = (P.N + 15) / 16, tt = (P.T + 15) / 16;
  const dim3 g((unsigned)((long long)nt * tt));
  if (P.gated) launch(k_linear_small<QM, true>, g, dim3(64 * kSmallWaves), 0, s, P, nt);
  else launch(k_linear_small<QM, false>, g, dim3(64 * kSmallWaves), 0, s, P, nt);
}

}  // namespace

extern "C" size_t moe_linear_workspace_size(const moe_linear_args* a) {
  (void)a;
  return 0;
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
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (a->T > 32 && linear_tile_fits(P)) launch_linear_tile(P, a->qmode, s);
  else if (a->qmode == MOE_Q_NONE) launch_small<MOE_Q_NONE>(P, s);
  else if (a->qmode == MOE_Q_FP8) launch_small<MOE_Q_FP8>(P, s);
  else launch_small<MOE_Q_MXFP8>(P, s);
  MOE_LAUNCHED();
  return MOE_OK;
}
