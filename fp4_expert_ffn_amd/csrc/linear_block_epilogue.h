// The epilogue of the block-scaled product's own tile kernels
// (linear_block_big.hip, linear_block_stream.hip).
#pragma once
#include "linear_tile.h"

namespace moe {

// Waves in WM x WN, each TM x TN 16 x 16 tiles; OS: 16-column groups of output
// staged at once, 16 rows of 16 OS + 4 floats a wave at `staging`.  Rows t0 ..
// t_end - 1 at most, output columns from n0 on.  Lane: row r16 of a 16-row
// group, weight rows 4 g + v of a group: bias, activation and gate in place;
// then, through LDS in fp32, rows of 8 columns a lane: the residual and whole
// 16-byte stores.  bf16 outputs.
template <bool GATED, int WM, int WN, int TM, int TN, int OS>
__device__ __forceinline__ void block_epilogue(const LinParams& P, const LinTiles& G, lf32x4_t (&acc)[TM][TN],
                                               float* staging, int t0, int t_end, int n0, int lane, int wave) {
  constexpr int OC = GATED ? TN / 2 : TN, Q = OC / OS;          // groups of output a wave; stagings a row group
  constexpr int SR = OS * 16 + 4;
  constexpr int LPR = OS * 2, RP = 64 / LPR, PS = 16 / RP;      // lanes a row, rows a pass, passes
  const int wm = wave / WN, wn = wave % WN, r16 = lane & 15, g = lane >> 4;
  const int er = lane / LPR, ec0 = n0 + wn * OC * 16 + (lane % LPR) * 8;
  const int tw = t0 + wm * TM * 16;  // the wave's first row
  const bool vec = G.vec_out && (G.vec_res || !P.res);
  if (P.bias) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int q = wn * TN + j, c = n0 + (GATED ? (q >> 1) * 16 : q * 16) + 4 * g;
      const float* b = P.bias + (GATED && (q & 1) ? P.N : 0);
      float bj[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) bj[v] = b[min(c + v, P.N - 1)];
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] += bj[v];
    }
  }
  // residual rows, four stagings ahead of their stores (out may be the
  // residual: a lane reads and writes the same places)
  constexpr int RD = TM * Q < 4 ? TM * Q : 4;
  uint4 rr[RD][PS];
  auto load_res = [&](int q) __attribute__((always_inline)) {
    const int ec = ec0 + q % Q * OS * 16;
    if (P.res && vec && ec + 8 <= P.N) {
#pragma unroll
      for (int p = 0; p < PS; ++p) {
        const int t = tw + q / Q * 16 + p * RP, rows = t_end - t;  // uniform
        if (rows > 0)
          rr[q % RD][p] = *reinterpret_cast<const uint4*>(P.res + (int64_t)t * P.ldr +
                                                          (uint32_t)(min(er, rows - 1) * (int)P.ldr + ec));
      }
    }
  };
#pragma unroll
  for (int q = 0; q < RD; ++q) load_res(q);
  auto activate = [&](int i, auto fc) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < TN; j += GATED ? 2 : 1)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][j][v] = act_of<decltype(fc)::value>(acc[i][j][v]);
  };
  float* stg = staging + wave * 16 * SR;
#pragma unroll
  for (int q = 0; q < TM * Q; ++q) {
    const int i = q / Q, o0 = q % Q * OS, ec = ec0 + o0 * 16;
    if (q % Q == 0) {
      switch (P.fn) {
        case MOE_FN_SILU: activate(i, std::integral_constant<int, MOE_FN_SILU>{}); break;
        case MOE_FN_GELU_TANH: activate(i, std::integral_constant<int, MOE_FN_GELU_TANH>{}); break;
        case MOE_FN_GELU_ERF: activate(i, std::integral_constant<int, MOE_FN_GELU_ERF>{}); break;
        case MOE_FN_RELU: activate(i, std::integral_constant<int, MOE_FN_RELU>{}); break;
        default: break;
      }
    }
    const bool whole = vec && ec + 8 <= P.N;
#pragma unroll
    for (int o = 0; o < OS; ++o) {
      float y[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) y[v] = GATED ? acc[i][2 * (o0 + o)][v] * acc[i][2 * (o0 + o) + 1][v] : acc[i][o0 + o][v];
      *reinterpret_cast<float4*>(stg + r16 * SR + o * 16 + 4 * g) = make_float4(y[0], y[1], y[2], y[3]);
    }
    asm volatile("" ::: "memory");  // a wave's LDS accesses keep their order
#pragma unroll
    for (int p = 0; p < PS; ++p) {
      const float4 a = *reinterpret_cast<const float4*>(stg + (p * RP + er) * SR + (lane % LPR) * 8);
      const float4 b = *reinterpret_cast<const float4*>(stg + (p * RP + er) * SR + (lane % LPR) * 8 + 4);
      float y[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      const int t = tw + i * 16 + p * RP + er;
      if (t < t_end && whole) {
        if (P.res) {
          const uint4 r = rr[q % RD][p];
          const uint32_t d[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[2 * e] += __uint_as_float(d[e] << 16);
            y[2 * e + 1] += __uint_as_float(d[e] & 0xFFFF0000u);
          }
        }
        const int64_t ob = (int64_t)(tw + i * 16 + p * RP) * P.ldo;  // uniform
        const uint32_t ol = (uint32_t)(er * (int)P.ldo + ec);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.out) + ob + ol) = make_uint4(
            bf16x2_rne(y[0], y[1]), bf16x2_rne(y[2], y[3]), bf16x2_rne(y[4], y[5]), bf16x2_rne(y[6], y[7]));
      } else if (t < t_end) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (ec + e < P.N)
            static_cast<uint16_t*>(P.out)[(int64_t)t * P.ldo + ec + e] =
                f32_to_bf16_rne(P.res ? y[e] + bf16_to_f32(P.res[(int64_t)t * P.ldr + ec + e]) : y[e]);
      }
    }
    asm volatile("" ::: "memory");
    if (q + RD < TM * Q) load_res(q + RD);
  }
}

}  // namespace moe
