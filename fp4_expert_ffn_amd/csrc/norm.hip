// RMS norm with the residual's addition, bf16 and 8-bit outputs (gfx950,
// wave64), and the 8-bit row encoding alone.
//
//   r = x + residual,  y = r w / sqrt(mean(r^2) + eps)
//
// One pass: a row lives in the registers of its TPR threads (8 values a
// thread and chunk) from its one read to its writes.  The encoding's maximum
// needs no second reduction: |y| = |r w| * rstd, and multiplying by rstd
// keeps the order after rounding, so max |y| = max |r w| * rstd; the sum of
// squares and max |r w| are reduced together.
// Bound: HBM (a few flops a byte); with few rows, one memory latency.  16384
// x 7168, bf16 residual in and out, MXFP8 out (826 MB): 145 us, 5.7 TB/s; a
// copy of 1 GiB reaches 5.0.  1027 x 2048, fp32 residual, FP8 and bf16 out (27
// MB): 7.8 us.  One row of 7168: 2.5 us, one of 64 2.1.  A scale per 128
// columns: 16 lanes hold a block, its maximum is four DPP steps; one row of
// 7168 with residual 3.3 us, the encoding of 32768 x 2048 (203 MB) 40, 5.1 TB/s.
#include <algorithm>

#include "common.h"
#include "wave.h"

namespace {

using namespace moe;

struct NormParams {
  int T, H;
  const uint16_t* x;
  const void* w;
  const void* res;
  void* res_out;
  uint16_t* out;
  uint8_t* q;
  void* qs;
  int64_t ldx, ldr, ldo, ldq;
  float eps;
  int w_f32;
};

enum { kResNone = 0, kResBf16 = 1, kResF32 = 2 };

__device__ __forceinline__ void unpack8(const uint4& u, float* v) {
  const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(d[j] << 16);
    v[2 * j + 1] = __uint_as_float(d[j] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7]));
}

// Clamps to the E4M3 range, NaN kept.
__device__ __forceinline__ float clamp_e4m3(float v) { return v != v ? v : fminf(fmaxf(v, -448.f), 448.f); }

__device__ __forceinline__ uint2 encode8(const float* v) {
  uint32_t d[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(v[4 * h]), clamp_e4m3(v[4 * h + 1]), 0, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(clamp_e4m3(v[4 * h + 2]), clamp_e4m3(v[4 * h + 3]), p, true);
    d[h] = (uint32_t)p;
  }
  return make_uint2(d[0], d[1]);
}

// The fp32 quotient by a row's scale.  The product with the rounded reciprocal
// alone would give values beside a tie of two codes the wrong one; with its
// remainder, exact in an FMA, divided once more the quotient is the nearest
// value (Markstein's division).  Both are taken times the power of two that
// brings the scale to [1, 2), so that no remainder underflows.  16384 x 7168
// rows alone 61 us with the product and with this, 72 with `/`.
struct RowScale {
  float unit, s, inv;
  __device__ __forceinline__ void set(float scale) {  // 2^-126 .. 2^120, or infinite: finite values give 0
    const uint32_t e = __float_as_uint(scale) >> 23;
    unit = e == 255u ? 0.f : __uint_as_float((254u - e) << 23);
    s = e == 255u ? 1.f : scale * unit;
    inv = 1.0f / s;
  }
  __device__ __forceinline__ float divide(float v) const {
    const float t = v * unit, q = t * inv;
    return copysignf(fmaf(fmaf(-q, s, t), inv, q), v);  // the sign: -0
  }
};

// The E8M0 code of a block's largest magnitude: floor(log2 amax) - 8 + 127.
// A subnormal amax lies below 2^-126: its code would be negative, so 0.
__device__ __forceinline__ uint32_t e8m0_of(float amax) {
  const uint32_t e = __float_as_uint(amax) >> 23;  // biased exponent; 255: infinite
  return amax == 0.f ? 127u : (e > 8u ? e - 8u : 0u);
}

// The largest magnitude of a 32-column block: its 4 lanes hold 8 values each.
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, dpp_f32<kDppQuadXor1>(v));
  return fmaxf(v, dpp_f32<kDppQuadXor2>(v));
}

__device__ __forceinline__ float wave_fmax(float v) {
  v = quad_max(v);
  v = fmaxf(v, dpp_f32<kDppRowHalfMirror>(v));
  v = fmaxf(v, dpp_f32<kDppRowMirror>(v));
  return max_rows4(v);
}

// TPR threads a row (64: four rows a workgroup), NV chunks of 8 TPR columns.
// NORM false: the encoding of x alone.
template <int TPR, int NV, int RES, int QM, bool NORM>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void k_norm(NormParams P) {
  constexpr int RPW = TPR == 64 ? 4 : 1;
  constexpr int WPR = TPR / 64;  // waves a row
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int rt = TPR == 64 ? lane : tid;
  const int row = blockIdx.x * RPW + (TPR == 64 ? wave : 0);
  if (row >= P.T) return;  // whole rows (whole waves) leave: no barrier below crosses rows
  float v[NV][8], wv[NV][8];
  const uint16_t* x = P.x + (int64_t)row * P.ldx;
  // every load of the row first
  uint4 xr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + rt) * 8;
    xr[i] = c < P.H ? *reinterpret_cast<const uint4*>(x + c) : make_uint4(0, 0, 0, 0);
  }
  uint4 rr[NV][RES == kResF32 ? 2 : 1];
  if constexpr (RES != kResNone) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + rt) * 8;
      if (c < P.H) {
        if constexpr (RES == kResBf16) {
          rr[i][0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(P.res) + (int64_t)row * P.ldr + c);
        } else {
          const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(P.res) + (int64_t)row * P.ldr + c);
          rr[i][0] = p[0];
          rr[i][1] = p[1];
        }
      } else {
        rr[i][0] = make_uint4(0, 0, 0, 0);
        if constexpr (RES == kResF32) rr[i][1] = make_uint4(0, 0, 0, 0);
      }
    }
  }
  if constexpr (NORM) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * TPR + rt) * 8;
      if (P.w == nullptr || c >= P.H) {
#pragma unroll
        for (int j = 0; j < 8; ++j) wv[i][j] = 1.f;
      } else if (P.w_f32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(P.w) + c);
        const float4 a = p[0], b = p[1];
        const float t[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) wv[i][j] = t[j];
      } else {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(P.w) + c), wv[i]);
      }
    }
  }
  float ss = 0.f, am = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + rt) * 8;
    unpack8(xr[i], v[i]);
    if constexpr (RES == kResBf16) {
      float t[8];
      unpack8(rr[i][0], t);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] += t[j];
    } else if constexpr (RES == kResF32) {
      const uint32_t t[8] = {rr[i][0].x, rr[i][0].y, rr[i][0].z, rr[i][0].w,
                             rr[i][1].x, rr[i][1].y, rr[i][1].z, rr[i][1].w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] += __uint_as_float(t[j]);
    }
    if constexpr (RES != kResNone) {
      if (P.res_out && c < P.H) {
        if constexpr (RES == kResBf16) {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.res_out) + (int64_t)row * P.ldr + c) = pack8(v[i]);
        } else {
          float4* p = reinterpret_cast<float4*>(static_cast<float*>(P.res_out) + (int64_t)row * P.ldr + c);
          p[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
          p[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (NORM) {
        ss = fmaf(v[i][j], v[i][j], ss);
        v[i][j] *= wv[i][j];
      }
      if constexpr (QM == MOE_Q_FP8) am = fmaxf(am, fabsf(v[i][j]));  // a NaN counts for no maximum
    }
  }
  if constexpr (NORM) ss = wave_sum(ss);
  if constexpr (QM == MOE_Q_FP8) am = wave_fmax(am);
  if constexpr (WPR > 1 && (NORM || QM == MOE_Q_FP8)) {
    __shared__ float s_sum[WPR], s_max[WPR];
    if (lane == 0) {
      s_sum[wave] = ss;
      s_max[wave] = am;
    }
    __syncthreads();
    ss = 0.f;
    am = 0.f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) {
      ss += s_sum[i];
      am = fmaxf(am, s_max[i]);
    }
  }
  float rstd = 1.f;
  if constexpr (NORM) rstd = 1.0f / sqrtf(ss / (float)P.H + P.eps);
  RowScale rs;
  if constexpr (QM == MOE_Q_FP8) {
    const float scale = fmaxf(am * rstd / 448.0f, 1.17549435e-38f)  /* 2^-126 */;
    rs.set(scale);
    if (rt == 0) static_cast<float*>(P.qs)[row] = scale;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + rt) * 8;
    if constexpr (NORM) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= rstd;
    }
    if constexpr (NORM) {
      if (P.out && c < P.H) *reinterpret_cast<uint4*>(P.out + (int64_t)row * P.ldo + c) = pack8(v[i]);
    }
    if constexpr (QM == MOE_Q_MXFP8) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[i][j]));
      const uint32_t code = e8m0_of(quad_max(m));
      // 2^-(code - 127) as a float: 254 - code is its biased exponent (code <= 247)
      const float inv = __uint_as_float((254u - code) << 23);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= inv;  // a power of two: exact
      // the four codes of a 128-column tile, from lanes 0, 4, 8, 12 of its 16
      const uint32_t up = dpp_u32<kDppRowHalfMirror>(code);  // lanes l <-> 7 - l within 8: the other block
      const uint32_t pair = (lane & 4) ? (up | (code << 8)) : (code | (up << 8));
      const uint32_t far = dpp_u32<kDppRowMirror>(pair);     // lanes l <-> 15 - l: the other pair
      if (c < P.H && (lane & 15) == 0)
        static_cast<uint32_t*>(P.qs)[(int64_t)(c >> 7) * P.T + row] = pair | (far << 16);
    }
    if constexpr (QM == MOE_Q_FP8_BLOCK) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[i][j]));
      // the 16 lanes of a block are a row of the wave
      m = quad_max(m);
      m = fmaxf(m, dpp_f32<kDppRowHalfMirror>(m));
      m = fmaxf(m, dpp_f32<kDppRowMirror>(m));
      const float scale = fmaxf(m / 448.0f, 1.17549435e-38f)  /* 2^-126 */;
      rs.set(scale);
      if (c < P.H && (lane & 15) == 0) static_cast<float*>(P.qs)[(int64_t)(c >> 7) * P.T + row] = scale;
    }
    if constexpr (QM == MOE_Q_FP8 || QM == MOE_Q_FP8_BLOCK)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = rs.divide(v[i][j]);
    if constexpr (QM != MOE_Q_NONE)
      if (c < P.H) *reinterpret_cast<uint2*>(P.q + (int64_t)row * P.ldq + c) = encode8(v[i]);
  }
}

template <int RES, int QM, bool NORM>
void launch_norm(const NormParams& P, hipStream_t s) {
  // Few values a thread, so that a CU holds many rows' loads; a wave a row
  // only where a wider row would leave most of its threads idle.  8000 rows,
  // bf16 and MXFP8 out, us: H = 1024 64 x 2 chunks 11.2 and 11.8, 256 x 1 12.7
  // and 13.8; 2048 256 x 1 21.7 and 19.9, 64 x 4 21.9 and 22.2 (one row 2.1
  // and 2.4 against 2.9 and 3.7); 4096 256 x 2 46.7 and 44.3, 512 x 1 47.9 and
  // 45.0; 8192 512 x 2 90.4 and 83.1, 256 x 4 98.4 and 91.5, 1024 x 1 94.2 and
  // 85.7; 16384 1024 x 2 192 and 165, 512 x 4 194 and 172, 1024 x 4 189 and
  // 188 (one row 3.3 against 3.9).
  const int chunks = (P.H + 7) / 8;
  if (chunks <= 128) {
    const dim3 g((unsigned)((P.T + 3) / 4));
    if (chunks <= 64) launch(k_norm<64, 1, RES, QM, NORM>, g, dim3(256), 0, s, P);
    else launch(k_norm<64, 2, RES, QM, NORM>, g, dim3(256), 0, s, P);
    return;
  }
  const dim3 g((unsigned)P.T);
  if (chunks <= 256) launch(k_norm<256, 1, RES, QM, NORM>, g, dim3(256), 0, s, P);
  else if (chunks <= 512) launch(k_norm<256, 2, RES, QM, NORM>, g, dim3(256), 0, s, P);
  else if (chunks <= 1024) launch(k_norm<512, 2, RES, QM, NORM>, g, dim3(512), 0, s, P);
  else if (chunks <= 2048) launch(k_norm<1024, 2, RES, QM, NORM>, g, dim3(1024), 0, s, P);
  else launch(k_norm<1024, 4, RES, QM, NORM>, g, dim3(1024), 0, s, P);
}

template <int RES>
void launch_norm_q(const NormParams& P, int qm, hipStream_t s) {
  if (qm == MOE_Q_NONE) launch_norm<RES, MOE_Q_NONE, true>(P, s);
  else if (qm == MOE_Q_FP8) launch_norm<RES, MOE_Q_FP8, true>(P, s);
  else if (qm == MOE_Q_MXFP8) launch_norm<RES, MOE_Q_MXFP8, true>(P, s);
  else launch_norm<RES, MOE_Q_FP8_BLOCK, true>(P, s);
}

constexpr int kMaxRows = 1 << 22;  // x 1024 threads: what a grid holds (below 2^32 threads)

bool misaligned(const void* p, unsigned a) { return ((uintptr_t)p & (a - 1)) != 0; }

}  // namespace

extern "C" moe_status moe_rmsnorm(const moe_norm_args* a, moe_stream_t stream) {
  MOE_CHECK_ARG(a, "moe_rmsnorm: null pointer");
  MOE_CHECK_ARG(a->T >= 0 && a->T < kMaxRows && a->H >= 8 && a->H <= 32768 && a->H % 8 == 0,
                "moe_rmsnorm: bad sizes T=%d H=%d (T below 2^22, H a multiple of 8, at most 32768)", a->T, a->H);
  MOE_CHECK_ARG(a->eps >= 0.f, "moe_rmsnorm: eps must be >= 0");
  MOE_CHECK_ARG(a->qmode >= MOE_Q_NONE && a->qmode <= MOE_Q_FP8_BLOCK, "moe_rmsnorm: bad qmode %d", a->qmode);
  MOE_CHECK_ARG((a->qmode != MOE_Q_MXFP8 && a->qmode != MOE_Q_FP8_BLOCK) || a->H % 128 == 0,
                "moe_rmsnorm: MXFP8 and FP8_BLOCK rows need H %% 128 == 0, H=%d", a->H);
  const int64_t ld[4] = {a->ldx ? a->ldx : a->H, a->ldr ? a->ldr : a->H, a->ldo ? a->ldo : a->H,
                         a->ldq ? a->ldq : a->H};
  for (int64_t l : ld)
    MOE_CHECK_ARG(l >= a->H && l % 8 == 0, "moe_rmsnorm: row stride %lld must be a multiple of 8, at least H=%d",
                  (long long)l, a->H);
  MOE_CHECK_ARG(!a->residual_out || a->residual, "moe_rmsnorm: residual_out without residual");
  MOE_CHECK_ARG(a->out || a->residual_out || a->qmode != MOE_Q_NONE, "moe_rmsnorm: no output");
  if (a->T == 0) return MOE_OK;
  MOE_CHECK_ARG(a->x && (a->qmode == MOE_Q_NONE || (a->q && a->q_scale)), "moe_rmsnorm: null pointer");
  MOE_CHECK_ARG(!misaligned(a->x, 16) && !misaligned(a->weight, 16) && !misaligned(a->residual, 16) &&
                    !misaligned(a->residual_out, 16) && !misaligned(a->out, 16) &&
                    (a->qmode == MOE_Q_NONE || (!misaligned(a->q, 8) && !misaligned(a->q_scale, 8))),
                "moe_rmsnorm: misaligned pointer (16 bytes; q and q_scale 8)");
  const NormParams P{a->T, a->H, a->x, a->weight, a->residual, a->residual_out, a->out, a->q, a->q_scale,
                     ld[0], ld[1], ld[2], ld[3], a->eps, a->weight_f32};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (!a->residual) launch_norm_q<kResNone>(P, a->qmode, s);
  else if (a->residual_f32) launch_norm_q<kResF32>(P, a->qmode, s);
  else launch_norm_q<kResBf16>(P, a->qmode, s);
  MOE_LAUNCHED();
  return MOE_OK;
}

extern "C" moe_status moe_quantize_fp8(const uint16_t* x, int64_t ldx, int rows, int cols, int qmode, uint8_t* q,
                                       void* q_scale, moe_stream_t stream) {
  MOE_CHECK_ARG(rows >= 0 && rows < kMaxRows && cols >= 8 && cols <= 32768 && cols % 8 == 0,
                "moe_quantize_fp8: bad sizes rows=%d cols=%d (rows below 2^22, cols a multiple of 8, at most 32768)",
                rows, cols);
  MOE_CHECK_ARG(qmode >= MOE_Q_FP8 && qmode <= MOE_Q_FP8_BLOCK, "moe_quantize_fp8: bad qmode %d", qmode);
  MOE_CHECK_ARG(qmode == MOE_Q_FP8 || cols % 128 == 0,
                "moe_quantize_fp8: MXFP8 and FP8_BLOCK rows need cols %% 128 == 0, cols=%d", cols);
  if (ldx == 0) ldx = cols;
  MOE_CHECK_ARG(ldx >= cols && ldx % 8 == 0, "moe_quantize_fp8: row stride %lld must be a multiple of 8, at least %d",
                (long long)ldx, cols);
  if (rows == 0) return MOE_OK;
  MOE_CHECK_ARG(x && q && q_scale, "moe_quantize_fp8: null pointer");
  MOE_CHECK_ARG(!misaligned(x, 16) && !misaligned(q, 8) && !misaligned(q_scale, 8),
                "moe_quantize_fp8: misaligned pointer (x 16 bytes; q and q_scale 8)");
  const NormParams P{rows, cols, x, nullptr, nullptr, nullptr, nullptr, q, q_scale, ldx, cols, cols, cols, 0.f, 0};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (qmode == MOE_Q_FP8) launch_norm<kResNone, MOE_Q_FP8, false>(P, s);
  else if (qmode == MOE_Q_MXFP8) launch_norm<kResNone, MOE_Q_MXFP8, false>(P, s);
  else launch_norm<kResNone, MOE_Q_FP8_BLOCK, false>(P, s);
  MOE_LAUNCHED();
  return MOE_OK;
}
