// Shared by the linear product's kernels: parameters, matrix steps, epilogue.
#pragma once
#include "common.h"
#include "wave.h"

namespace moe {

typedef __bf16 lbf16x8_t __attribute__((ext_vector_type(8)));
typedef int li32x8_t __attribute__((ext_vector_type(8)));
typedef float lf32x4_t __attribute__((ext_vector_type(4)));

struct LinParams {
  int T, N, K, R;
  int kb;              // bytes of an operand row
  const uint8_t* x;
  const uint8_t* w;
  int64_t ldx, ldw;    // bytes
  const void* xs;
  const void* ws;
  const float* bias;
  const uint16_t* res;
  void* out;
  int64_t ldr, ldo;    // elements
  int fn, gated, out_f32;
};

struct Frag {
  uint4 a, b;  // the 32 bytes
};

// 8 E4M3 codes as bf16 values times 2^(e8m0 - 127) (the scale of MXFP8 codes; exact unless the value leaves bf16's range).
__device__ __forceinline__ lbf16x8_t e4m3_bf16(uint32_t lo, uint32_t hi, float scale) {
  const uint4 u = make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false)),
                             __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true)),
                             __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false)),
                             __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true)));
  return __builtin_bit_cast(lbf16x8_t, u);
}

__device__ __forceinline__ lf32x4_t mma_bf16(lbf16x8_t w, lbf16x8_t x, lf32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, c, 0, 0, 0);
}

// One K-step of 128 bytes, a fragment of each operand: lane l holds the
// 16-byte pieces l / 16 and 4 + l / 16 of its row.
__device__ __forceinline__ lf32x4_t mma_bf16_step(const Frag& w, const Frag& x, lf32x4_t c) {
  c = mma_bf16(__builtin_bit_cast(lbf16x8_t, w.a), __builtin_bit_cast(lbf16x8_t, x.a), c);
  return mma_bf16(__builtin_bit_cast(lbf16x8_t, w.b), __builtin_bit_cast(lbf16x8_t, x.b), c);
}

// E4M3 operands on the FP8 matrix instruction, block scales in byte J (I) of
// sw (sx) for columns 32 (l / 16) .. + 31 (127: none).  The instruction adds 8
// neighbouring products after cutting each below 2^-13 of the exponent of the
// largest (measured on the GPU; a sum is then within 2e-5 of its norm), which
// a bf16 output cannot show; fp32 outputs take mma_decoded.
template <int J, int I>
__device__ __forceinline__ lf32x4_t mma_fp8(const Frag& w, const Frag& x, lf32x4_t c, int sw, int sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(li32x8_t, w),
                                                          __builtin_bit_cast(li32x8_t, x), c, 0, 0, J, sw, I, sx);
}

// E4M3 operands decoded to bf16: every product exact, every sum in fp32 (four
// bf16 instructions in the place of one).  sw, sx: the rows' four block
// scales; lane group g's pieces g and 4 + g lie in blocks g / 2 and 2 + g / 2.
template <bool MX>
__device__ __forceinline__ lf32x4_t mma_decoded(const Frag& w, const Frag& x, lf32x4_t c, uint32_t sw, uint32_t sx,
                                                int g) {
  float w0 = 1.f, w1 = 1.f, x0 = 1.f, x1 = 1.f;
  if constexpr (MX) {
    const int sh = 8 * (g >> 1);
    w0 = e8m0_to_f32((sw >> sh) & 255u);
    w1 = e8m0_to_f32((sw >> (sh + 16)) & 255u);
    x0 = e8m0_to_f32((sx >> sh) & 255u);
    x1 = e8m0_to_f32((sx >> (sh + 16)) & 255u);
  }
  c = mma_bf16(e4m3_bf16(w.a.x, w.a.y, w0), e4m3_bf16(x.a.x, x.a.y, x0), c);
  c = mma_bf16(e4m3_bf16(w.a.z, w.a.w, w0), e4m3_bf16(x.a.z, x.a.w, x0), c);
  c = mma_bf16(e4m3_bf16(w.b.x, w.b.y, w1), e4m3_bf16(x.b.x, x.b.y, x1), c);
  return mma_bf16(e4m3_bf16(w.b.z, w.b.w, w1), e4m3_bf16(x.b.z, x.b.w, x1), c);
}

// exp(z) by the hardware exp2 (1 ulp), the rounding of z log2(e) put back:
// within 2 ulp where the result lies in the normal range.  From 2^128 on exp2
// is infinite and nothing is put back: infinity and a correction below zero
// would be NaN.
__device__ __forceinline__ float exp_f32(float z) {
  const float hi = z * 1.44269502f;
  const float lo = fmaf(z, 1.44269502f, -hi) + z * 1.92596303e-8f;  // log2(e) = 1.44269502 + 1.92596303e-8
  const float e = __builtin_amdgcn_exp2f(hi);
  return fabsf(hi) < 128.f ? fmaf(e, lo * 0.693147182f, e) : e;  // past the range: 0 or infinity
}

// The activation in fp32.  GELU's two forms as z * sigmoid(2 u) and with
// erfc: no cancellation for negative z.
template <int FN>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (FN == MOE_FN_SILU) return z * __builtin_amdgcn_rcpf(1.0f + exp_f32(-z));
  if constexpr (FN == MOE_FN_GELU_TANH)
    return z * __builtin_amdgcn_rcpf(1.0f + exp_f32(-1.5957691216057308f * fmaf(0.044715f * z * z, z, z)));
  if constexpr (FN == MOE_FN_GELU_ERF) return 0.5f * z * erfcf(-0.70710678118654752f * z);
  if constexpr (FN == MOE_FN_RELU) return z < 0.f ? 0.f : z;
  return z;
}

__device__ __forceinline__ float act_fn(float z, int fn) {
  switch (fn) {
    case MOE_FN_SILU: return act_of<MOE_FN_SILU>(z);
    case MOE_FN_GELU_TANH: return act_of<MOE_FN_GELU_TANH>(z);
    case MOE_FN_GELU_ERF: return act_of<MOE_FN_GELU_ERF>(z);
    case MOE_FN_RELU: return act_of<MOE_FN_RELU>(z);
    default: return z;
  }
}

// One output: what its epilogue reads, then the output from its sums (g: the
// gate's or the only one, u: the up's).
template <int QM, bool GATED>
struct Epilogue {
  float sg = 1.f, su = 1.f, bg = 0.f, bu = 0.f, r = 0.f;
  __device__ __forceinline__ void load(const LinParams& P, int t, int n) {
    if constexpr (QM == MOE_Q_FP8) {
      const float xs = static_cast<const float*>(P.xs)[t];
      sg = xs * static_cast<const float*>(P.ws)[n];
      if (GATED) su = xs * static_cast<const float*>(P.ws)[P.N + n];
    }
    if (P.bias) {
      bg = P.bias[n];
      if (GATED) bu = P.bias[P.N + n];
    }
    if (P.res) r = bf16_to_f32(P.res[(int64_t)t * P.ldr + n]);
  }
  __device__ __forceinline__ float finish(const LinParams& P, float g, float u) const {
    float y = act_fn(fmaf(g, sg, bg), P.fn);
    if (GATED) y *= fmaf(u, su, bu);
    return y + r;
  }
};

__device__ __forceinline__ void put(const LinParams& P, int t, int n, float y) {
  if (P.out_f32) static_cast<float*>(P.out)[(int64_t)t * P.ldo + n] = y;
  else static_cast<uint16_t*>(P.out)[(int64_t)t * P.ldo + n] = f32_to_bf16_rne(y);
}

// The tile kernel (linear_tile.hip).  False: the call's strides do not fit it.
bool linear_tile_fits(const LinParams& P);
// Its workspace: 0 unless K is split.  kb: bytes of a row; exact: fp32 sums
// of 8-bit operands (fp32 outputs).
size_t linear_tile_workspace(int T, int R, int kb, bool exact);
void launch_linear_tile(const LinParams& P, int qm, void* workspace, hipStream_t s);

}  // namespace moe
