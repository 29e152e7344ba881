// Scored routing (gfx950, wave64): softmax or sigmoid scores, a balancing
// bias, groups of experts, top-k and the weights, and the permutation behind
// it.
//
// Method: as for the plain routing (route.hip); the rule is this library's
// reading (include/moe.h).
//
// The choice has to be the rule's in 64 bits, but 64-bit keys of every expert
// would be most of the work.  So a row is chosen by 32-bit keys first, and
// every comparison that decided something is checked against a bound of its
// error.  Groups whose place is open are ranked again in 64 bits, and so are
// the last places taken and their neighbours; a row that more than 16
// candidates are open for, or that holds equal words, is chosen again whole
// by one wave with 64-bit keys.
//
// Fast choice: LR lanes a row (64 / LR rows a wave), NPL consecutive experts a
// lane.  A lane sorts its keys once (a Batcher network on 32-bit words that
// carry the expert's place in the lane in their last bits), so a round of the
// top-k is a maximum over the lanes' first words (DPP) and a shift in the lane
// that had it.  Bound: VALU issue and the latency of dependent cross-lane
// steps (the logits' bytes need a tenth of the time), for few rows a chain of
// one memory latency, the rounds and the scan.  Kernel times at 256 experts
// in 8 groups, k = 8: one token 7.4 us; 16384 tokens 27 us for the rows, 5 + 4
// for the permutation; 4099 tokens of 128 experts without groups 10 + 5 + 4.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "route_hook.h"
#include "topk.h"
#include "wave.h"

namespace {

using namespace moe;

// Threads of a workgroup at most: 1024 (128 registers a lane) while a lane's
// keys fit them, else 512 or 256.  No kernel here spills
// vector registers or calls: a register saved where a branch has switched
// lanes off is lost to them (a CPU test checks the compiled code).
template <int LR, int NPL>
constexpr int kMaxThreads = NPL > 16 ? 256 : (NPL >= 8 ? 512 : 1024);

constexpr int kChunk = 64;  // tokens of a chunk of the permutation at most: a bit each of an expert's 64-bit mask

struct RouterP {
  const float* bias;
  float scale;
  int sigmoid, n_group, topk_group, top2, renorm;
  int gs;        // experts a group
  int lg, lgs;   // lanes a group (a power of two), its logarithm
  int vec;       // rows and groups in whole 16-byte pieces
};

// ------------------------------------------------------------------ 64 bits

// Order-preserving map of a double to uint64: larger value -> larger key, -0
// folded onto +0, NaN 1 (below -inf); 0 is left for "no expert".
__device__ __forceinline__ uint64_t rank64(double v) {
  uint64_t u = (uint64_t)__double_as_longlong(v);
  if (v != v) return 1ull;
  if ((u << 1) == 0) u = 0;
  return ((u >> 63) ? ~u : (u | 0x8000000000000000ull)) + 1ull;
}

// The value of a key in a group's sum: NaN and "no expert" count as -inf.
__device__ __forceinline__ double unrank64(uint64_t k) {
  if (k <= 1ull) return -INFINITY;
  const uint64_t u = k - 1ull;
  return __longlong_as_double((long long)((u >> 63) ? u & 0x7FFFFFFFFFFFFFFFull : ~u));
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
  const uint32_t hi = (uint32_t)(v >> 32);
  const uint32_t mh = wave_max_u32(hi);
  const uint32_t ml = wave_max_u32(hi == mh ? (uint32_t)v : 0u);
  return ((uint64_t)mh << 32) | ml;
}

__device__ __forceinline__ double sigmoid64(double l) { return l != l ? 0.0 : 1.0 / (1.0 + exp(-l)); }

// exp(d) for d <= 0 within 2^-41 of it: 2^n times the Taylor sum of degree 10
// on |r| <= ln 2 / 2 (next term 2^-42).  From -746 down (-inf among it) 0.
__device__ __forceinline__ double exp_neg64(double d) {
  const double x = fmax(d, -746.0);
  const double n = rint(x * 1.4426950408889634);
  double r = fma(n, -0.6931471805599453, x);
  r = fma(n, -2.3190468138462996e-17, r);  // ln 2 = 0.6931471805599453 + 2.3190468138462996e-17
  double p = 2.755731922398589e-7;         // 1 / 10!
  p = fma(p, r, 2.755731922398589e-6);
  p = fma(p, r, 2.48015873015873e-5);
  p = fma(p, r, 1.984126984126984e-4);
  p = fma(p, r, 1.3888888888888889e-3);
  p = fma(p, r, 8.333333333333333e-3);
  p = fma(p, r, 4.1666666666666664e-2);
  p = fma(p, r, 1.6666666666666666e-1);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return ldexp(p, (int)n);
}

// The softmax numerator exp(l - m), as unnorm() of the plain routing: m is
// the largest logit, NaN counts for nothing.  For the weights' denominator;
// keys take exp() itself (unnorm64_key).
__device__ __forceinline__ double unnorm64(float l, float m) {
  return l != l ? 0.0 : (l == m ? 1.0 : exp_neg64((double)l - (double)m));
}

__device__ __forceinline__ double unnorm64_key(float l, float m) {
  return l != l ? 0.0 : (l == m ? 1.0 : exp((double)l - (double)m));
}

// rank_bits without branches.
__device__ __forceinline__ uint32_t rank32(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);  // -0 -> +0
  const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return v != v ? 0u : k;
}

__device__ __forceinline__ float unrank32(uint32_t k) {  // of rank_bits
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// ------------------------------------------------------------------ lanes of a row

template <int LR>
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
  v = max(v, dpp_u32<kDppQuadXor1>(v));
  v = max(v, dpp_u32<kDppQuadXor2>(v));
  v = max(v, dpp_u32<kDppRowHalfMirror>(v));
  v = max(v, dpp_u32<kDppRowMirror>(v));
  if constexpr (LR > 16) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(a[0], a[1]);
  }
  if constexpr (LR > 32) {
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(b[0], b[1]);
  }
  return v;
}

template <int LR>
__device__ __forceinline__ float row_sum_f32(float v) {
  v += dpp_f32<kDppQuadXor1>(v);
  v += dpp_f32<kDppQuadXor2>(v);
  v += dpp_f32<kDppRowHalfMirror>(v);
  v += dpp_f32<kDppRowMirror>(v);
  if constexpr (LR > 16) v = sum_rowpair(v);
  if constexpr (LR > 32) v = sum_halves(v);
  return v;
}

template <int LR>
__device__ __forceinline__ double row_sum_f64(double v) {
#pragma unroll
  for (int o = 1; o < LR; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// The softmax denominator of a row for its keys, from the lanes' parts of it in LDS.
template <int LR>
__device__ __forceinline__ double softmax_den64(const float* lg, int base, int have, float m) {
  double part = 0.0;
#pragma unroll 1
  for (int i = 0; i < have; ++i) part += unnorm64_key(lg[base + i], m);
  return row_sum_f64<LR>(part);
}

// A group's two largest, from two disjoint parts of it.
__device__ __forceinline__ void merge2(float& a, float& b, float a2, float b2) {
  const float lo = fminf(a, a2);
  a = fmaxf(a, a2);
  b = fmaxf(lo, fmaxf(b, b2));
}

// Batcher's odd-even merge sort of N words, descending.
template <int N>
__device__ __forceinline__ void sort_desc(uint32_t (&s)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t hi = max(s[i + j], s[i + j + q]), lo = min(s[i + j], s[i + j + q]);
            s[i + j] = hi;
            s[i + j + q] = lo;
          }
}

// The choice of one row by a whole wave with 64-bit keys: ids[0 .. k).  lg:
// the row's logits; den: the softmax denominator, m its largest logit.
template <int NPER>
__device__ __forceinline__ void choose64(const RouterP& R, const float* lg, int E, int k, float m, double den,
                                                   int32_t* ids) {
  const int lane = threadIdx.x & 63;
  uint64_t rk[NPER];   // keys
  uint64_t gr[NPER];   // what the groups are ranked by
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const int e = lane + 64 * i;
    rk[i] = gr[i] = 0;
    if (e < E) {
      const float l = lg[e];
      const double s = l != l ? (double)l : (R.sigmoid ? sigmoid64((double)l) : unnorm64_key(l, m) / den);
      const double key = R.bias ? s + (double)R.bias[e] : (double)l;
      rk[i] = rank64(key);
      gr[i] = R.bias || !R.top2 ? rk[i] : rank64(s);
    }
  }
  if (R.n_group > 1) {
    // lane g keeps group g's rank
    uint64_t mine = 0;
    for (int g = 0; g < R.n_group; ++g) {
      uint64_t best = 0, two[NPER];
      bool taken = false;
#pragma unroll
      for (int i = 0; i < NPER; ++i) {
        const int e = lane + 64 * i;
        two[i] = e < E && e / R.gs == g ? gr[i] : 0;
        best = max(best, two[i]);
      }
      best = wave_max_u64(best);
      uint64_t rank = best;
      if (R.top2 && R.gs > 1) {
        // without one of the largest (which one does not matter), the largest again
        uint64_t b2 = 0;
#pragma unroll
        for (int i = 0; i < NPER; ++i) {
          const uint64_t has = __ballot(!taken && two[i] == best);
          if (has) {
            // the lowest lane of the lowest slot that holds it gives it up, once for the wave
            if (lane == __builtin_ctzll(has)) two[i] = 0;
            taken = true;
          }
          b2 = max(b2, two[i]);
        }
        b2 = wave_max_u64(b2);
        rank = rank64(unrank64(best) + unrank64(b2));
      }
      if (lane == g) mine = rank;
    }
    uint64_t live = 0;
    for (int r = 0; r < R.topk_group; ++r) {
      const uint64_t mx = wave_max_u64(mine);
      const int g = __builtin_ctzll(__ballot(lane < R.n_group && mine == mx));
      live |= 1ull << g;
      if (lane == g) mine = 0;
    }
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((live >> (e / R.gs)) & 1)) rk[i] = 0;
    }
  }
  for (int r = 0; r < k; ++r) {
    uint64_t lm = rk[0];
#pragma unroll
    for (int i = 1; i < NPER; ++i) lm = max(lm, rk[i]);
    const uint64_t mx = wave_max_u64(lm);
    int ws = 0;
    uint64_t bw = 1;
#pragma unroll
    for (int i = NPER - 1; i >= 0; --i) {
      const uint64_t b = __ballot(rk[i] == mx);
      ws = b ? i : ws;
      bw = b ? b : bw;
    }
    const int wl = __builtin_ctzll(bw);
#pragma unroll
    for (int i = 0; i < NPER; ++i) rk[i] = i == ws && lane == wl ? 0ull : rk[i];
    if (lane == 0) ids[r] = wl + 64 * ws;
  }
}

// One row by LR >= 16 lanes (lane p of it): ids[0 .. k) and, in lane j < k, the
// weight of position j.  bias_s: the bias in LDS.  lg: E floats of LDS, the row's own, filled here; the
// wave's rows have theirs side by side, and so have the ids (kRouteMaxK words a row).
template <int LR, int NPL>
__device__ __forceinline__ float route_row(const RouterP& R, const float* __restrict__ row, bool valid, int E, int k,
                                           const float* bias_s, float* lg, int32_t* ids) {
  constexpr int NPER = LR * NPL / 64 > 16 ? 16 : LR * NPL / 64;  // E <= 1024
  constexpr float kCut = NPL * 0x1p-22f;                        // a word is cut by less than half of this
  const int lane = threadIdx.x & 63, p = lane & (LR - 1);
  const int group = p >> R.lgs, in_group = (p & (R.lg - 1)) * NPL;  // this lane's group and first place in it
  const int base = group * R.gs + in_group;
  const int have = group < R.n_group ? min(max(R.gs - in_group, 0), NPL) : 0;  // experts of this lane
  // the row to LDS in order (a lane's own experts lie too far from its
  // neighbours' for loads of its own), then each lane's from there
  if (R.vec) {
    for (int c = 4 * p; c < E; c += 4 * LR)
      *reinterpret_cast<float4*>(lg + c) =
          valid ? *reinterpret_cast<const float4*>(row + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
    for (int c = p; c < E; c += LR) lg[c] = valid ? row[c] : 0.f;
  }
  __builtin_amdgcn_wave_barrier();  // a wave's LDS accesses keep their order
  float val[NPL], bs[NPL];
  if (R.vec) {
#pragma unroll
    for (int i = 0; i < NPL; i += 4) {
      const int at = i < have ? base + i : 0;  // groups are whole pieces: all four or none
      const float4 v = *reinterpret_cast<const float4*>(lg + at);
      val[i] = v.x, val[i + 1] = v.y, val[i + 2] = v.z, val[i + 3] = v.w;
      if (R.bias) {
        const float4 u = *reinterpret_cast<const float4*>(bias_s + at);
        bs[i] = u.x, bs[i + 1] = u.y, bs[i + 2] = u.z, bs[i + 3] = u.w;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      val[i] = i < have ? lg[base + i] : 0.f;
      if (R.bias) bs[i] = i < have ? bias_s[base + i] : 0.f;
    }
  }

  // softmax: largest logit and denominator, in 32 bits for the keys; in 64
  // bits where a weight divides by it
  float m = 0.f, inv = 1.f;
  double den = 1.0;
  if (!R.sigmoid) {
    uint32_t mk = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) mk = max(mk, i < have ? rank32(val[i]) : 0u);
    mk = row_max_u32<LR>(mk);
    m = mk == 0 ? 0.f : unrank32(mk);
    if (R.bias || R.top2) {
      float part = 0.f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const float e = val[i] == m ? 1.f : __expf(val[i] - m);
        part += i < have && val[i] == val[i] ? e : 0.f;
      }
      inv = 1.0f / row_sum_f32<LR>(part);
    }
    if (!R.renorm) {
      double part64 = 0.0;
#pragma unroll 2
      for (int i = 0; i < NPL; ++i) {  // from LDS again: unrolled whole, its temporaries would cost a wave's place
        const float l = i < have ? lg[base + i] : NAN;
        const double d = l == m ? 0.0 : (double)l - (double)m;
        part64 += l == l ? exp_neg64(d) : 0.0;
      }
      den = row_sum_f64<LR>(part64);
    }
  }
  // keys (a NaN logit: NaN), and the two largest of what the groups are ranked by
  float key[NPL], a = -INFINITY, b = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    float sc = val[i];
    if (R.bias || R.top2)
      sc = R.sigmoid ? __builtin_amdgcn_rcpf(1.0f + __expf(-val[i]))
                     : (val[i] == m ? inv : __expf(val[i] - m) * inv);
    key[i] = R.bias ? sc + bs[i] : val[i];
    const float v = i < have ? (R.bias ? key[i] : sc) : -INFINITY;
    nan = nan || v != v;
    b = fmaxf(b, fminf(a, v));
    a = fmaxf(a, v);
  }
  // what a comparison of two keys may be off by beside their own rounding: a
  // score's error, below 2^-21 under sigmoid (four roundings of a value below
  // 1) and 2^-19 of the largest under softmax (1 / den, its sum of up to 32
  // terms a lane)
  const float s_err = R.bias ? (R.sigmoid ? 0x1p-20f : inv * 0x1p-18f) : 0.f;
  bool live = group < R.n_group;
  if (R.n_group > 1) {
    if (R.lg > 1) merge2(a, b, dpp_f32<kDppQuadXor1>(a), dpp_f32<kDppQuadXor1>(b));
    if (R.lg > 2) merge2(a, b, dpp_f32<kDppQuadXor2>(a), dpp_f32<kDppQuadXor2>(b));
    if (R.lg > 4) merge2(a, b, dpp_f32<kDppRowHalfMirror>(a), dpp_f32<kDppRowHalfMirror>(b));
    if (R.lg > 8) merge2(a, b, dpp_f32<kDppRowMirror>(a), dpp_f32<kDppRowMirror>(b));
    if (LR > 16 && R.lg > 16) merge2(a, b, __shfl_xor(a, 16), __shfl_xor(b, 16));
    const float rank = R.top2 && R.gs > 1 ? a + b : a;
    // its place: the groups that are larger, or equal and lower.  Logits
    // compare exactly; scores alone are off by 2^-17 of themselves at most
    // (exp of a difference of up to 88).  Two keys of opposite signs were each
    // rounded at their own size, beside which their sum may be small: the
    // row's largest such loss counts for all its groups.
    const bool exact = !R.top2 && !R.bias;
    float size = fabsf(rank);
    if (R.bias && R.top2) {
      const float lost = a > 0.f && b < 0.f && b > -INFINITY ? 2.f * fminf(a, -b) : 0.f;  // |a| + |b| - |a + b|
      size += __uint_as_float(row_max_u32<LR>(__float_as_uint(lost)));
    }
    const float tol = 2.f * s_err + (R.bias ? 0x1p-19f : 0x1p-16f) * size + 0x1p-100f;
    int above = 0, maybe = 0;  // groups surely before this one, and possibly
    const int lanes = R.n_group << R.lgs, first = lane - p;
    for (int d = 1; d < R.n_group; ++d) {
      int q = p + (d << R.lgs);
      q = q >= lanes ? q - lanes : q;
      const float other = __shfl(rank, first + (q & (LR - 1)));
      const bool before = other > rank || (other == rank && q < p);
      above += exact ? before : other - rank > tol;
      maybe += exact ? before : !(rank - other > tol);
    }
    live = live && maybe < R.topk_group;
    // rows whose groups are open (a NaN among the keys leaves the ranks above
    // without meaning): their groups in 64 bits
    const uint64_t open =
        __ballot(valid && group < R.n_group && (nan || (maybe >= R.topk_group && above < R.topk_group)));
    if (open != 0ull) {
      const uint64_t row_mask = (LR == 64 ? ~0ull : (1ull << (LR & 63)) - 1ull) << (lane - p);
      double den64 = 1.0;
      if (!R.sigmoid && !exact) den64 = softmax_den64<LR>(lg, base, have, m);
      double a64 = -INFINITY, b64 = -INFINITY;
      int real = 0;
#pragma unroll 1
      for (int i = 0; i < have; ++i) {
        const float l = lg[base + i];
        double v = (double)l;
        if (!exact) {
          v = l != l ? v : (R.sigmoid ? sigmoid64((double)l) : unnorm64_key(l, m) / den64);
          if (R.bias) v += (double)bias_s[base + i];
        }
        real |= v == v;
        v = v != v ? -INFINITY : v;
        b64 = fmax(b64, fmin(a64, v));
        a64 = fmax(a64, v);
      }
      for (int o = 1; o < R.lg; o <<= 1) {
        const double a2 = __shfl_xor(a64, o), b2 = __shfl_xor(b64, o);
        real |= __shfl_xor(real, o);
        b64 = fmax(fmin(a64, a2), fmax(b64, b2));
        a64 = fmax(a64, a2);
      }
      const uint64_t mine = R.top2 && R.gs > 1 ? rank64(a64 + b64) : (real ? rank64(a64) : 1ull);
      int place = 0;
      for (int d = 1; d < R.n_group; ++d) {
        int q = p + (d << R.lgs);
        q = q >= lanes ? q - lanes : q;
        const int src = first + (q & (LR - 1));
        const uint64_t other =
            ((uint64_t)(uint32_t)__shfl((int)(mine >> 32), src) << 32) | (uint32_t)__shfl((int)(uint32_t)mine, src);
        place += other > mine || (other == mine && q < p);
      }
      if (open & row_mask) live = group < R.n_group && place < R.topk_group;
    }
  }

  // words: the key's order with its last bits replaced by the place in the lane (the lower place the larger); a NaN
  // key takes the lowest of them that is not 0, the word of no expert
  uint32_t w[NPL];
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const uint32_t k1 = (max(rank32(key[i]), (uint32_t)NPL) & ~(uint32_t)(NPL - 1)) | (uint32_t)(NPL - 1 - i);
    w[i] = i < have && live ? k1 : 0u;
  }
  sort_desc<NPL>(w);
  // Candidates in the words' order: the first k, and after them while one
  // could still belong before the last (lanes 0 .. 15 hold one each below).
  float last = 0.f;
  int took = 0, n = kRouteMaxK + 1;  // n: the row's candidates, once its end is certain
  bool near = false;
  for (int r = 0; r <= kRouteMaxK; ++r) {
    const uint32_t mx = row_max_u32<LR>(w[0]);
    const float v = unrank32(mx & ~(uint32_t)(NPL - 1));
    const bool close = r > 0 && !(last - v > s_err + kCut * fmaxf(fabsf(last), fabsf(v)));
    if (r >= k && (mx == 0u || !close || !valid)) n = min(n, r);  // (a row past the batch is all ties)
    if (r >= k && __ballot(n > r) == 0ull) break;  // every row of the wave ends here
    if (r == kRouteMaxK) break;
    near = near || (close && r < n);
    last = v;
    const bool hit = w[0] == mx;  // more lanes than one: equal words, counted below
    if (hit && r < n) ids[r] = base + NPL - 1 - (int)(mx & (NPL - 1));
    took += hit && r < n;
    // by bits (v_bfi): of selects between neighbours the compiler makes an indexed array, 430 instructions a round
    const uint32_t up = hit ? ~0u : 0u;
#pragma unroll
    for (int i = 0; i + 1 < NPL; ++i) w[i] = (w[i + 1] & up) | (w[i] & ~up);
    w[NPL - 1] &= ~up;
  }
  const bool unsure = row_sum_f32<LR>((float)took) != (float)n || n > kRouteMaxK;
  near = near && !unsure;
  // rows whose order is open among their candidates alone: those in 64 bits
  if (__ballot(near && valid) != 0ull) {
    double den64 = 1.0;
    if (R.bias && !R.sigmoid) den64 = softmax_den64<LR>(lg, base, have, m);
    const int id = p < n && p < kRouteMaxK && near ? ids[p] : 0;
    uint64_t mine = 0;
    if (p < n && p < kRouteMaxK && near) {
      const float l = lg[id];
      double key64 = (double)l;
      if (R.bias)
        key64 = (l != l ? key64 : (R.sigmoid ? sigmoid64((double)l) : unnorm64_key(l, m) / den64)) + (double)bias_s[id];
      mine = rank64(key64);
    }
    int place = 0;
    for (int q = 0; q < kRouteMaxK; ++q) {
      const uint64_t other = ((uint64_t)(uint32_t)__shfl((int)(mine >> 32), lane - p + q) << 32) |
                             (uint32_t)__shfl((int)(uint32_t)mine, lane - p + q);
      const int oid = __shfl(id, lane - p + q);
      place += other > mine || (other == mine && oid < id);
    }
    if (mine != 0 && place < k) ids[place] = id;
  }
  // rows whose choice could differ in 64 bits: again, one wave each
  uint64_t again = __ballot(unsure && valid);
  while (again) {
    const int l0 = __builtin_ctzll(again) & ~(LR - 1);
    again &= LR == 64 ? 0ull : ~(((1ull << (LR & 63)) - 1) << l0);
    const float mr = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(m), l0));
    const int seg = l0 / LR;
    const float* lrow = lg + (seg - (lane / LR)) * E;
    int32_t* irow = ids + (seg - (lane / LR)) * kRouteMaxK;
    double dr = 1.0;
    if (!R.sigmoid && (R.bias || R.top2)) {
      double part = 0.0;
      for (int e = lane; e < E; e += 64) part += unnorm64_key(lrow[e], mr);
      dr = row_sum_f64<64>(part);
    }
    choose64<NPER>(R, lrow, E, k, mr, dr, irow);
  }
  // weights: lane j < k of the row, in 64 bits
  double s = 0.0;
  if (p < k && valid) {
    const float l = lg[ids[p]];
    s = R.sigmoid ? sigmoid64((double)l) : unnorm64(l, m);
  }
  if (R.renorm) den = row_sum_f64<16>(s);  // k <= 16: lanes 0 .. 15 of the row
  return (float)((den > 0.0 ? s / den : 1.0 / k) * (double)R.scale);
}

// `rows` rows from token t0 on by the workgroup: ids to LDS (ids_s [64][kRouteMaxK])
// and memory, weights to memory.  lg_s: E floats of the bias, then E for each row in work.
template <int LR, int NPL>
__device__ __forceinline__ void route_rows(const RouterP& R, const float* __restrict__ logits, int t0, int rows, int E,
                                           int k, float* lg_s, int32_t* ids_s, int32_t* __restrict__ ids,
                                           float* __restrict__ wts) {
  constexpr int RPW = 64 / LR;  // rows a wave
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, rpp = (int)(blockDim.x >> 6) * RPW;
  const int slot = wave * RPW + lane / LR, p = lane & (LR - 1);
  if (R.bias) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) lg_s[e] = R.bias[e];
    __syncthreads();
  }
  for (int r0 = 0; r0 < rows; r0 += rpp) {
    const int r = r0 + slot;
    if (r0 + wave * RPW >= rows) break;  // whole waves
    const bool valid = r < rows;
    const float w = route_row<LR, NPL>(R, logits + (size_t)(t0 + (valid ? r : 0)) * E, valid, E, k, lg_s,
                                       lg_s + (slot + 1) * E, ids_s + r * kRouteMaxK);
    if (p < k && valid) {
      ids[(size_t)(t0 + r) * k + p] = ids_s[r * kRouteMaxK + p];
      wts[(size_t)(t0 + r) * k + p] = w;
    }
  }
}

template <int LR, int NPL>
__global__ __launch_bounds__(256) void k_route_scored(RouterP R, const float* __restrict__ logits, int T, int E, int k,
                                                      int32_t* __restrict__ ids, float* __restrict__ wts) {
  extern __shared__ __align__(16) float lg_s[];
  constexpr int ROWS = 4 * (64 / LR);
  __shared__ int32_t ids_s[ROWS * kRouteMaxK];
  const int t0 = (int)blockIdx.x * ROWS;
  route_rows<LR, NPL>(R, logits, t0, min(ROWS, T - t0), E, k, lg_s, ids_s, ids, wts);
}

// ------------------------------------------------------------------ permutation
//
// In chunks of 16, 32 or 64 tokens.  A token takes an expert at most once, so
// an expert's rows of a chunk are the set bits of a 64-bit mask of its tokens, and
// the position of (t, e) is offsets[e] + (rows of e in earlier chunks) + (set
// bits below t): no sort and no order-dependent atomics.

// tmask[e] of a chunk (cleared before) from its ids (LDS, kRouteMaxK words a token).
__device__ __forceinline__ void set_masks(const int32_t* ids, int n, int k, uint64_t* tmask) {
  for (int f = threadIdx.x; f < n; f += blockDim.x) {
    const int t = f / k;
    atomicOr(reinterpret_cast<unsigned long long*>(&tmask[ids[t * kRouteMaxK + f - t * k]]), 1ull << t);
  }
}

// Exclusive scan over the experts of cnt(e) by the workgroup; calls
// out(e, exclusive, count) and returns the total.  wsum: LDS of a word a wave.
template <typename C, typename O>
__device__ __forceinline__ int scan_experts(int E, int32_t* wsum, C cnt, O out) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, nt = blockDim.x, nw = nt >> 6;
  const int per = (E + nt - 1) / nt;
  int run = 0;
  for (int i = 0; i < per; ++i)
    if (tid * per + i < E) run += cnt(tid * per + i);
  int incl = run;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int base = incl - run, total = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < wave) base += wsum[w];
    total += wsum[w];
  }
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e < E) {
      const int c = cnt(e);
      out(e, base, c);
      base += c;
    }
  }
  return total;
}

// Places a chunk's flat indices [f0, f0 + n): off[e] is the position of e's first row of the chunk.
__device__ __forceinline__ void place(const int32_t* ids, int f0, int n, int k, const uint64_t* tmask,
                                      const int32_t* off, int32_t* __restrict__ perm, int32_t* __restrict__ inv) {
  for (int f = threadIdx.x; f < n; f += blockDim.x) {
    const int t = f / k, e = ids[t * kRouteMaxK + f - t * k];
    const int pos = off[e] + (int)__popcll(tmask[e] & ((1ull << t) - 1ull));
    perm[pos] = f0 + f;
    inv[f0 + f] = pos;
  }
}

// Up to 64 tokens: everything in one workgroup.  LDS: E masks, E offsets, then the rows' logits.
template <int LR, int NPL>
__global__ __launch_bounds__((kMaxThreads<LR, NPL>)) void k_route_one(RouterP R, const float* __restrict__ logits, int T, int E, int k,
                                                    int32_t* __restrict__ ids, float* __restrict__ wts,
                                                    int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                    int32_t* __restrict__ perm, int32_t* __restrict__ inv) {
  extern __shared__ __align__(16) uint64_t tmask[];
  __shared__ int32_t ids_s[kChunk * kRouteMaxK], wsum[16];
  int32_t* off = reinterpret_cast<int32_t*>(tmask + E);
  float* lg_s = reinterpret_cast<float*>(off + E);
  for (int e = threadIdx.x; e < E; e += blockDim.x) tmask[e] = 0ull;
  route_rows<LR, NPL>(R, logits, 0, T, E, k, lg_s, ids_s, ids, wts);
  __syncthreads();
  set_masks(ids_s, T * k, k, tmask);
  __syncthreads();
  scan_experts(
      E, wsum, [&](int e) { return (int)__popcll(tmask[e]); },
      [&](int e, int base, int c) {
        off[e] = base;
        counts[e] = c;
        offsets[e] = base;
      });
  if (threadIdx.x == 0) offsets[E] = T * k;
  __syncthreads();
  place(ids_s, 0, T * k, k, tmask, off, perm, inv);
}

// Longer batches, first pass: a chunk's rows (C tokens), and the counts of a
// whole chunk to the chunk's own part of inv (E <= C k words; the last pass
// replaces it).
template <int LR, int NPL>
__global__ __launch_bounds__((kMaxThreads<LR, NPL>)) void k_route_chunk(RouterP R, const float* __restrict__ logits,
                                                                       int T, int E, int k, int C,
                                                                       int32_t* __restrict__ ids,
                                                                       float* __restrict__ wts,
                                                                       int32_t* __restrict__ inv) {
  extern __shared__ __align__(16) int32_t cnt[];  // [E], then the bias and the rows' logits
  __shared__ int32_t ids_s[kChunk * kRouteMaxK];
  const int t0 = (int)blockIdx.x * C, rows = min(C, T - t0);
  for (int e = threadIdx.x; e < E; e += blockDim.x) cnt[e] = 0;
  route_rows<LR, NPL>(R, logits, t0, rows, E, k, reinterpret_cast<float*>(cnt + E), ids_s, ids, wts);
  if (rows < C) return;
  __syncthreads();
  for (int f = threadIdx.x; f < rows * k; f += blockDim.x)
    atomicAdd(&cnt[ids_s[f / k * kRouteMaxK + f % k]], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) inv[(size_t)t0 * k + e] = cnt[e];
}

// Second pass, a workgroup an expert: the chunks' counts become the rows of
// the earlier chunks; counts[e] their sum, with the last, partial chunk's.
__global__ __launch_bounds__(256) void k_chunk_scan(const int32_t* __restrict__ ids, int T, int k, int C,
                                                    int32_t* __restrict__ inv, int32_t* __restrict__ counts) {
  __shared__ int32_t wsum[4];
  const int e = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int whole = T / C;
  int run = 0;
  for (int c0 = 0; c0 < whole; c0 += 256) {
    const int c = c0 + tid;
    int32_t* at = inv + (size_t)c * C * k + e;
    const int n = c < whole ? *at : 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int u = __shfl_up(incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 63) wsum[wave] = incl;
    __syncthreads();
    int base = run;
    for (int w = 0; w < 4; ++w) {
      if (w < wave) base += wsum[w];
      run += wsum[w];
    }
    if (c < whole) *at = base + incl - n;
    __syncthreads();
  }
  int mine = 0;  // the partial chunk's rows
  for (int f = whole * C * k + tid; f < T * k; f += 256) mine += ids[f] == e;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) mine += __shfl_xor(mine, o);
  if (lane == 0) wsum[wave] = mine;
  __syncthreads();
  if (tid == 0) counts[e] = run + wsum[0] + wsum[1] + wsum[2] + wsum[3];
}

// Third pass, a workgroup a chunk.  LDS: E masks, E offsets.
__global__ __launch_bounds__(512) void k_chunk_place(const int32_t* __restrict__ ids, int T, int E, int k, int C,
                                                     const int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                     int32_t* __restrict__ perm, int32_t* __restrict__ inv) {
  extern __shared__ uint64_t tmask[];
  __shared__ int32_t wsum[8], ids_s[kChunk * kRouteMaxK];
  int32_t* off = reinterpret_cast<int32_t*>(tmask + E);
  const int t0 = (int)blockIdx.x * C, rows = min(C, T - t0), n = rows * k, f0 = t0 * k;
  for (int e = threadIdx.x; e < E; e += blockDim.x) tmask[e] = 0ull;
  for (int f = threadIdx.x; f < n; f += blockDim.x) ids_s[f / k * kRouteMaxK + f % k] = ids[f0 + f];
  __syncthreads();
  set_masks(ids_s, n, k, tmask);
  __syncthreads();
  scan_experts(
      E, wsum, [&](int e) { return counts[e]; },
      [&](int e, int base, int c) {
        // a partial chunk is the last one: its rows end the expert's
        off[e] = base + (rows == C ? inv[(size_t)f0 + e] : c - (int)__popcll(tmask[e]));
        if (blockIdx.x == 0) offsets[e] = base;
      });
  if (blockIdx.x == 0 && threadIdx.x == 0) offsets[E] = T * k;
  __syncthreads();  // every count of the chunk is read: its part of inv takes the positions
  place(ids_s, f0, n, k, tmask, off, perm, inv);
}

// ------------------------------------------------------------------ host

moe_status check_router(const char* who, const moe_router* r, int T, int E, int k) {
  MOE_CHECK_ARG(r, "%s: null router", who);
  // T: four rows a workgroup of 256 threads at least, in a grid below 2^32 threads
  MOE_CHECK_ARG(T >= 0 && T < (1 << 25) && E >= 1 && E <= 1024, "%s: bad sizes T=%d E=%d (T < 2^25, E <= 1024)", who, T,
                E);
  MOE_CHECK_ARG(r->score == MOE_SCORE_SOFTMAX || r->score == MOE_SCORE_SIGMOID, "%s: bad score %d", who, r->score);
  MOE_CHECK_ARG(r->group_rank == MOE_GROUP_MAX || r->group_rank == MOE_GROUP_TOP2, "%s: bad group_rank %d", who,
                r->group_rank);
  MOE_CHECK_ARG(r->n_group >= 1 && r->n_group <= 64 && E % r->n_group == 0,
                "%s: n_group=%d must divide E=%d and be at most 64", who, r->n_group, E);
  MOE_CHECK_ARG(r->topk_group >= 1 && r->topk_group <= r->n_group, "%s: topk_group=%d must be in [1, n_group=%d]", who,
                r->topk_group, r->n_group);
  static_assert(kScoredMaxK == kRouteMaxK, "ids and words of a row in LDS");
  const int most = router_most(*r, E);
  MOE_CHECK_ARG(k >= 1 && k <= most, "%s: k=%d must be in [1, min(topk_group * E / n_group, 16)] = [1, %d]", who, k,
                most);
  return MOE_OK;
}

// Whether n_group groups of gs experts fit lr lanes of npl experts, whole
// groups to a power of two of lanes; the logarithm of that in *lgs.
bool lanes_fit(int n_group, int gs, int lr, int npl, int* lgs) {
  int l = 0;
  while ((npl << l) < gs) ++l;
  *lgs = l;
  return (n_group << l) <= lr;
}

// Calls f(LR, NPL) with the shape for the router.  one: few rows in one
// workgroup, so a whole wave a row while it fits (its chain of instructions
// is the time of the call); otherwise the fewest lanes.  64 x 32 takes every
// E <= 1024 with n_group <= 64.
template <typename F>
void with_shape(RouterP& R, int E, bool one, F f) {
  auto fits = [&](int lr, int npl) {
    int l;
    if (!lanes_fit(R.n_group, R.gs, lr, npl, &l)) return false;
    R.lgs = l;
    R.lg = 1 << l;
    return true;
  };
  using std::integral_constant;
  if (one && fits(64, 4)) f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
  else if (fits(16, 4)) f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  else if (fits(16, 8)) f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  else if (fits(16, 16)) f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  else if (fits(32, 16)) f(integral_constant<int, 32>{}, integral_constant<int, 16>{});
  else if (fits(64, 16)) f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
  else {
    fits(64, 32);
    f(integral_constant<int, 64>{}, integral_constant<int, 32>{});
  }
}

RouterP router_params(const moe_router* r, const float* logits, int E) {
  RouterP R{};
  R.bias = r->bias;
  R.scale = r->scale;
  R.sigmoid = r->score == MOE_SCORE_SIGMOID;
  R.n_group = r->n_group;
  R.topk_group = r->topk_group;
  R.top2 = r->n_group > 1 && r->group_rank == MOE_GROUP_TOP2;
  R.renorm = r->renormalize;
  R.gs = E / r->n_group;
  R.vec = E % 4 == 0 && R.gs % 4 == 0 && ((uintptr_t)logits & 15) == 0;
  return R;
}

}  // namespace

extern "C" moe_status moe_route_scored(const moe_router* r, const float* logits, int T, int E, int k,
                                       int32_t* topk_ids, float* topk_w, moe_stream_t stream) {
  moe_status st = check_router("moe_route_scored", r, T, E, k);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  MOE_CHECK_ARG(logits && topk_ids && topk_w, "moe_route_scored: null pointer");
  RouterP R = router_params(r, logits, E);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  with_shape(R, E, T <= 64, [&](auto lr, auto npl) {
    constexpr int LR = decltype(lr)::value, NPL = decltype(npl)::value, ROWS = 4 * (64 / LR);
    const size_t lds = (size_t)(ROWS + 1) * E * sizeof(float);  // at most 20 KiB
    launch(k_route_scored<LR, NPL>, dim3((unsigned)((T + ROWS - 1) / ROWS)), dim3(256), lds, s, R, logits, T, E, k,
           topk_ids, topk_w);
  });
  MOE_LAUNCHED();
  return MOE_OK;
}

extern "C" moe_status moe_route_scored_permute(const moe_router* r, const float* logits, int T, int E, int k,
                                               int32_t* topk_ids, float* topk_w, int32_t* counts, int32_t* offsets,
                                               int32_t* perm, int32_t* inv, moe_stream_t stream) {
  moe_status st = check_router("moe_route_scored_permute", r, T, E, k);
  if (st != MOE_OK) return st;
  MOE_CHECK_ARG((long long)T * k <= kScoredMaxRows, "moe_route_scored_permute: T*k = %lld exceeds %d", (long long)T * k,
                kScoredMaxRows);
  MOE_CHECK_ARG(counts && offsets && (T == 0 || (logits && topk_ids && topk_w && perm && inv)),
                "moe_route_scored_permute: null pointer");
  RouterP R = router_params(r, logits, E);
  // the smallest chunk whose part of inv holds its counts: the most workgroups
  const int C = E <= 16 * k ? 16 : (E <= 32 * k ? 32 : kChunk);
  // A workgroup that takes its rows in several passes is late while others
  // idle: routed by a launch of its own over all CUs, then permuted.  Before
  // and after (us, k = 8): 64 tokens of 512 experts 27 -> 15, 1000 of 3 x 160
  // 63 -> 21, of 200 experts (one pass) 16 -> 15, 4000 of 320 (4 passes) 33 ->
  // 31; 4000 of 8 x 32 (one pass) 22 -> 24, 16384 of 512 41 -> 87.  A second
  // pass over short rows without groups costs less than a launch: 64 tokens
  // of 128 11.4 -> 12.1.
  int passes = 1;
  with_shape(R, E, T <= 16, [&](auto lr, auto npl) {
    const int rows = kMaxThreads<decltype(lr)::value, decltype(npl)::value> / decltype(lr)::value;
    if (decltype(npl)::value > 8 || R.n_group > 1) passes = (std::min(T, T <= kChunk ? kChunk : C) + rows - 1) / rows;
  });
  // or nothing to route, or more experts than a chunk's part of inv has words for their counts
  if (T == 0 || (T > kChunk && E > kChunk * k) || (passes > 1 && T <= 1024 * passes)) {
    st = moe_route_scored(r, logits, T, E, k, topk_ids, topk_w, stream);
    if (st != MOE_OK) return st;
    return moe_permute(topk_ids, T, k, E, counts, offsets, perm, inv, stream);
  }
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  // dynamic LDS below: at most 48 KiB (E = 1024 by 64 x 16, eight rows in work)
  if (T <= kChunk) {
    with_shape(R, E, T <= 16, [&](auto lr, auto npl) {
      constexpr int LR = decltype(lr)::value, NPL = decltype(npl)::value, RPW = 64 / LR;
      const int waves = std::min(kMaxThreads<LR, NPL> / 64, (T + RPW - 1) / RPW);
      // (at least) four waves for the scan over the experts
      const int nw = std::max(waves, std::min(4, (E + 63) / 64));
      const size_t lds = (size_t)E * 12 + (size_t)(nw * RPW + 1) * E * sizeof(float);
      launch(k_route_one<LR, NPL>, dim3(1), dim3((unsigned)(64 * nw)), lds, s, R, logits, T, E, k, topk_ids, topk_w,
             counts, offsets, perm, inv);
    });
  } else {
    const unsigned chunks = (unsigned)((T + C - 1) / C);
    with_shape(R, E, false, [&](auto lr, auto npl) {
      constexpr int LR = decltype(lr)::value, NPL = decltype(npl)::value;
      const int nt = std::min(kMaxThreads<LR, NPL>, C * LR);
      const size_t lds = (size_t)E * 4 + (size_t)(nt / LR + 1) * E * sizeof(float);
      launch(k_route_chunk<LR, NPL>, dim3(chunks), dim3((unsigned)nt), lds, s, R, logits, T, E, k, C, topk_ids, topk_w,
             inv);
    });
    launch(k_chunk_scan, dim3((unsigned)E), dim3(256), 0, s, topk_ids, T, k, C, inv, counts);
    launch(k_chunk_place, dim3(chunks), dim3(E <= 256 ? 256 : 512), (size_t)E * 12, s, topk_ids, T, E, k, C, counts,
           offsets, perm, inv);
  }
  MOE_LAUNCHED();
  return MOE_OK;
}

namespace {

moe_status route_of_cache(const moe_router* r, const float* logits, int T, int E, int k, int32_t* topk_ids,
                          float* topk_w, int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv,
                          int32_t* host_counts, uint32_t* flag, uint32_t seq, hipStream_t s) {
  moe_status st = moe_route_scored_permute(r, logits, T, E, k, topk_ids, topk_w, counts, offsets, perm, inv,
                                           reinterpret_cast<moe_stream_t>(s));
  if (st != MOE_OK || !host_counts) return st;
  const hipError_t e = launch_publish_counts(counts, E, host_counts, flag, seq, s);
  if (e != hipSuccess) return set_error(MOE_EHIP, "count handoff launch failed: %s", hipGetErrorString(e));
  return MOE_OK;
}

}  // namespace

extern "C" moe_status moe_cache_use_router(moe_cache* c, int layer, const moe_router* r) {
  MOE_CHECK_ARG(c, "moe_cache_use_router: null cache");
  int layers = 0, experts = 0;
  cache_shape(c, &layers, &experts);
  MOE_CHECK_ARG(layer >= -1 && layer < layers, "moe_cache_use_router: layer %d out of range", layer);
  if (r) {
    const moe_status st = check_router("moe_cache_use_router", r, 0, experts, 1);
    if (st != MOE_OK) return st;
  }
  cache_set_router(c, layer, r, route_of_cache);
  return MOE_OK;
}
