// Scored routing (gfx950, wave64): softmax or sigmoid scores, a balancing
// bias, groups of experts, top-k and the weights; one wave per token.
//
// Method: as for the plain routing (route.hip); the rule is this library's
// reading (include/moe.h).
#include <algorithm>

#include "common.h"
#include "topk.h"
#include "wave.h"

namespace {

using namespace moe;

struct RouterP {
  const float* bias;
  float scale;
  int sigmoid, n_group, topk_group, top2, renorm;
};

// Order-preserving map of a double to uint64: larger value -> larger key, -0
// folded onto +0, NaN 1 (below -inf); 0 is left for "no expert".
__device__ __forceinline__ uint64_t rank64(double v) {
  uint64_t u = (uint64_t)__double_as_longlong(v);
  if (v != v) return 1ull;
  if ((u << 1) == 0) u = 0;
  return ((u >> 63) ? ~u : (u | 0x8000000000000000ull)) + 1ull;
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
  const uint32_t hi = (uint32_t)(v >> 32);
  const uint32_t mh = wave_max_u32(hi);
  const uint32_t ml = wave_max_u32(hi == mh ? (uint32_t)v : 0u);
  return ((uint64_t)mh << 32) | ml;
}

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

__device__ __forceinline__ double sigmoid64(double l) { return l != l ? 0.0 : 1.0 / (1.0 + exp(-l)); }

// The softmax numerator exp(l - m), as unnorm() of the plain routing.
__device__ __forceinline__ double unnorm64(double l, double m) { return l != l ? 0.0 : (l == m ? 1.0 : exp(l - m)); }

// Selects in one row by the wave: lane r < k returns expert id and logit of
// rank r.  Lane l holds experts l + 64 i.  kd: LDS of E doubles, the wave's own.
template <int NPER>
__device__ __forceinline__ void select_row(const RouterP& R, const float (&val)[NPER], int E, int k, double m,
                                           double den, double* kd, int& id, float& logit) {
  const int lane = threadIdx.x & 63;
  uint64_t rk[NPER];
  const int gs = E / R.n_group;
#pragma unroll
  for (int i = 0; i < NPER; ++i) {
    const int e = lane + 64 * i;
    double key = 0.0;
    if (e < E) {
      const double l = (double)val[i];
      double s = 0.0;
      if (R.bias || R.top2) s = l != l ? l : (R.sigmoid ? sigmoid64(l) : unnorm64(l, m) / den);
      key = R.bias ? s + (double)R.bias[e] : l;
      if (R.n_group > 1) kd[e] = R.bias || !R.top2 ? key : s;
    }
    rk[i] = e < E ? rank64(key) : 0ull;
  }
  if (R.n_group > 1) {
    __builtin_amdgcn_wave_barrier();
    uint64_t gk = 0;
    if (lane < R.n_group) {
      double a = -INFINITY, b = -INFINITY;  // the two largest
      bool any = false;
      for (int j = 0; j < gs; ++j) {
        double v = kd[lane * gs + j];
        any = any || v == v;
        if (v != v) v = -INFINITY;
        if (v > a) {
          b = a;
          a = v;
        } else if (v > b) {
          b = v;
        }
      }
      gk = rank64(R.top2 && gs > 1 ? a + b : (any ? a : NAN));
    }
    uint64_t live = 0;
    for (int r = 0; r < R.topk_group; ++r) {
      const uint64_t mx = wave_max_u64(gk);
      const int g = __builtin_ctzll(__ballot(gk == mx));
      live |= 1ull << g;
      if (lane == g) gk = 0;
    }
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !((live >> (e / gs)) & 1)) rk[i] = 0;
    }
  }
  id = 0;
  logit = 0.f;
  for (int r = 0; r < k; ++r) {
    uint64_t lm = rk[0];
#pragma unroll
    for (int i = 1; i < NPER; ++i) lm = max(lm, rk[i]);
    const uint64_t mx = wave_max_u64(lm);
    int ws = 0;
    uint64_t bw = 0;
#pragma unroll
    for (int i = NPER - 1; i >= 0; --i) {
      const uint64_t b = __ballot(rk[i] == mx);
      ws = b ? i : ws;
      bw = b ? b : bw;
    }
    const int wl = __builtin_ctzll(bw);
    float v = val[0];
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
      v = i == ws ? val[i] : v;
      rk[i] = i == ws && lane == wl ? 0ull : rk[i];
    }
    v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), wl));
    if (lane == r) {
      id = wl + 64 * ws;
      logit = v;
    }
  }
}

template <int NPER>
__global__ __launch_bounds__(256) void k_route_scored(RouterP R, const float* __restrict__ logits, int T, int E, int k,
                                                      int32_t* __restrict__ ids, float* __restrict__ wts) {
  extern __shared__ double kd_all[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * 4 + wave;
  if (t >= T) return;
  float val[NPER];
  wave_topk_load<NPER>(logits + (size_t)t * E, E, val);
  double m = 0.0, den = 1.0;
  if (!R.sigmoid) {
    uint32_t mk = 0;
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      if (lane + 64 * i < E) mk = max(mk, rank_bits(val[i]));
    mk = wave_max_u32(mk);
    m = mk == 0 ? 0.0 : (double)__uint_as_float((mk & 0x80000000u) ? mk & 0x7FFFFFFFu : ~mk);
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < NPER; ++i)
      if (lane + 64 * i < E) part += unnorm64((double)val[i], m);
    den = wave_sum_f64(part);
  }
  int id;
  float l;
  select_row<NPER>(R, val, E, k, m, den, kd_all + (size_t)wave * E, id, l);
  double s = 0.0;
  if (lane < k) s = R.sigmoid ? sigmoid64((double)l) : unnorm64((double)l, m);
  double d = R.sigmoid ? 1.0 : den;
  if (R.renorm) d = wave_sum_f64(s);
  if (lane < k) {
    ids[(size_t)t * k + lane] = id;
    wts[(size_t)t * k + lane] = (float)((d > 0.0 ? s / d : 1.0 / k) * (double)R.scale);
  }
}

moe_status check_router(const char* who, const moe_router* r, int T, int E, int k) {
  MOE_CHECK_ARG(r, "%s: null router", who);
  MOE_CHECK_ARG(T >= 0 && E >= 1 && E <= 1024, "%s: bad sizes T=%d E=%d (E <= 1024)", who, T, E);
  MOE_CHECK_ARG(r->score == MOE_SCORE_SOFTMAX || r->score == MOE_SCORE_SIGMOID, "%s: bad score %d", who, r->score);
  MOE_CHECK_ARG(r->group_rank == MOE_GROUP_MAX || r->group_rank == MOE_GROUP_TOP2, "%s: bad group_rank %d", who,
                r->group_rank);
  MOE_CHECK_ARG(r->n_group >= 1 && r->n_group <= 64 && E % r->n_group == 0,
                "%s: n_group=%d must divide E=%d and be at most 64", who, r->n_group, E);
  MOE_CHECK_ARG(r->topk_group >= 1 && r->topk_group <= r->n_group, "%s: topk_group=%d must be in [1, n_group=%d]", who,
                r->topk_group, r->n_group);
  const int most = std::min(r->topk_group * (E / r->n_group), kRouteMaxK);
  MOE_CHECK_ARG(k >= 1 && k <= most, "%s: k=%d must be in [1, min(topk_group * E / n_group, 16)] = [1, %d]", who, k,
                most);
  return MOE_OK;
}

}  // namespace

extern "C" moe_status moe_route_scored(const moe_router* r, const float* logits, int T, int E, int k,
                                       int32_t* topk_ids, float* topk_w, moe_stream_t stream) {
  moe_status st = check_router("moe_route_scored", r, T, E, k);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  MOE_CHECK_ARG(logits && topk_ids && topk_w, "moe_route_scored: null pointer");
  const RouterP R{r->bias, r->scale, r->score == MOE_SCORE_SIGMOID, r->n_group, r->topk_group,
                  r->n_group > 1 && r->group_rank == MOE_GROUP_TOP2, r->renormalize};
  const dim3 g((unsigned)((T + 3) / 4));
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const size_t lds = r->n_group > 1 ? 4 * sizeof(double) * (size_t)E : 0;  // at most 32 KiB
  if (E <= 64) launch(k_route_scored<1>, g, dim3(256), lds, s, R, logits, T, E, k, topk_ids, topk_w);
  else if (E <= 128) launch(k_route_scored<2>, g, dim3(256), lds, s, R, logits, T, E, k, topk_ids, topk_w);
  else if (E <= 256) launch(k_route_scored<4>, g, dim3(256), lds, s, R, logits, T, E, k, topk_ids, topk_w);
  else launch(k_route_scored<16>, g, dim3(256), lds, s, R, logits, T, E, k, topk_ids, topk_w);
  MOE_LAUNCHED();
  return MOE_OK;
}

extern "C" moe_status moe_route_scored_permute(const moe_router* r, const float* logits, int T, int E, int k,
                                               int32_t* topk_ids, float* topk_w, int32_t* counts, int32_t* offsets,
                                               int32_t* perm, int32_t* inv, moe_stream_t stream) {
  moe_status st = check_router("moe_route_scored_permute", r, T, E, k);
  if (st != MOE_OK) return st;
  MOE_CHECK_ARG((long long)T * k <= (1 << 17), "moe_route_scored_permute: T*k = %lld exceeds 131072", (long long)T * k);
  MOE_CHECK_ARG(counts && offsets && (T == 0 || (logits && topk_ids && topk_w && perm && inv)),
                "moe_route_scored_permute: null pointer");
  st = moe_route_scored(r, logits, T, E, k, topk_ids, topk_w, stream);
  if (st != MOE_OK) return st;
  return moe_permute(topk_ids, T, k, E, counts, offsets, perm, inv, stream);
}
