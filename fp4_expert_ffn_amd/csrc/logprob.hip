// Log probabilities of given tokens, their ranks, the rows' entropies and the
// k most likely tokens, in one read of the logits (gfx950, wave64).
//
// With m the row's largest logit l, c = scale * log2(e) and d_i = c (l_i - m):
//
//   s0 = sum 2^d_i, s1 = sum d_i 2^d_i
//   log p_i = scale (l_i - m) - ln s0,  lse = scale m + ln s0,
//   entropy = ln s0 - ln 2 s1 / s0
//
// A thread takes its sums against b, the rounded c times its own maximum, so
// that an exponent is one FMA, and rescales them when the maximum grows.
// Threads, waves and the pieces of a row are joined the same way, in 64 bits,
// and b - c m is put back there: the largest logit counts as exactly 1.
//
// The k best are keys of 64 bits (the logit's order, then the lower id).  A
// wave gathers in LDS what passes the bar: at first the k-th best of its lanes'
// largest, later the best k-th best of the workgroup's waves.  When 3 k have
// gathered, the upper 16 bits of the k-th are found bit by bit with ballots,
// become the bar, and what lies below goes: whatever the order of the logits, a
// key is looked at a few times.  Only the row's last 64 are sorted.  The best
// alone (k = 1) needs none of it: a thread remembers where its maximum stood.
//
// Ranks are counted by ballots, on the scalar unit, and only where some lane's
// largest reaches the given logit.
//
// Bound: HBM on long batches, 4096 rows of 131072 bf16 logits (1.07 GB), k = 1,
// 205 us, 5.2 TB/s; else latency and the instructions of the lists: 333 rows of
// 50021 fp32 (67 MB), most masked, k = 5, 24 us and 7 for the join; one row of
// 131072, k = 20, 7.4 and 6.  The lists of few keys wait on LDS, ballots and
// cold instructions: sorting instead took 269 us where this took 212.
//
// Rows whose c m is beyond 1e8, infinite ones among them, or that hold a NaN,
// are summed once more, in 64 bits (finish_row).
#include <algorithm>

#include "common.h"
#include "wave.h"

namespace {

using namespace moe;

constexpr int kMaxTop = 64;
constexpr int kThreads = 256, kWaves = kThreads / 64;

struct LogprobParams {
  int T, V;
  const void* logits;
  int64_t ld;
  float scale, c;  // c = scale * log2(e)
  const int32_t* ids;
  float* logprob;
  int32_t* rank;
  float* entropy;
  float* lse;
  int k;
  int32_t* top_ids;
  float* top_logprob;
  int splits, piece;  // logits a piece
  uint8_t* ws;        // splits > 1: [T * splits] Piece, then keys: [T * splits][64], one each with k = 1
};

// What a piece of a row leaves: its maximum, the two sums against b, and the
// tokens in front of the given one.
struct Piece {
  double s0, s1;
  float m, b;
  int rank, held;  // held: keys it leaves, 64 at most
};

// The order of tokens as one number: the logit's order (equal values equal,
// -0 as +0, NaN lowest), then the lower id; 0: none.
__device__ __forceinline__ uint64_t key_of(float v, int i) {
  uint32_t u = __float_as_uint(v);
  u = (u & 0x7FFFFFFFu) == 0u ? 0u : u;
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  u = v != v ? 0u : u;
  return ((uint64_t)u << 32) | (uint32_t)~i;
}

// The logit of a key; its id.
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return u == 0u ? __builtin_nanf("") : __uint_as_float((u & 0x80000000u) ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ int key_id(uint64_t k) { return (int)~(uint32_t)k; }

// The value of lane l ^ D.
template <int D>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v) {
  if constexpr (D == 1) return dpp_u32<kDppQuadXor1>(v);
  if constexpr (D == 2) return dpp_u32<kDppQuadXor2>(v);
  if constexpr (D == 3) return dpp_u32<0x1B>(v);               // quad_perm [3,2,1,0]
  if constexpr (D == 4) return lane_xor<3>(lane_xor<7>(v));
  if constexpr (D == 7) return dpp_u32<kDppRowHalfMirror>(v);
  if constexpr (D == 8) return lane_xor<7>(lane_xor<15>(v));
  if constexpr (D == 15) return dpp_u32<kDppRowMirror>(v);
  if constexpr (D == 16) {
    auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (threadIdx.x & 16) ? r[0] : r[1];
  }
  if constexpr (D == 31) return lane_xor<15>(lane_xor<16>(v));
  if constexpr (D == 32) {
    auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (threadIdx.x & 32) ? r[0] : r[1];
  }
  if constexpr (D == 63) return lane_xor<31>(lane_xor<32>(v));
  return 0;
}
template <int D>
__device__ __forceinline__ uint64_t lane_xor64(uint64_t v) {
  return ((uint64_t)lane_xor<D>((uint32_t)(v >> 32)) << 32) | lane_xor<D>((uint32_t)v);
}

// Lane l and its partner l ^ D: the larger to the lower lane.
template <int D, int BIT>
__device__ __forceinline__ uint64_t exchange(uint64_t v) {
  const uint64_t o = lane_xor64<D>(v);
  const bool low = (threadIdx.x & BIT) == 0;
  return (v > o) == low ? v : o;
}

// A bitonic run of 2 * HALF lanes in descending order.
template <int HALF>
__device__ __forceinline__ uint64_t settle(uint64_t v) {
  v = exchange<HALF, HALF>(v);
  if constexpr (HALF > 1) v = settle<HALF / 2>(v);
  return v;
}

// Keys in descending order over the lanes, all but the first n (uniform) of
// them 0: runs of twice the length by a first step against the mirrored
// partner, as far as there are keys.
__device__ __forceinline__ uint64_t sort64(uint64_t v, int n) {
  v = exchange<1, 1>(v);
  v = settle<1>(exchange<3, 2>(v));
  if (n > 4) v = settle<2>(exchange<7, 4>(v));
  if (n > 8) v = settle<4>(exchange<15, 8>(v));
  if (n > 16) v = settle<8>(exchange<31, 16>(v));
  if (n > 32) v = settle<16>(exchange<63, 32>(v));
  return v;
}

// The k-th largest of the lanes' 32-bit keys, n registers of them, its lower
// half cut off (0: there are fewer; uniform).
template <int N>
__device__ __forceinline__ uint32_t kth_of_lanes(const uint32_t (&x)[N], int n, int k) {
  uint32_t t = 0;
#pragma unroll 1
  for (uint32_t bit = 1u << 31; bit >= 1u << 16; bit >>= 1) {
    const uint32_t c = t | bit;
    int have = __popcll(__ballot(x[0] >= c));
#pragma unroll
    for (int i = 1; i < N; ++i)
      if (i < n) have += __popcll(__ballot(x[i] >= c));
    t = have >= k ? c : t;
  }
  return t;
}

// The workgroup's bar, in LDS: the largest of its waves'.
__device__ __forceinline__ uint64_t shared_bar(uint64_t* s_bar) {
  const uint64_t o = __hip_atomic_load(s_bar, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  return ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(o >> 32)) << 32) |
         (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)o);
}
__device__ __forceinline__ void raise_shared(uint64_t* s_bar, uint64_t to) {
  if ((threadIdx.x & 63) == 0) __hip_atomic_fetch_max(s_bar, to, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}

// A wave's keys, unordered, in LDS.
constexpr int kKeys = 256;
struct Keys {
  uint64_t* at;  // [kKeys]
  int k, held;   // how many are wanted; uniform
  int limit;     // held beyond it: time to cut
  uint64_t bar;  // what a key has to pass (uniform); 0: all do
  float bar_v;   // its logit; -inf where it is no number's

  // Until it is cut the bar stands, and the share of logits that pass it, and
  // go the long way, is k to what had been seen when it was set; a cut costs as
  // much as some ten additions.
  __device__ __forceinline__ Keys(uint64_t* lds, int wanted, int least)
      : at(lds), k(wanted), held(0), limit(min(kKeys - 64, max(least, 3 * k))), bar(0), bar_v(-__builtin_inff()) {}
  __device__ __forceinline__ void raise(uint64_t to) {
    if (to > bar) {
      bar = to;
      bar_v = (uint32_t)(bar >> 32) < 0x007FFFFFu ? -__builtin_inff() : key_value(bar);  // below the key of -inf
    }
  }
  // Takes the lanes' keys that pass; 64 places at least are free.
  __device__ __forceinline__ void add(uint64_t key) {
    const bool pass = key > bar;
    const uint64_t mask = __ballot(pass);
    if (pass) at[held + __popcll(mask & ((1ull << (threadIdx.x & 63)) - 1))] = key;
    held += __popcll(mask);
    __builtin_amdgcn_wave_barrier();  // a wave's LDS accesses keep their order
  }
  // Keeps the k best and those that share the upper 16 bits with the k-th, 64 at
  // most in all; raises the bar to those bits.
  __device__ __forceinline__ void cut() {
    const int lane = threadIdx.x & 63;
    constexpr int N = kKeys / 64;
    const int n = (held + 63) / 64;
    uint64_t r[N];
    uint32_t x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      r[i] = i * 64 + lane < held ? at[i * 64 + lane] : 0u;
      x[i] = (uint32_t)(r[i] >> 32);
    }
    uint64_t t = (uint64_t)kth_of_lanes(x, n, k) << 32;
    int have = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) have += __popcll(__ballot(r[i] != 0u && r[i] >= t));
    if (have > 64) {  // many equal logits: the k-th key itself
      for (uint64_t bit = 1ull << 47; bit; bit >>= 1) {
        const uint64_t c = t | bit;
        have = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) have += __popcll(__ballot(r[i] >= c));
        if (have >= k) t = c;
        if (have == k) break;
      }
    }
    const uint64_t low = t ? t - 1 : 0u;  // keys are whole numbers: what reaches t passes
    held = 0;
    bar = low;
#pragma unroll
    for (int i = 0; i < N; ++i) add(r[i]);
    bar = 0;
    raise(low);
    limit = min(kKeys - 64, max(limit, 2 * held));
  }
  // Cuts where the limit is passed; the workgroup's bar follows.
  __device__ __forceinline__ void room(uint64_t* s_bar) {
    if (held > limit) {
      const uint64_t had = bar;
      cut();
      raise_shared(s_bar, bar);
      raise(had);
    }
  }
  // A wave's keys, 64 at most, and its bar for wave 0 ..
  __device__ __forceinline__ void publish(int* s_held, uint64_t* s_bar, int wave) {
    if (held > 64) cut();
    if ((threadIdx.x & 63) == 0) s_held[wave] = held;
    raise_shared(s_bar, bar);
  }
  // .. which adds the others' to its own, behind a barrier: one a lane, unordered.
  // The waves' keys lie kKeys apart.
  __device__ __forceinline__ uint64_t gather(const int* s_held, uint64_t* s_bar) {
    const int lane = threadIdx.x & 63;
    raise(shared_bar(s_bar));
#pragma unroll
    for (int w = 1; w < kWaves; ++w) add(lane < s_held[w] ? at[w * kKeys + lane] : 0u);
    if (held > 64) cut();
    return lane < held ? at[lane] : 0u;
  }
};

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp_f32<kDppQuadXor1>(v));
  v = fmaxf(v, dpp_f32<kDppQuadXor2>(v));
  v = fmaxf(v, dpp_f32<kDppRowHalfMirror>(v));
  v = fmaxf(v, dpp_f32<kDppRowMirror>(v));
  return max_rows4(v);
}

// Sums taken against b as sums against `to`.  The factor in fp32: a part of
// the sum is off by 2^-23 of itself.
__device__ __forceinline__ void rebase(double& s0, double& s1, float b, float to) {
  const float d = fmaxf(b - to, -1000.f);
  const double f = (double)__builtin_amdgcn_exp2f(d);
  s1 = f * (s1 + (double)d * s0);
  s0 = f * s0;
}

template <bool F32>
__device__ __forceinline__ float logit(const void* row, int i) {
  return F32 ? static_cast<const float*>(row)[i] : bf16_to_f32(static_cast<const uint16_t*>(row)[i]);
}

// A row's given token; its logit, NaN where there is none.
struct Given {
  int id;
  float v;
};
template <bool F32>
__device__ __forceinline__ Given given_of(const LogprobParams& P, int t, const void* row) {
  const int id = P.ids ? P.ids[t] : -1;
  return Given{id, id >= 0 && id < P.V ? logit<F32>(row, id) : __builtin_nanf("")};
}

// b, rounded, is off by up to 2^-24 |c m|: 2^(c m - b), which the joins put
// back, stays small below 1e8.  kLeast: b of what has seen no c l above it.
constexpr float kHuge = 1e8f, kLeast = -1e8f;

// The outputs of a row from its joined sums against b, by the whole workgroup
// of NT threads: lane l of wave 0 holds the l-th best key.
// ONE: the best alone is wanted; 0 where no logit is above -inf.
template <bool F32, bool ONE, int NT>
__device__ __forceinline__ void finish_row(const LogprobParams& P, int t, const void* row, Given gt, float m, float b,
                                           double s0, double s1, int rank, uint64_t best) {
  __shared__ double s_sum[NT / 64][2];
  __shared__ int s_nan, s_low;
  const int tid = threadIdx.x;
  const bool endless = !(fabsf(m) < __builtin_inff());
  const double mc = (double)m * (double)P.c;
  const bool odd = !(fabs(mc) < (double)kHuge) || s0 != s0;
  bool nan = false;
  if (!odd) {
    const double d = (double)b - mc, f = exp2(d);
    s1 = f * (s1 + d * s0);
    s0 = f * s0;
  } else {  // uniform: the sums once more.  An endless m: tokens equal to it share the row
    if (tid == 0) {
      s_nan = 0;
      s_low = P.V;
    }
    __syncthreads();
    double a0 = 0, a1 = 0;
    bool bad = false;
    int low = P.V;  // the first logit equal to m
    for (int i = tid; i < P.V; i += NT) {
      const float v = logit<F32>(row, i);
      bad = bad || v != v;
      if (ONE && v == m) low = min(low, i);
      const double d = v == m ? 0.0 : (endless ? -2000.0 : fmax((double)P.c * (double)v - mc, -2000.0));
      const double e = d <= -2000.0 ? 0.0 : exp2(d);
      a0 += e;
      a1 += d * e;
    }
    if (bad) atomicOr(&s_nan, 1);
    if (ONE) atomicMin(&s_low, low);
    a0 = wave_sum64(a0);
    a1 = wave_sum64(a1);
    if ((tid & 63) == 0) {
      s_sum[tid >> 6][0] = a0;
      s_sum[tid >> 6][1] = a1;
    }
    __syncthreads();
    nan = s_nan != 0;
    if (ONE && best == 0u) best = s_low < P.V ? key_of(m, s_low) : key_of(__builtin_nanf(""), 0);
    s0 = s1 = 0;
    for (int w = 0; w < NT / 64; ++w) {
      s0 += s_sum[w][0];
      s1 += s_sum[w][1];
    }
  }
  if (tid >= 64) return;
  const double log_s = nan ? (double)__builtin_nanf("") : log(s0);
  auto prob = [&](float v) {
    if (v == m) return -log_s;
    if (endless) return nan ? log_s : -(double)__builtin_inff();
    return (double)P.scale * ((double)v - (double)m) - log_s;
  };
  if (tid == 0) {
    if (P.lse) P.lse[t] = (float)((double)P.scale * (double)m + log_s);
    if (P.entropy) P.entropy[t] = (float)(log_s - s1 * 0.69314718055994530942 / s0);
    if (P.logprob) P.logprob[t] = gt.id < 0 ? 0.f : (gt.v != gt.v ? __builtin_nanf("") : (float)prob(gt.v));
    if (P.rank) P.rank[t] = gt.v != gt.v ? -1 : rank;
  }
  if (tid < P.k) {
    const float v = key_value(best);
    if (P.top_ids) P.top_ids[(int64_t)t * P.k + tid] = key_id(best);
    if (P.top_logprob) P.top_logprob[(int64_t)t * P.k + tid] = v != v ? v : (float)prob(v);
  }
}

// A wave's joined maximum, sums and rank, in every lane.
__device__ __forceinline__ void join_wave(float& m, float& b, double& s0, double& s1) {
  m = wave_max(m);
  const float to = wave_max(b);
  rebase(s0, s1, b, to);
  b = to;
  s0 = wave_sum64(s0);
  s1 = wave_sum64(s1);
}

// The wave's largest key, in every lane.
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
  auto larger = [](uint64_t a, uint64_t b) { return a > b ? a : b; };
  v = larger(v, lane_xor64<1>(v));
  v = larger(v, lane_xor64<2>(v));
  v = larger(v, lane_xor64<7>(v));
  v = larger(v, lane_xor64<15>(v));
  v = larger(v, lane_xor64<16>(v));
  return larger(v, lane_xor64<32>(v));
}

// What of the k best a call wants.
enum { kNoTop, kBest, kList };

// A workgroup: one piece of one row.  A thread takes 8 logits at a time.
template <bool F32, int WANT>
__global__ __launch_bounds__(kThreads) void k_logprob(LogprobParams P) {
  constexpr int E = 8, ES = F32 ? 4 : 2, NL = F32 ? 2 : 1;
  constexpr bool TOP = WANT == kList;
  __shared__ uint64_t s_best[kWaves];
  __shared__ uint64_t s_keys[TOP ? kWaves : 1][kKeys], s_bar;
  __shared__ int s_held[kWaves];
  __shared__ double s_sum[kWaves][2];
  __shared__ float s_m[kWaves][2];
  __shared__ int s_rank[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t = (int)(blockIdx.x / P.splits), sp = (int)(blockIdx.x % P.splits);
  const uint8_t* row = static_cast<const uint8_t*>(P.logits) + (int64_t)t * P.ld * ES;
  const int lo = sp * P.piece, hi = min(lo + P.piece, P.V);
  const Given gt = given_of<F32>(P, t, row);
  const int id = gt.id;
  const bool given = P.rank && id >= 0 && id < P.V;
  const float gv = given ? gt.v : __builtin_inff();  // nothing lies in front of +inf
  // the largest number below gv (for +-0: the least negative one): v > under says v >= gv (-inf has none: see below)
  const uint32_t gu = __float_as_uint(gv);
  const float under = (gu & 0x7FFFFFFFu) == 0u ? __uint_as_float(0x80000001u)
                      : (gv == -__builtin_inff() ? gv : __uint_as_float((gu & 0x80000000u) ? gu + 1u : gu - 1u));
  if constexpr (TOP) {
    if (tid == 0) s_bar = 0;
    __syncthreads();
  }
  // pieces of 8 logits of the row's memory, on 16-byte boundaries: piece q holds logits 8 q - shift ..
  const int shift = (int)(((uintptr_t)row & 15) / ES);
  const int q0 = (lo + shift) / E, q1 = (hi + shift + E - 1) / E;
  float m = -__builtin_inff(), b = kLeast, s0 = 0.f, s1 = 0.f;
  int rank = 0;  // uniform
  int mq = 0;    // kBest: the piece of 8 that m is from
  Keys keys(s_keys[TOP ? wave : 0], P.k, P.piece <= 16 * E * kThreads ? 64 : 8);
  auto whole = [&](int q) { return q < q1 && q * E - shift >= lo && q * E - shift + E <= hi; };
  auto load = [&](int q, uint4 (&u)[NL]) __attribute__((always_inline)) {
    if (whole(q)) {
      const uint4* p = reinterpret_cast<const uint4*>(row + (int64_t)(q * E - shift) * ES);
#pragma unroll
      for (int j = 0; j < NL; ++j) u[j] = p[j];
    }
  };
  auto unpack = [&](int q, const uint4 (&u)[NL], float (&v)[E]) __attribute__((always_inline)) {
    if (whole(q)) {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const uint32_t d[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          if constexpr (F32) {
            v[4 * j + w] = __uint_as_float(d[w]);
          } else {
            v[2 * w] = __uint_as_float(d[w] << 16);
            v[2 * w + 1] = __uint_as_float(d[w] & 0xFFFF0000u);
          }
        }
      }
    } else {  // the ends of the piece: what is not its own counts as -inf
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int i = q * E - shift + j;
        v[j] = q < q1 && i >= lo && i < hi ? logit<F32>(row, i) : -__builtin_inff();
      }
    }
  };
  auto take = [&](int q, const float (&v)[E], bool first) __attribute__((always_inline)) {
    const int i0 = q * E - shift;
    float top = v[0];
#pragma unroll
    for (int j = 1; j < E; ++j) top = fmaxf(top, v[j]);
    if (top > m) {
      m = top;
      if (WANT == kBest) mq = q;
      const float to = fmaxf(m * P.c, kLeast), d = fmaxf(b - to, -200.f), f = __builtin_amdgcn_exp2f(d);
      s1 = f * fmaf(d, s0, s1);
      s0 = f * s0;
      b = to;
    }
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float d = fmaf(v[j], P.c, -b);
      const float e = __builtin_amdgcn_exp2f(d);  // 0 at -inf; NaN stays
      s0 += e;
      s1 = fmaf(fmaxf(d, -200.f), e, s1);
    }
    if (given) {
      // equal logits count where their ids are lower; those of the given one's own 8 are looked at below
      const float g = i0 + E <= id ? under : gv;
      if (__any(top > g)) {
#pragma unroll
        for (int j = 0; j < E; ++j) rank += __popcll(__ballot(v[j] > g));
      }
    }
    if constexpr (TOP) {
      if (first) {  // a bar from the lanes' largest: the k-th of them
        const uint32_t x[1] = {whole(q) ? (uint32_t)(key_of(top, 0) >> 32) : 0u};
        keys.raise((uint64_t)kth_of_lanes(x, 1, P.k) << 32);
      }
      // a bar below all numbers lets NaN pass too
      if ((uint32_t)(keys.bar >> 32) == 0u || __any(top >= keys.bar_v)) {
        keys.raise(shared_bar(&s_bar));  // what the other waves hold counts too
        // the lane's logits that reach it, each of its own lane's in turn: mostly one turn
        const bool all = (uint32_t)(keys.bar >> 32) == 0u;  // NaN passes too
        uint32_t left = 0;
#pragma unroll
        for (int j = 0; j < E; ++j)
          left |= (all || v[j] >= keys.bar_v) && q < q1 && i0 + j >= lo && i0 + j < hi ? 1u << j : 0u;
#pragma unroll 1
        while (__any(left != 0u)) {
          const int j = left ? __builtin_ctz(left) : 0;
          float x = v[0];
#pragma unroll
          for (int o = 1; o < E; ++o) x = j == o ? v[o] : x;
          keys.add(left ? key_of(x, i0 + j) : 0u);
          left &= left - 1u;  // 0 stays 0
          keys.room(&s_bar);
        }
      }
    }
  };
  // a load ahead: with eight waves a SIMD it has their whole turn to land
  uint4 u[NL];
  int q = q0 + wave * 64;  // uniform
  load(q + lane, u);
#pragma unroll 1
  for (bool first = true; q < q1; q += kThreads, first = false) {
    float v[E];
    unpack(q + lane, u, v);
    load(q + kThreads + lane, u);
    take(q + lane, v, first);
  }
  if constexpr (TOP) keys.publish(s_held, &s_bar, wave);
  if (given) {
    // equal logits of the 8 that hold the given one, which may lie in two pieces: in each those that are its own; of -inf all
    const bool least = gv == -__builtin_inff();
    const int to = min(id, hi), from = least ? lo : max((id + shift) / E * E - shift, lo);
    for (int i = from + wave * 64; i < to; i += kThreads)  // uniform
      rank += __popcll(__ballot(i + lane < to && logit<F32>(row, min(i + lane, to - 1)) == gv));
  }
  if constexpr (WANT == kBest) {  // the first of the 8 that equals m
    int at = hi;
    if (m > -__builtin_inff()) {
#pragma unroll
      for (int j = E - 1; j >= 0; --j) {
        const int i = min(max(mq * E - shift + j, lo), hi - 1);
        at = logit<F32>(row, i) == m ? i : at;
      }
    }
    const uint64_t key = wave_max64(at < hi ? key_of(m, at) : 0u);
    if (lane == 0) s_best[wave] = key;
  }
  // the waves' sums
  double d0 = s0, d1 = s1;
  join_wave(m, b, d0, d1);
  if (lane == 0) {
    s_m[wave][0] = m;
    s_m[wave][1] = b;
    s_sum[wave][0] = d0;
    s_sum[wave][1] = d1;
    s_rank[wave] = rank;
  }
  __syncthreads();
  float gm = s_m[0][0], gb = s_m[0][1];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) {
    gm = fmaxf(gm, s_m[w][0]);
    gb = fmaxf(gb, s_m[w][1]);
  }
  double g0 = 0, g1 = 0;
  int gr = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    double a0 = s_sum[w][0], a1 = s_sum[w][1];
    rebase(a0, a1, s_m[w][1], gb);
    g0 += a0;
    g1 += a1;
    gr += s_rank[w];
  }
  uint64_t best = 0;  // wave 0: the piece's best, 64 at most, one a lane, unordered
  if constexpr (TOP) {
    if (wave == 0) best = keys.gather(s_held, &s_bar);
  }
  if constexpr (WANT == kBest) {  // in every lane
#pragma unroll
    for (int w = 0; w < kWaves; ++w) best = s_best[w] > best ? s_best[w] : best;
  }
  if (P.splits == 1) {
    if (TOP && wave == 0) best = sort64(best, keys.held);
    finish_row<F32, WANT == kBest, kThreads>(P, t, row, gt, gm, gb, g0, g1, gr, best);
    return;
  }
  if (tid == 0) reinterpret_cast<Piece*>(P.ws)[blockIdx.x] = Piece{g0, g1, gm, gb, gr, keys.held};
  uint64_t* left = reinterpret_cast<uint64_t*>(P.ws + (int64_t)P.T * P.splits * sizeof(Piece));
  if (TOP && tid < keys.held) left[(int64_t)blockIdx.x * 64 + tid] = best;  // wave 0's
  if (WANT == kBest && tid == 0) left[blockIdx.x] = best;
}

// A workgroup: one row from its pieces, at most kMaxSplits.  Every wave joins
// the sums (lane l: piece l) and takes every fourth piece's best.
constexpr int kMaxSplits = 64;
template <bool F32, int WANT>
__global__ __launch_bounds__(kThreads) void k_logprob_join(LogprobParams P) {
  constexpr bool TOP = WANT == kList;
  __shared__ uint64_t s_keys[TOP ? kWaves : 1][kKeys], s_bar;
  __shared__ int s_held[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), t = blockIdx.x;
  const uint8_t* row = static_cast<const uint8_t*>(P.logits) + (int64_t)t * P.ld * (F32 ? 4 : 2);
  const Piece* pc = reinterpret_cast<const Piece*>(P.ws) + (int64_t)t * P.splits;
  const Given gt = given_of<F32>(P, t, row);
  Piece p{0, 0, -__builtin_inff(), kLeast, 0, 0};
  if (lane < P.splits) p = pc[lane];
  uint64_t best = 0;
  const uint64_t* left = reinterpret_cast<const uint64_t*>(P.ws + (int64_t)P.T * P.splits * sizeof(Piece));
  if constexpr (WANT == kBest) best = wave_max64(lane < P.splits ? left[(int64_t)t * P.splits + lane] : 0u);
  if constexpr (TOP) {
    const uint64_t* src = left + (int64_t)t * P.splits * 64 + lane;
    if (tid == 0) s_bar = 0;
    __syncthreads();
    Keys keys(s_keys[wave], P.k, 64);
    // the k-th best of the pieces' largest is a bar (-inf may stand for a piece of nothing but NaN)
    const uint32_t x[1] = {p.m > -__builtin_inff() ? (uint32_t)(key_of(p.m, 0) >> 32) : 0u};
    const uint32_t least = kth_of_lanes(x, 1, P.k);
    keys.raise((uint64_t)least << 32);
    uint64_t todo = __ballot(p.held > 0 && x[0] >= least) & (0x1111111111111111ull << wave);  // pieces that can pass it
    constexpr int U = 8;                                                                      // loaded at once
    while (todo) {
      const int n = min(__popcll(todo), U);
      uint64_t v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int s = todo ? __builtin_ctzll(todo) : 0;
        v[u] = todo && lane < __builtin_amdgcn_readlane(p.held, s) ? src[s * 64] : 0u;
        todo &= todo - 1;  // 0 stays 0
      }
#pragma unroll 1
      for (int u = 0; u < n; ++u) {
        uint64_t y = v[0];
#pragma unroll
        for (int o = 1; o < U; ++o) y = u == o ? v[o] : y;
        keys.add(y);
        if (keys.held > kKeys - 64) keys.cut();
      }
    }
    keys.publish(s_held, &s_bar, wave);
    __syncthreads();
    if (wave == 0) {
      best = keys.gather(s_held, &s_bar);
      best = sort64(best, keys.held);
    }
  }
  float m = p.m, b = p.b;
  double s0 = p.s0, s1 = p.s1;
  join_wave(m, b, s0, s1);
  int rank = p.rank;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) rank += __shfl_xor(rank, d);
  finish_row<F32, WANT == kBest, kThreads>(P, t, row, gt, m, b, s0, s1, rank, best);
}

template <bool F32, int WANT>
void launch_want(const LogprobParams& P, hipStream_t s) {
  launch(k_logprob<F32, WANT>, dim3((unsigned)((int64_t)P.T * P.splits)), dim3(kThreads), 0, s, P);
  if (P.splits > 1) launch(k_logprob_join<F32, WANT>, dim3((unsigned)P.T), dim3(kThreads), 0, s, P);
}

template <bool F32>
void launch_logprob(const LogprobParams& P, hipStream_t s) {
  if (P.k > 1) launch_want<F32, kList>(P, s);
  else if (P.k == 1) launch_want<F32, kBest>(P, s);
  else launch_want<F32, kNoTop>(P, s);
}

// Pieces of a row: about four workgroups a CU, none with less than 8 logits a
// thread.  us with 512, 1024 and 2048 workgroups: 333 rows of 50021 fp32 logits,
// k = 5, 36, 33 and 36; 64 rows of 131072, k = 20, 28, 26 and 28.  Up to 32
// logits a thread the join's launch costs more than pieces save, us cut and
// whole: 1 row of 4000, k = 1, 9.7 and 6.2; 128 rows of 8000, k = 20, 14.4 and
// 13.4; 1 row of 16000, k = 1, 10.1 and 11.4.
int row_splits(int T, int V) {
  if (V <= 32 * kThreads) return 1;
  const int most = (V + 8 * kThreads - 1) / (8 * kThreads);
  return std::max(1, std::min({most, 1024 / T, kMaxSplits}));
}

bool bad_sizes(const moe_logprob_args* a) {
  return a->T < 0 || a->T >= (1 << 22) || a->V < 1 || a->V >= (1 << 30) || a->k < 0 || a->k > kMaxTop || a->k > a->V;
}

}  // namespace

extern "C" size_t moe_logprobs_workspace_size(const moe_logprob_args* a) {
  if (!a || a->T < 1 || bad_sizes(a)) return 0;
  const size_t n = row_splits(a->T, a->V);
  return n == 1 ? 0 : (size_t)a->T * n * (sizeof(Piece) + (a->k > 1 ? 64 * 8 : 8 * a->k));
}

extern "C" moe_status moe_logprobs(const moe_logprob_args* a, moe_stream_t stream) {
  MOE_CHECK_ARG(a, "moe_logprobs: null pointer");
  MOE_CHECK_ARG(!bad_sizes(a), "moe_logprobs: bad sizes T=%d V=%d k=%d (T below 2^22, V below 2^30, k at most 64 and V)",
                a->T, a->V, a->k);
  MOE_CHECK_ARG(a->scale > 0.f && a->scale < __builtin_inff(), "moe_logprobs: scale must be positive and finite");
  const int64_t ld = a->ld ? a->ld : a->V;
  MOE_CHECK_ARG(ld >= a->V, "moe_logprobs: row stride %lld must be at least V=%d", (long long)ld, a->V);
  const bool top = a->top_ids || a->top_logprob;
  MOE_CHECK_ARG(a->logprob || a->rank || a->entropy || a->lse || top, "moe_logprobs: no output");
  MOE_CHECK_ARG(top == (a->k > 0), "moe_logprobs: k=%d %s top_ids or top_logprob", a->k, top ? "with" : "without");
  MOE_CHECK_ARG(a->ids || !(a->logprob || a->rank), "moe_logprobs: logprob and rank need ids");
  if (a->T == 0) return MOE_OK;
  MOE_CHECK_ARG(a->logits, "moe_logprobs: null pointer");
  MOE_CHECK_ARG(((uintptr_t)a->logits & (a->logits_f32 ? 3 : 1)) == 0 &&
                    (((uintptr_t)a->ids | (uintptr_t)a->logprob | (uintptr_t)a->rank | (uintptr_t)a->entropy |
                      (uintptr_t)a->lse | (uintptr_t)a->top_ids | (uintptr_t)a->top_logprob) & 3) == 0,
                "moe_logprobs: misaligned pointer");
  const size_t need = moe_logprobs_workspace_size(a);
  if (need > 0) {
    if (!a->workspace || a->workspace_bytes < need)
      return set_error(MOE_ENOMEM, "moe_logprobs: workspace %zu bytes, needs %zu", a->workspace ? a->workspace_bytes : 0,
                       need);
    MOE_CHECK_ARG(((uintptr_t)a->workspace & 15) == 0, "moe_logprobs: workspace must lie on a 16-byte boundary");
  }
  const int splits = row_splits(a->T, a->V);
  // whole 16-byte loads a piece, as far as the row's start allows
  const int piece = ((a->V + splits - 1) / splits + 7) / 8 * 8;
  const LogprobParams P{a->T, a->V, a->logits, ld, a->scale, (float)((double)a->scale * 1.44269504088896340736), a->ids,
                        a->logprob, a->rank, a->entropy, a->lse, a->k, a->top_ids, a->top_logprob, splits, piece,
                        static_cast<uint8_t*>(a->workspace)};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  a->logits_f32 ? launch_logprob<true>(P, s) : launch_logprob<false>(P, s);
  MOE_LAUNCHED();
  return MOE_OK;
}
