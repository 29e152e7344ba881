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
// The k best are keys of 64 bits (the logit's order, then the lower id), which
// a wave holds sorted over its lanes.  What passes the bar (the best k-th best
// of the workgroup's waves; at first the k-th best of the lanes' largest) is
// gathered in LDS, and every 64 of them are sorted and merged into the list:
// no order of the logits costs more than one sort per 64.
//
// Ranks are counted by ballots, on the scalar unit, and only where some lane's
// largest reaches the given logit.
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
  uint8_t* ws;        // splits > 1: [T * splits] Piece, then [T * splits][k] keys
};

// What a piece of a row leaves: its maximum, the two sums against b, and the
// tokens in front of the given one.
struct Piece {
  double s0, s1;
  float m, b;
  int rank, pad;
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

// 64 keys in descending order over the lanes: runs of twice the length by a
// first step against the mirrored partner.
__device__ __forceinline__ uint64_t sort64(uint64_t v) {
  v = exchange<1, 1>(v);
  v = settle<1>(exchange<3, 2>(v));
  v = settle<2>(exchange<7, 4>(v));
  v = settle<4>(exchange<15, 8>(v));
  v = settle<8>(exchange<31, 16>(v));
  return settle<16>(exchange<63, 32>(v));
}

// The 64 best of two descending lists, descending.
__device__ __forceinline__ uint64_t merge64(uint64_t a, uint64_t b) {
  const uint64_t r = lane_xor64<63>(b);
  return settle<32>(a > r ? a : r);
}

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

// Sums taken against b as sums against `to`.
__device__ __forceinline__ void rebase(double& s0, double& s1, double b, double to) {
  const double d = fmax(b - to, -1000.0), f = exp2(d);
  s1 = f * (s1 + d * s0);
  s0 = f * s0;
}

template <bool F32>
__device__ __forceinline__ float logit(const void* row, int i) {
  return F32 ? static_cast<const float*>(row)[i] : bf16_to_f32(static_cast<const uint16_t*>(row)[i]);
}

// b, rounded, is off by up to 2^-24 |c m|: 2^(c m - b), which the joins put
// back, stays small below 1e8.  kLeast: b of what has seen no c l above it.
constexpr float kHuge = 1e8f, kLeast = -1e8f;

// The outputs of a row from its joined sums against b, by the whole workgroup
// of NT threads: lane l of wave 0 holds the l-th best key.
template <bool F32, int NT>
__device__ __forceinline__ void finish_row(const LogprobParams& P, int t, const void* row, float m, float b, double s0,
                                           double s1, int rank, uint64_t best) {
  __shared__ double s_sum[NT / 64][2];
  __shared__ int s_nan;
  const int tid = threadIdx.x;
  const bool endless = !(fabsf(m) < __builtin_inff());
  const double mc = (double)m * (double)P.c;
  const bool odd = !(fabs(mc) < (double)kHuge) || s0 != s0;
  bool nan = false;
  if (!odd) {
    rebase(s0, s1, b, mc);
  } else {  // uniform: the sums once more.  An endless m: tokens equal to it share the row
    if (tid == 0) s_nan = 0;
    __syncthreads();
    double a0 = 0, a1 = 0;
    bool bad = false;
    for (int i = tid; i < P.V; i += NT) {
      const float v = logit<F32>(row, i);
      bad = bad || v != v;
      const double d = v == m ? 0.0 : (endless ? -2000.0 : fmax((double)P.c * (double)v - mc, -2000.0));
      const double e = d <= -2000.0 ? 0.0 : exp2(d);
      a0 += e;
      a1 += d * e;
    }
    if (bad) atomicOr(&s_nan, 1);
    a0 = wave_sum64(a0);
    a1 = wave_sum64(a1);
    if ((tid & 63) == 0) {
      s_sum[tid >> 6][0] = a0;
      s_sum[tid >> 6][1] = a1;
    }
    __syncthreads();
    nan = s_nan != 0;
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
    if (P.ids) {
      const int id = P.ids[t];
      const bool in = id >= 0 && id < P.V;
      const float v = in ? logit<F32>(row, id) : __builtin_nanf("");
      if (P.logprob) P.logprob[t] = id < 0 ? 0.f : (v != v ? __builtin_nanf("") : (float)prob(v));
      if (P.rank) P.rank[t] = v != v ? -1 : rank;
    }
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

// A workgroup: one piece of one row.  A thread takes 8 logits at a time.
template <bool F32, bool TOP>
__global__ __launch_bounds__(kThreads) void k_logprob(LogprobParams P) {
  constexpr int E = 8, ES = F32 ? 4 : 2, NL = F32 ? 2 : 1;
  __shared__ uint64_t s_buf[TOP ? kWaves : 1][128], s_list[TOP ? kWaves : 1][64], s_bar[kWaves];
  __shared__ double s_sum[kWaves][2];
  __shared__ float s_m[kWaves][2];
  __shared__ int s_rank[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t = (int)(blockIdx.x / P.splits), sp = (int)(blockIdx.x % P.splits);
  const uint8_t* row = static_cast<const uint8_t*>(P.logits) + (int64_t)t * P.ld * ES;
  const int lo = sp * P.piece, hi = min(lo + P.piece, P.V);
  const int id = P.rank ? P.ids[t] : -1;
  const bool given = id >= 0 && id < P.V;
  const float gv = given ? logit<F32>(row, id) : __builtin_inff();  // nothing lies in front of +inf
  // the largest number below gv (for +-0: the least negative one): v > under says v >= gv (-inf has none: see below)
  const uint32_t gu = __float_as_uint(gv);
  const float under = (gu & 0x7FFFFFFFu) == 0u ? __uint_as_float(0x80000001u)
                      : (gv == -__builtin_inff() ? gv : __uint_as_float((gu & 0x80000000u) ? gu + 1u : gu - 1u));
  if constexpr (TOP) {
    if (tid < kWaves) s_bar[tid] = 0;
    __syncthreads();
  }
  // pieces of 8 logits of the row's memory, on 16-byte boundaries: piece q holds logits 8 q - shift ..
  const int shift = (int)(((uintptr_t)row & 15) / ES);
  const int q0 = (lo + shift) / E, q1 = (hi + shift + E - 1) / E;
  float m = -__builtin_inff(), b = kLeast, s0 = 0.f, s1 = 0.f;
  int rank = 0;                 // uniform
  uint64_t list = 0, bar = 0;   // the wave's k best; what a key has to pass (uniform)
  float bar_v = -__builtin_inff();
  int held = 0;                 // keys in the buffer (uniform)
  auto raise = [&](uint64_t to) __attribute__((always_inline)) {
    if (to > bar) {
      bar = to;
      bar_v = (uint32_t)(bar >> 32) == 0u ? -__builtin_inff() : key_value(bar);
    }
  };
  auto flush = [&](int n) {  // the buffer's first n <= 64 keys into the list
    const uint64_t key = lane < n ? s_buf[wave][lane] : 0u;
    list = merge64(list, sort64(key));
    const int l = P.k - 1;
    const uint64_t kth = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(list >> 32), l) << 32) |
                         (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)list, l);
    if (lane == 0) s_bar[wave] = kth;
    raise(kth);
  };
  auto whole = [&](int q) { return q < q1 && q * E - shift >= lo && q * E - shift + E <= hi; };
  auto load = [&](int q, uint4 (&u)[NL]) __attribute__((always_inline)) {
    if (whole(q)) {
      const uint4* p = reinterpret_cast<const uint4*>(row + (int64_t)(q * E - shift) * ES);
#pragma unroll
      for (int j = 0; j < NL; ++j) u[j] = p[j];
    }
  };
  auto take = [&](int q, const uint4 (&u)[NL], bool first) __attribute__((always_inline)) {
    const int i0 = q * E - shift;
    float v[E];
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
        const int i = i0 + j;
        v[j] = q < q1 && i >= lo && i < hi ? logit<F32>(row, i) : -__builtin_inff();
      }
    }
    float top = v[0];
#pragma unroll
    for (int j = 1; j < E; ++j) top = fmaxf(top, v[j]);
    if (top > m) {
      m = top;
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
        uint32_t x = whole(q) ? (uint32_t)(key_of(top, 0) >> 32) : 0u;
        x = (uint32_t)(sort64((uint64_t)x << 32) >> 32);
        raise((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)x, P.k - 1) << 32);
      }
      if ((uint32_t)(bar >> 32) == 0u || __any(top >= bar_v)) {
        // what the other waves hold counts too
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const uint64_t o = *(volatile uint64_t*)&s_bar[w];
          raise(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(o >> 32)) << 32) |
                (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)o));
        }
#pragma unroll
        for (int j = 0; j < E; ++j) {
          // a list that is not full, or holds NaN, takes all
          if ((uint32_t)(bar >> 32) != 0u && !__any(v[j] >= bar_v)) continue;
          const int i = i0 + j;
          const uint64_t key = q < q1 && i >= lo && i < hi ? key_of(v[j], i) : 0u;
          const bool pass = key > bar;
          const uint64_t mask = __ballot(pass);
          if (pass) s_buf[wave][held + __popcll(mask & ((1ull << lane) - 1))] = key;
          held += __popcll(mask);
          __builtin_amdgcn_wave_barrier();  // a wave's LDS accesses keep their order
          if (held >= 64) {
            flush(64);
            if (lane < held - 64) s_buf[wave][lane] = s_buf[wave][64 + lane];
            __builtin_amdgcn_wave_barrier();
            held -= 64;
          }
        }
      }
    }
  };
  // two loads ahead
  uint4 u0[NL], u1[NL];
  int q = q0 + wave * 64;  // uniform
  load(q + lane, u0);
  load(q + kThreads + lane, u1);
  for (bool first = true; q < q1; q += 2 * kThreads) {
    take(q + lane, u0, first);
    first = false;
    load(q + 2 * kThreads + lane, u0);
    if (q + kThreads < q1) {
      take(q + kThreads + lane, u1, false);
      load(q + 3 * kThreads + lane, u1);
    }
  }
  if constexpr (TOP) {
    if (held > 0) flush(held);
    s_list[wave][lane] = list;
  }
  if (given) {  // equal logits of the 8 that hold the given one; of -inf all
    const bool least = gv == -__builtin_inff();
    const int to = min(id, hi), from = least ? lo : max((id + shift) / E * E - shift, lo);
    if (least || (id >= lo && id < hi))
      for (int i = from + wave * 64; i < to; i += kThreads)  // uniform
        rank += __popcll(__ballot(i + lane < to && logit<F32>(row, min(i + lane, to - 1)) == gv));
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
  if constexpr (TOP) {
    if (wave == 0) {
#pragma unroll
      for (int w = 1; w < kWaves; ++w) list = merge64(list, s_list[w][lane]);
    }
  }
  if (P.splits == 1) {
    finish_row<F32, kThreads>(P, t, row, gm, gb, g0, g1, gr, list);
    return;
  }
  if (tid == 0) reinterpret_cast<Piece*>(P.ws)[blockIdx.x] = Piece{g0, g1, gm, gb, gr, 0};
  if (TOP && tid < P.k)
    reinterpret_cast<uint64_t*>(P.ws + (int64_t)P.T * P.splits * sizeof(Piece))[(int64_t)blockIdx.x * P.k + tid] = list;
}

// A workgroup of NW waves: one row from its pieces, at most kMaxSplits.
constexpr int kMaxSplits = 64;
template <bool F32, bool TOP, int NW>
__global__ __launch_bounds__(64 * NW) void k_logprob_join(LogprobParams P) {
  __shared__ uint64_t s_list[TOP ? NW : 1][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, t = blockIdx.x;
  const uint8_t* row = static_cast<const uint8_t*>(P.logits) + (int64_t)t * P.ld * (F32 ? 4 : 2);
  const Piece* pc = reinterpret_cast<const Piece*>(P.ws) + (int64_t)t * P.splits;
  // lane l: piece l
  Piece p{0, 0, -__builtin_inff(), kLeast, 0, 0};
  if (lane < P.splits) p = pc[lane];
  uint64_t list = 0;
  if constexpr (TOP) {
    // the pieces' lists, those of a wave loaded at once
    const uint64_t* keys = reinterpret_cast<const uint64_t*>(P.ws + (int64_t)P.T * P.splits * sizeof(Piece)) +
                           (int64_t)t * P.splits * P.k;
    constexpr int PER = kMaxSplits / NW;
    uint64_t k[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int s = wave + i * NW;
      k[i] = s < P.splits && lane < P.k ? keys[(int64_t)s * P.k + lane] : 0u;
    }
    list = k[0];
#pragma unroll
    for (int i = 1; i < PER; ++i)
      if (i * NW < P.splits) list = merge64(list, k[i]);
    s_list[wave][lane] = list;
    // pairs of waves, then pairs of those
#pragma unroll
    for (int h = NW / 2; h > 0; h /= 2) {
      __syncthreads();
      if (wave < h) {
        list = merge64(list, s_list[wave + h][lane]);
        s_list[wave][lane] = list;
      }
    }
  }
  float m = p.m, b = p.b;
  double s0 = p.s0, s1 = p.s1;
  join_wave(m, b, s0, s1);
  int rank = p.rank;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) rank += __shfl_xor(rank, d);
  finish_row<F32, 64 * NW>(P, t, row, m, b, s0, s1, rank, list);
}

template <bool F32, bool TOP>
void launch_logprob(const LogprobParams& P, hipStream_t s) {
  launch(k_logprob<F32, TOP>, dim3((unsigned)((int64_t)P.T * P.splits)), dim3(kThreads), 0, s, P);
  if (P.splits > 16 && TOP) launch(k_logprob_join<F32, TOP, 16>, dim3((unsigned)P.T), dim3(1024), 0, s, P);
  else if (P.splits > 1) launch(k_logprob_join<F32, TOP, 4>, dim3((unsigned)P.T), dim3(256), 0, s, P);
}

// Pieces of a row: about eight workgroups a CU, none with less than 8 logits
// a thread.
int row_splits(int T, int V) {
  const int most = (V + 8 * kThreads - 1) / (8 * kThreads);
  return std::max(1, std::min({most, 2048 / T, kMaxSplits}));
}

bool bad_sizes(const moe_logprob_args* a) {
  return a->T < 0 || a->T >= (1 << 22) || a->V < 1 || a->V >= (1 << 30) || a->k < 0 || a->k > kMaxTop || a->k > a->V;
}

}  // namespace

extern "C" size_t moe_logprobs_workspace_size(const moe_logprob_args* a) {
  if (!a || a->T < 1 || bad_sizes(a)) return 0;
  const size_t n = row_splits(a->T, a->V);
  return n == 1 ? 0 : (size_t)a->T * n * (sizeof(Piece) + 8 * (size_t)a->k);
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
  if (a->logits_f32) top ? launch_logprob<true, true>(P, s) : launch_logprob<true, false>(P, s);
  else top ? launch_logprob<false, true>(P, s) : launch_logprob<false, false>(P, s);
  MOE_LAUNCHED();
  return MOE_OK;
}
