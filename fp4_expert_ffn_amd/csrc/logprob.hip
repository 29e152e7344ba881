// Log probabilities of given tokens, their ranks, the rows' entropies and the
// k most likely tokens, in one read of the logits (gfx950, wave64).
//
// With z = scale * l, m the row's largest logit and d_i = scale * (l_i - m):
//
//   s0 = sum exp(d_i), s1 = sum d_i exp(d_i)
//   lse = scale * m + log s0, log p_i = d_i - log s0, entropy = log s0 - s1 / s0
//
// A thread keeps its own maximum and sums over what it reads and rescales
// them when the maximum grows; threads, waves and the pieces of a row are
// joined the same way, in 64 bits.  The k best are keys of 64 bits (the
// logit's order, then the lower id), which a wave holds sorted over its lanes:
// logits that pass its k-th best are gathered in LDS, and every 64 of them are
// sorted and merged into the list, so that no order of the logits costs more
// than one sort per 64.
//
// Few rows are cut into pieces of one workgroup each, joined by a second
// kernel.
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

// What a piece of a row leaves: its maximum, the two sums in base 2 (s1 of
// log2(e) d), and the tokens in front of the given one.
struct Piece {
  double s0, s1;
  float m;
  int rank;
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

// Sums taken against maximum m as sums against a larger one (c: log2(e) scale).
template <typename F>
__device__ __forceinline__ void rebase(F& s0, F& s1, float m, float to, float c) {
  if (m == to) return;
  const F d = m == -__builtin_inff() ? (F)-2000 : (F)(m - to) * (F)c;  // nothing below: sums of 0
  const F f = (F)exp2((F)(d < (F)-1000 ? (F)-1000 : d));
  s1 = f * (s1 + (d < (F)-1000 ? (F)0 : d) * s0);
  s0 = f * s0;
}

template <bool F32>
__device__ __forceinline__ float logit(const void* row, int i) {
  return F32 ? static_cast<const float*>(row)[i] : bf16_to_f32(static_cast<const uint16_t*>(row)[i]);
}

// A row whose largest logit is infinite (nothing but -inf, or +inf among
// them), or that has a NaN logit (s0 is NaN then, as with +inf): the tokens
// equal to the maximum share it, and `nan` says whether there is a NaN.
template <bool F32>
__device__ void count_equal(const LogprobParams& P, const void* row, float m, int tid, int* s_equal, int* s_nan) {
  int n = 0, bad = 0;
  for (int i = tid; i < P.V; i += kThreads) {
    const float v = logit<F32>(row, i);
    n += v == m;
    bad |= v != v;
  }
  if (n) atomicAdd(s_equal, n);
  if (bad) atomicOr(s_nan, 1);
}

// The outputs of a row from its joined sums, by the whole workgroup: lane l
// of wave 0 holds the l-th best key.
template <bool F32>
__device__ __forceinline__ void finish_row(const LogprobParams& P, int t, const void* row, float m, double s0, double s1,
                                           int rank, uint64_t best) {
  __shared__ int s_equal, s_nan;
  const int tid = threadIdx.x;
  const bool odd = !(fabsf(m) < __builtin_inff()) || s0 != s0;
  bool nan = false;
  if (odd) {  // uniform
    if (tid == 0) s_equal = s_nan = 0;
    __syncthreads();
    count_equal<F32>(P, row, m, tid, &s_equal, &s_nan);
    __syncthreads();
    nan = s_nan != 0;
    s0 = s_equal;
    s1 = 0;
  }
  if (tid >= 64) return;
  const double log_s = nan ? (double)__builtin_nanf("") : log(s0);
  auto prob = [&](float v) {
    if (v == m) return -log_s;
    if (odd) return nan ? log_s : -(double)__builtin_inff();
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

// A workgroup: one piece of one row.
template <bool F32, bool TOP>
__global__ __launch_bounds__(kThreads) void k_logprob(LogprobParams P) {
  constexpr int E = F32 ? 4 : 8;  // logits of a 16-byte load
  __shared__ uint64_t s_buf[TOP ? kWaves : 1][128], s_list[TOP ? kWaves : 1][64];
  __shared__ double s_s0[kWaves], s_s1[kWaves];
  __shared__ float s_m[kWaves];
  __shared__ int s_rank[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int t = (int)(blockIdx.x / P.splits), sp = (int)(blockIdx.x % P.splits);
  const uint8_t* row = static_cast<const uint8_t*>(P.logits) + (int64_t)t * P.ld * (F32 ? 4 : 2);
  const int lo = sp * P.piece, hi = min(lo + P.piece, P.V);
  const int id = P.ids ? P.ids[t] : -1;
  const bool given = P.rank && id >= 0 && id < P.V;
  const unsigned ahead = (unsigned)max(min(id, hi) - lo, 0);  // tokens of this piece with a lower id
  const float gv = given ? logit<F32>(row, id) : __builtin_inff();  // nothing lies in front of +inf
  // 16-byte pieces of the row's memory: piece q holds logits q * E - shift ..
  const int shift = (int)(((uintptr_t)row & 15) / (F32 ? 4 : 2));
  const int q0 = (lo + shift) / E, q1 = (hi + shift + E - 1) / E;
  float m = -__builtin_inff(), s0 = 0.f, s1 = 0.f;
  int rank = 0;
  uint64_t list = 0, bar = 0;  // the wave's k best; the k-th
  float bar_v = -__builtin_inff();
  int held = 0;  // keys in the buffer (uniform)
  auto flush = [&](int n) {  // the buffer's first n <= 64 keys into the list
    const uint64_t key = lane < n ? s_buf[wave][lane] : 0u;
    list = merge64(list, sort64(key));
    const int l = P.k - 1;
    bar = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(list >> 32), l) << 32) |
          (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)list, l);
    bar_v = key_value(bar);
  };
  for (int qb = q0 + wave * 64; qb < q1; qb += kThreads) {
    const int q = qb + lane, i0 = q * E - shift;
    float v[E];
    const bool whole = q < q1 && i0 >= lo && i0 + E <= hi;
    if (whole) {
      const uint4 u = *reinterpret_cast<const uint4*>(row + (int64_t)i0 * (F32 ? 4 : 2));
      const uint32_t d[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (F32) {
          v[j] = __uint_as_float(d[j]);
        } else {
          v[2 * j] = __uint_as_float(d[j] << 16);
          v[2 * j + 1] = __uint_as_float(d[j] & 0xFFFF0000u);
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
      rebase(s0, s1, m, top, P.c);
      m = top;
    }
    const float base = m == -__builtin_inff() ? 0.f : m;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float d = (v[j] - base) * P.c;
      const float e = __builtin_amdgcn_exp2f(d);  // 0 at -inf; NaN stays
      s0 += e;
      s1 = fmaf(fmaxf(d, -200.f), e, s1);
    }
    if (given && __any(top >= gv)) {
#pragma unroll
      for (int j = 0; j < E; ++j) rank += v[j] > gv || (v[j] == gv && (unsigned)(i0 + j - lo) < ahead);
    }
    if constexpr (TOP) {
      // equal logits of a higher id never pass a full list; one that is not full, or holds NaN, takes all
      if ((uint32_t)(bar >> 32) == 0u || __any(top > bar_v)) {
#pragma unroll
        for (int j = 0; j < E; ++j) {
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
  }
  if constexpr (TOP) {
    if (held > 0) flush(held);
    s_list[wave][lane] = list;
  }
  // the waves' sums
  const float wm = wave_max(m);
  double d0 = s0, d1 = s1;
  rebase(d0, d1, m, wm, P.c);
  d0 = wave_sum64(d0);
  d1 = wave_sum64(d1);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) rank += __shfl_xor(rank, d);
  if (lane == 0) {
    s_m[wave] = wm;
    s_s0[wave] = d0;
    s_s1[wave] = d1;
    s_rank[wave] = rank;
  }
  __syncthreads();
  float gm = s_m[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) gm = fmaxf(gm, s_m[w]);
  double g0 = 0, g1 = 0;
  int gr = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    double a = s_s0[w], b = s_s1[w];
    rebase(a, b, s_m[w], gm, P.c);
    g0 += a;
    g1 += b;
    gr += s_rank[w];
  }
  if constexpr (TOP) {
    if (wave == 0) {
#pragma unroll
      for (int w = 1; w < kWaves; ++w) list = merge64(list, s_list[w][lane]);
    }
  }
  if (P.splits == 1) {
    finish_row<F32>(P, t, row, gm, g0, g1, gr, list);
    return;
  }
  if (tid == 0) reinterpret_cast<Piece*>(P.ws)[blockIdx.x] = Piece{g0, g1, gm, gr};
  if (TOP && tid < P.k)
    reinterpret_cast<uint64_t*>(P.ws + (int64_t)P.T * P.splits * sizeof(Piece))[(int64_t)blockIdx.x * P.k + tid] = list;
}

// A workgroup: one row from its pieces.
template <bool F32, bool TOP>
__global__ __launch_bounds__(kThreads) void k_logprob_join(LogprobParams P) {
  __shared__ uint64_t s_list[TOP ? kWaves : 1][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, t = blockIdx.x;
  const uint8_t* row = static_cast<const uint8_t*>(P.logits) + (int64_t)t * P.ld * (F32 ? 4 : 2);
  const Piece* pc = reinterpret_cast<const Piece*>(P.ws) + (int64_t)t * P.splits;
  uint64_t list = 0;
  if constexpr (TOP) {
    const uint64_t* keys = reinterpret_cast<const uint64_t*>(P.ws + (int64_t)P.T * P.splits * sizeof(Piece)) +
                           (int64_t)t * P.splits * P.k;
    for (int s = wave; s < P.splits; s += kWaves) {
      const uint64_t b = lane < P.k ? keys[(int64_t)s * P.k + lane] : 0u;
      list = merge64(list, b);
    }
    s_list[wave][lane] = list;
  }
  // every wave joins the sums: lane l those of pieces l, l + 64, ..
  float m = -__builtin_inff();
  for (int s = lane; s < P.splits; s += 64) m = fmaxf(m, pc[s].m);
  m = wave_max(m);
  double s0 = 0, s1 = 0;
  int rank = 0;
  for (int s = lane; s < P.splits; s += 64) {
    double a = pc[s].s0, b = pc[s].s1;
    rebase(a, b, pc[s].m, m, P.c);
    s0 += a;
    s1 += b;
    rank += pc[s].rank;
  }
  s0 = wave_sum64(s0);
  s1 = wave_sum64(s1);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) rank += __shfl_xor(rank, d);
  if constexpr (TOP) {
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int w = 1; w < kWaves; ++w) list = merge64(list, s_list[w][lane]);
    }
  }
  finish_row<F32>(P, t, row, m, s0, s1, rank, list);
}

template <bool F32, bool TOP>
void launch_logprob(const LogprobParams& P, hipStream_t s) {
  launch(k_logprob<F32, TOP>, dim3((unsigned)((int64_t)P.T * P.splits)), dim3(kThreads), 0, s, P);
  if (P.splits > 1) launch(k_logprob_join<F32, TOP>, dim3((unsigned)P.T), dim3(kThreads), 0, s, P);
}

// Pieces of a row: enough workgroups for the chip, none shorter than one
// 16-byte load a thread.
int row_splits(int T, int V, bool f32) {
  const int least = kThreads * (f32 ? 4 : 8);
  const int most = (V + least - 1) / least;
  return std::max(1, std::min(most, 512 / T));
}

bool bad_sizes(const moe_logprob_args* a) {
  return a->T < 0 || a->T >= (1 << 22) || a->V < 1 || a->V >= (1 << 30) || a->k < 0 || a->k > kMaxTop || a->k > a->V;
}

}  // namespace

extern "C" size_t moe_logprobs_workspace_size(const moe_logprob_args* a) {
  if (!a || a->T < 1 || bad_sizes(a)) return 0;
  const size_t n = row_splits(a->T, a->V, a->logits_f32 != 0);
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
  const int splits = row_splits(a->T, a->V, a->logits_f32 != 0);
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
