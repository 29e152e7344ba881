// The body of the tile kernels of the linear product (linear_tile.hip,
// linear_block_tile.hip) and the join of a split K.
#pragma once
#include <type_traits>

#include "ffn_common.h"
#include "linear.h"
#include "linear_block.h"

namespace moe {

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// Direct global->LDS loads of a wave: lane l's 16 (4) bytes at base + off
// land at dst + 16 l (4 l); dst is wave-uniform.  They write no register, and
// the kernel orders them by its own counted waits.  The compiler uses M0
// nowhere else in the kernels that call them (CPU tests check it).
__device__ __forceinline__ void dma16s(uint32_t off, const uint8_t* base, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(dst)
               : "memory", "m0");
}
__device__ __forceinline__ void dma4s(uint32_t off, const uint8_t* base, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "s"(dst)
               : "memory", "m0");
}
#pragma clang diagnostic pop

template <int N>
__device__ __forceinline__ void wait_loads() {  // at most N vector-memory operations outstanding
  static_assert(N >= 0 && N <= 63, "vmcnt range");
  constexpr int enc = (N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(enc);
  asm volatile("" ::: "memory");
}

struct LinTiles {
  int mt, nt;            // row and column tiles
  int vec_out, vec_res;  // 16-byte accesses of out and residual rows
  int splits, per;       // K in `splits` runs of `per` steps
  float* part;           // splits > 1: the sums [splits][T][R]
};

// One output tile a workgroup.
// WM x WN waves, each TM x TN 16 x 16 tiles; EXACT: E4M3 operands decoded to
// bf16 (fp32 outputs).  With K split, each tile's run of steps leaves its
// sums in G.part and k_linear_join makes the outputs of them.
//
// MOE_Q_FP8_BLOCK (B: what LinParams does not say): a step is a block of 128
// columns.  Its matrix instruction starts from zero, and its sums are added to
// the running ones times the scales' product: 4 FMA beside each instruction,
// some instructions late so that none waits for its own result.  The step's
// scales, the rows' and one of each 16 weight rows, ride in the ring.
// GROUPED: row tiles of the experts' rows, found from their offsets; the rows
// of x by index.
template <int QM, bool GATED, bool EXACT, bool GROUPED, int WM, int WN, int TM, int TN, int S>
__device__ __forceinline__ void tile_product(LinParams P, const LinTiles& G, const BlockParams* B) {
  constexpr int NW = WM * WN, BM = WM * TM * 16, BN = WN * TN * 16;
  constexpr int CA = BM / 8 / NW, CB = BN / 8 / NW;  // 1 KiB loads a wave and step
  constexpr bool MX = QM == MOE_Q_MXFP8, BLK = QM == MOE_Q_FP8_BLOCK;
  constexpr bool RS = MX || BLK;                     // scales in the ring
  constexpr int SC = BLK ? BM / 64 + 1 : (BM + BN) / 64;  // scale pieces of 64 words: 64 rows (the last of BLK: 16-row groups)
  constexpr int kStage = (BM + BN) * 128;
  constexpr int kScales = RS ? SC * 256 : 0;         // a step's scales, in a ring of S + 1
  constexpr int kWait = (S - 1) * (CA + CB + (RS ? 1 : 0));  // loads of S - 1 steps
  constexpr int TH = TM / 2;
  constexpr int OC = GATED ? TN / 2 : TN;            // 16-column groups of output a wave
  constexpr int BO = GATED ? BN / 2 : BN;            // output columns a tile
  constexpr int SR = OC * 16 + 4;                    // staging row, floats
  static_assert(CA * 8 * NW == BM && CB * 8 * NW == BN && SC <= NW && TN % 2 == 0 && CA % 2 == 0, "tile shape");
  static_assert(!RS || (BM % 64 == 0 && BN % 64 == 0), "whole scale pieces");
  static_assert(!BLK || TN * 16 <= 64, "a wave's weight rows lie in one block");
  static_assert(NW * 16 * SR * 4 <= S * kStage, "staging fits the ring");
  __shared__ __align__(1024) uint8_t ring[S * kStage];
  __shared__ __align__(256) uint8_t s_mx[RS ? (S + 1) * kScales : 16];
  __shared__ __align__(16) float s_ws[BN], s_bias[BN], s_xs[BM];  // scales and bias of the tile's rows

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int r16 = lane & 15, g = lane >> 4;

  // Workgroup b runs on XCD b % 8: each XCD takes a contiguous eighth of the
  // tile list, which walks blocks of 4 row tiles column by column, so that
  // the workgroups running at once on an XCD share operand rows in its L2.
  // Runs of a split K follow each other, the tiles of one run together.
  int mt = G.mt;
  if constexpr (GROUPED) mt = count_row_blocks<BM>(*B);
  const int tiles = mt * G.nt, total = tiles * G.splits, per = (total + 7) / 8;
  if (GROUPED && (int)(blockIdx.x / 8) >= per) return;  // the grid holds the most tiles there can be
  const int LS = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
  if (LS >= total) return;
  const int split = LS / tiles, L = LS - split * tiles;
  const int band = L / (4 * G.nt), in_band = L - band * 4 * G.nt;
  const int bh = min(4, mt - 4 * band);
  const int n0 = (in_band / bh) * BO;
  int t0 = (4 * band + in_band % bh) * BM, t_end = P.T;
  if constexpr (GROUPED) {
    const RowBlock rb = find_row_block<BM>(*B, 4 * band + in_band % bh);
    t0 = rb.t0;
    t_end = rb.end;
    if (t0 >= t_end) return;  // rows past the last of out
    to_slot(*B, rb.e, P);
  }

  const uint32_t ring0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)ring;
  const uint32_t mx0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)s_mx;
  const int k0 = split * G.per * 128, kb = min(P.kb - k0, G.per * 128);  // this run's bytes of a row
  const int steps = (kb + 127) / 128;
  const int tail = RS ? 0 : kb & 127;  // bytes of a partial last step, 0: none

  // ---- load addresses: piece (l % 8) ^ (row bits 3:1) of row 8 c + l / 8 of chunk c
  const uint8_t* abase = P.x + (GROUPED ? 0 : (int64_t)t0 * P.ldx) + k0;
  const uint8_t* bbase = P.w + (int64_t)n0 * P.ldw + k0;
  uint32_t aoff[CA], boff[CB];
  const int lr = lane >> 3;
  auto piece = [&](int c) { return (lane & 7) ^ ((4 * (c & 1) + (lr >> 1)) & 7); };
  // A chunk u of this wave: the first CA / 2 hold rows of the waves' first
  // TH tiles, the others rows of the second
  auto a_chunk = [&](int u) {
    const int h = u / (CA / 2), n = wave * (CA / 2) + u % (CA / 2);
    return n / (2 * TH) * (2 * TM) + n % (2 * TH) + h * 2 * TH;
  };
#pragma unroll
  for (int u = 0; u < CA; ++u) {
    const int c = a_chunk(u);
    const int i = min(8 * c + lr, t_end - 1 - t0);
    aoff[u] = (uint32_t)(GROUPED ? x_row(*B, t0 + i) : i) * (uint32_t)P.ldx + piece(c) * 16;
  }
#pragma unroll
  for (int u = 0; u < CB; ++u) {
    const int c = wave * CB + u, j = 8 * c + lr;
    const int col = GATED ? (j >> 5) * 16 + (j & 15) : j;
    boff[u] = (uint32_t)min(col, P.N - 1 - n0) * (uint32_t)P.ldw + piece(c) * 16;
  }
  uint32_t soff = 0;
  const uint8_t* sbase = nullptr;
  int64_t sstep = 0;
  const int sc = wave % SC;
  if constexpr (MX) {
    const int j = 64 * sc + lane;
    if (sc < BM / 64) {
      soff = (uint32_t)min(t0 + j, P.T - 1) * 4u;
      sbase = static_cast<const uint8_t*>(P.xs);
      sstep = (int64_t)P.T * 4;
    } else {
      const int jb = j - BM;
      const int col = min(n0 + (GATED ? (jb >> 5) * 16 + (jb & 15) : jb), P.N - 1);
      soff = (uint32_t)((GATED && ((jb >> 4) & 1) ? P.N : 0) + col) * 4u;
      sbase = static_cast<const uint8_t*>(P.ws);
      sstep = (int64_t)P.R * 4;
    }
    sbase += split * (int64_t)G.per * sstep;
  }
  if constexpr (BLK) {
    if (sc < BM / 64) {
      const int t = min(t0 + 64 * sc + lane, t_end - 1);
      soff = (uint32_t)(GROUPED ? x_row(*B, t) : t) * 4u;
      sbase = static_cast<const uint8_t*>(P.xs);
      sstep = (int64_t)B->X * 4;
    } else {  // the row block of each 16-row group: gate and up by turns
      const int q = min(lane, BN / 16 - 1);
      const int c = min(n0 + (GATED ? (q >> 1) * 16 : q * 16), P.N - 1) >> 7;
      soff = (uint32_t)((GATED && (q & 1) ? B->nb : 0) + c) * (uint32_t)B->steps * 4u;
      sbase = static_cast<const uint8_t*>(P.ws);
      sstep = 4;
    }
    sbase += split * (int64_t)G.per * sstep;
  }
  const int64_t up = GATED ? (int64_t)P.N * P.ldw : 0;
  // a partial step's pieces past the row's end re-read its last piece
  const uint32_t back0 = tail != 0 ? (uint32_t)max(piece(0) * 16 - (tail - 16), 0) : 0u;  // even chunks
  const uint32_t back1 = tail != 0 ? (uint32_t)max(piece(1) * 16 - (tail - 16), 0) : 0u;  // odd chunks
  // The load side: step f goes to the stage at ring offset `fill`, in two
  // parts: the weights, the scales and the first half of x; the second half
  // of x.  Past the end the last step again (the counted waits need the same
  // number of loads every step).  Running pointers and offsets: products and
  // remainders of the step number would stand in every wave's way.
  const uint8_t *pa = abase, *pb = bbase, *ps = sbase;
  uint32_t cut = steps == 1 ? ~0u : 0u;  // all ones from the last step on
  uint32_t fill = 0, fill_mx = 0;
  int f = 0;
  auto load_a = [&](int u) __attribute__((always_inline)) {
    const int c = a_chunk(u);
    dma16s(aoff[u] - ((c & 1 ? back1 : back0) & cut), pa, ring0 + fill + c * 1024);
  };
  // load k of part 1
  constexpr int kPart1 = CB + CA / 2 + (RS ? 1 : 0);
  auto load1 = [&](int k) __attribute__((always_inline)) {
    if (k < CB) {
      const int c = wave * CB + k;
      dma16s(boff[k < CB ? k : 0] - ((c & 1 ? back1 : back0) & cut), pb + (GATED && ((c >> 1) & 1) ? up : 0),
             ring0 + fill + BM * 128 + c * 1024);
    } else if (k < CB + CA / 2) {
      load_a(k - CB);
    } else if (RS && k == CB + CA / 2) {
      dma4s(soff, ps, mx0 + fill_mx + sc * 256);
    }
  };
  // after both parts of a step
  auto filled = [&]() __attribute__((always_inline)) {
    ++f;
    if (f < steps) {
      pa += 128;
      pb += 128;
      if constexpr (RS) ps += sstep;
    }
    cut = f >= steps - 1 ? ~0u : 0u;
    if constexpr (RS) fill_mx = fill_mx == S * kScales ? 0 : fill_mx + kScales;
    fill = fill == (S - 1) * kStage ? 0 : fill + kStage;
  };
  auto issue = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kPart1; ++k) load1(k);
#pragma unroll
    for (int u = CA / 2; u < CA; ++u) load_a(u);
    filled();
  };

  lf32x4_t acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = lf32x4_t{0.f, 0.f, 0.f, 0.f};

  // fragment row r16 of a 16-row group: pieces g and 4 + g (64 bytes apart in the permuted row too)
  const uint32_t rd = r16 * 128 + ((g ^ (r16 >> 1)) << 4);
  const uint32_t rda = wm * TM * 2048 + rd, rdb = BM * 128 + wn * TN * 2048 + rd;
  const uint32_t rda4 = rda ^ 64, rdb4 = rdb ^ 64;
  const uint32_t rsa = (wm * TM * 16 + r16) * 4, rsb = BLK ? (BM + wn * TN) * 4 : (BM + wn * TN * 16 + r16) * 4;

  auto frag = [&](const uint8_t* p, const uint8_t* p4) __attribute__((always_inline)) {
    Frag f;
    f.a = *reinterpret_cast<const uint4*>(p);
    f.b = *reinterpret_cast<const uint4*>(p4);
    return f;
  };
  // The matrix step of fragments j and i.  Block scales: the instruction
  // takes one byte of a register (its number a constant), so the scales of a
  // half's fragments share one.
  static_assert(TH <= 4 && TN <= 4, "scale bytes of a half");
  Frag fw[TN], fx[TM];
  int sw = 0x7F7F7F7F, sx[2] = {0x7F7F7F7F, 0x7F7F7F7F};            // MX
  uint32_t rw[MX ? TN : 1], rx[MX ? TH : 1];                        // MX: scale bytes as read
  uint32_t ew[MX && EXACT ? TN : 1], ex[MX && EXACT ? TM : 1];     // MX, EXACT: the rows' four scales
  float bw[BLK ? 2 : 1], bx[BLK ? TH : 1];  // BLK: scales of the step's weights (gated: gate, up), of the half's rows
  float nw[BLK ? 2 : 1], nx[BLK ? TH : 1];  // those of the next step, of the next half
  // sums of the last instructions, not added yet, and their scales: instruction
  // n of a half leaves its own in place n % kLate, whose former ones are added first
  constexpr int kLate = EXACT ? 2 : 4;
  lf32x4_t late[BLK ? kLate : 1];
  float late_f[BLK ? kLate : 1];
  static_assert(!BLK || TN * TH % kLate == 0, "places go on from half to half");
  // adds what instruction kLate before number n of half h left (n < kLate: of the other half)
  auto settle = [&](auto nc, auto hc) __attribute__((always_inline)) {
    constexpr int N = TN * TH, n = decltype(nc)::value, k = (n + N - kLate) % N;
    constexpr int h = n < kLate ? 1 - decltype(hc)::value : decltype(hc)::value, j = k / TH, i = h * TH + k % TH;
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(late[n % kLate][v], late_f[n % kLate], acc[i][j][v]);
  };
  auto mma = [&](auto jc, auto ic) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value, i = decltype(ic)::value;
    if constexpr (BLK) {
      constexpr int n = j * TH + i % TH, l = n % kLate;
      settle(std::integral_constant<int, n>{}, std::integral_constant<int, i / TH>{});
      __builtin_amdgcn_sched_barrier(0);
      lf32x4_t c = lf32x4_t{0.f, 0.f, 0.f, 0.f};
      if constexpr (EXACT) c = mma_decoded<false>(fw[j], fx[i], c, 0, 0, g);
      else c = mma_fp8<0, 0>(fw[j], fx[i], c, 0x7F7F7F7F, 0x7F7F7F7F);
      late[l] = c;
      late_f[l] = bx[i % TH] * bw[GATED ? j & 1 : 0];
      __builtin_amdgcn_sched_barrier(0);
      return;
    }
    lf32x4_t c = acc[i][j];
    if constexpr (QM == MOE_Q_NONE) c = mma_bf16_step(fw[j], fx[i], c);
    else if constexpr (EXACT) c = mma_decoded<MX>(fw[j], fx[i], c, MX ? ew[MX ? j : 0] : 0, MX ? ex[MX ? i : 0] : 0, g);
    else c = mma_fp8<j, i % TH>(fw[j], fx[i], c, sw, sx[i / TH]);
    acc[i][j] = c;
  };
  // Fragments of the step in work; the halves of fx are read half a step apart.
  auto read_w = [&](const uint8_t* st, const uint8_t* mx, int j) __attribute__((always_inline)) {
    if constexpr (MX && EXACT) ew[j] = *reinterpret_cast<const uint32_t*>(mx + rsb + j * 64);
    if constexpr (MX && !EXACT) rw[j] = mx[rsb + g + j * 64];
    fw[j] = frag(st + rdb + j * 2048, st + rdb4 + j * 2048);
    if constexpr (BLK) nw[j & 1] = *reinterpret_cast<const float*>(mx + rsb + (j & 1) * 4);
  };
  auto read_x = [&](const uint8_t* st, const uint8_t* mx, int half) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TH; ++i) {
      if constexpr (MX && EXACT) ex[half * TH + i] = *reinterpret_cast<const uint32_t*>(mx + rsa + (half * TH + i) * 64);
      if constexpr (MX && !EXACT) rx[i] = mx[rsa + g + (half * TH + i) * 64];
      if constexpr (BLK) nx[i] = *reinterpret_cast<const float*>(mx + rsa + (half * TH + i) * 64);
    }
#pragma unroll
    for (int i = half * TH; i < (half + 1) * TH; ++i)
      fx[i] = frag(st + rda + i * 2048, st + rda4 + i * 2048);
  };
  // the scale bytes read by read_x / read_w as the instruction takes them
  auto pack = [&](const uint32_t* r, int n) __attribute__((always_inline)) {
    uint32_t p = r[0];
#pragma unroll
    for (int i = 1; i < n; ++i) p |= r[i] << (8 * i);
    return (int)p;
  };
  // Fragment j of the weights against half h of x.  S = 2: part 1 of step s
  // is loaded beside the first half, part 2 beside the second, spread between
  // the matrix instructions: issued together they would hold back every
  // wave's instructions behind the texture unit (3 us less at the FP8
  // and MXFP8 prefills above).
  auto mma_j = [&](auto jc, auto hc) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value, h = decltype(hc)::value;
    constexpr int from = S == 2 && h == 1 ? kPart1 : 0;           // loads [from, to) beside this half
    constexpr int to = S > 2 ? 0 : (h == 0 ? kPart1 : kPart1 + CA / 2);
    constexpr int slots = TN * TH;
    auto one = [&](auto ic) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value, at = j * TH + i;
      mma(jc, std::integral_constant<int, h * TH + i>{});
      constexpr int k0 = from + (to - from) * at / slots, k1 = from + (to - from) * (at + 1) / slots;
      if constexpr (k1 > k0) {
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = k0; k < k1; ++k) {
          if (k < kPart1) load1(k);
          else load_a(CA / 2 + k - kPart1);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    one(std::integral_constant<int, 0>{});
    if constexpr (TH > 1) one(std::integral_constant<int, 1>{});
    if constexpr (TH > 2) one(std::integral_constant<int, 2>{});
    if constexpr (TH > 3) one(std::integral_constant<int, 3>{});
  };
  // the pieces of a partial step past the rows' end: zero
  auto zero_tail = [&](uint8_t* st) __attribute__((always_inline)) {
    wait_loads<0>();
    lds_sync();
    for (int i = tid; i < (BM + BN) * 8; i += 64 * NW) {
      const int row = i >> 3, pc = (i & 7) ^ ((row >> 1) & 7);
      if (pc * 16 >= tail) *reinterpret_cast<uint4*>(st + i * 16) = make_uint4(0, 0, 0, 0);
    }
    lds_sync();
  };
  // BLK: the next half's scales
  auto end_half = [&](auto hc) __attribute__((always_inline)) {
    if constexpr (BLK) {
#pragma unroll
      for (int i = 0; i < TH; ++i) bx[i] = nx[i];
      if constexpr (decltype(hc)::value == 1) bw[0] = nw[0], bw[1] = nw[1];
    }
  };
  // the sums stay where they are: no matrix instruction moves past this
  auto pin = [&](int i0, int i1) __attribute__((always_inline)) {
#pragma unroll
    for (int i = i0; i < i1; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) asm volatile("" : "+v"(acc[i][j]));
  };

#pragma unroll
  for (int s = 0; s < S; ++s) issue();
  for (int i = tid; i < BN; i += 64 * NW) {
    const int col = min(n0 + (GATED ? (i >> 5) * 16 + (i & 15) : i), P.N - 1) + (GATED && ((i >> 4) & 1) ? P.N : 0);
    if constexpr (QM == MOE_Q_FP8) s_ws[i] = static_cast<const float*>(P.ws)[col];
    s_bias[i] = P.bias ? P.bias[col] : 0.f;
  }
  if constexpr (QM == MOE_Q_FP8)
    for (int i = tid; i < BM; i += 64 * NW) s_xs[i] = static_cast<const float*>(P.xs)[min(t0 + i, P.T - 1)];
  wait_loads<kWait>();
  lds_sync();
  if (!RS && tail != 0 && steps == 1) zero_tail(ring);
#pragma unroll
  for (int j = 0; j < TN; ++j) read_w(ring, s_mx, j);
  read_x(ring, s_mx, 0);
  if constexpr (MX && !EXACT) {
    sw = pack(rw, TN);
    sx[0] = pack(rx, TH);
  }
  if constexpr (BLK) {
    bw[0] = nw[0], bw[1] = nw[1];
#pragma unroll
    for (int i = 0; i < TH; ++i) bx[i] = nx[i];
#pragma unroll
    for (int l = 0; l < kLate; ++l) {
      late[l] = lf32x4_t{0.f, 0.f, 0.f, 0.f};
      late_f[l] = 0.f;
    }
  }
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2 % TN>;
  using I3 = std::integral_constant<int, 3 % TN>;
  // Step s, whose weights and first half of x are in registers.  First half:
  // tokens 0 .. TH - 1 of the wave's tiles, while the other tokens' fragments
  // are read.  Second half: the other tokens, while step s + 1's fragments
  // replace those used up.  Before the second half every wave has read the
  // whole stage.  S = 2: part 1 of step s + 2 already refills, beside the
  // first half, what every wave had read by then, at the price of a second
  // barrier, so that a load has a step and a half to land; with S = 3 two
  // steps are in flight, and one barrier with the loads right behind it is
  // faster (4096 x 2048 x 2048 bf16, 128 x 256 tiles: 36 against 44 us; loads
  // spread between the matrix instructions 41).
  uint32_t at = 0, at_mx = 0;  // stage of step s
#pragma unroll 1
  for (int s = 0; s < steps; ++s) {
    const uint8_t* st = ring + at;
    const uint8_t* mx = s_mx + at_mx;
    at = at == (S - 1) * kStage ? 0 : at + kStage;
    if constexpr (RS) at_mx = at_mx == S * kScales ? 0 : at_mx + kScales;
    uint8_t* nx = ring + at;
    const uint8_t* mxn = s_mx + at_mx;
    if constexpr (S == 2) {
      wait_loads<kWait>();  // part 2 of step s
      lds_sync();
    }
    read_x(st, mx, 1);
    __builtin_amdgcn_sched_barrier(0);
    mma_j(I0{}, I0{});
    mma_j(I1{}, I0{});
    if constexpr (TN > 2) mma_j(I2{}, I0{});
    if constexpr (TN > 3) mma_j(I3{}, I0{});
    end_half(I0{});
    pin(0, TH);
    if constexpr (MX && !EXACT) sx[1] = pack(rx, TH);
    wait_loads<S == 2 ? kWait : kWait - kWait / (S - 1)>();  // S = 2: part 1 of step s + 1; else both parts
    lds_sync();
    if (!RS && tail != 0 && s == steps - 2) zero_tail(nx);
    if constexpr (S > 2) issue();
    read_x(nx, mxn, 0);
    auto second = [&](auto jc) __attribute__((always_inline)) {
      __builtin_amdgcn_sched_barrier(0);
      mma_j(jc, I1{});
      __builtin_amdgcn_sched_barrier(0);
      read_w(nx, mxn, decltype(jc)::value);
    };
    second(I0{});
    second(I1{});
    if constexpr (TN > 2) second(I2{});
    if constexpr (TN > 3) second(I3{});
    end_half(I1{});
    pin(TH, TM);
    if constexpr (S == 2) filled();
    if constexpr (MX && !EXACT) {
      sw = pack(rw, TN);
      sx[0] = pack(rx, TH);
    }
  }
  if constexpr (BLK) {  // what the last half left
    settle(I0{}, I0{});
    settle(std::integral_constant<int, 1>{}, I0{});
    if constexpr (kLate > 2) {
      settle(std::integral_constant<int, 2>{}, I0{});
      settle(std::integral_constant<int, 3>{}, I0{});
    }
  }
  // (the largest tile never splits: its grids fill the chip)
  if constexpr (TM * TN <= 16 && !GROUPED) if (G.splits > 1) {
    // the sums as they are, 4 columns a lane
    float* part = G.part + (int64_t)split * P.T * P.R;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const int q = wn * TN + j;  // 16-row group of the tile
      const int c = n0 + (GATED ? (q >> 1) * 16 : q * 16) + 4 * g;
      const int64_t row0 = GATED && (q & 1) ? P.N : 0;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int t = t0 + (wm * TM + i) * 16 + r16;
        if (t >= P.T) continue;
        float* d = part + (int64_t)t * P.R + row0 + c;
        if (c + 4 <= P.N && P.N % 4 == 0) {
          *reinterpret_cast<float4*>(d) = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (c + v < P.N) d[v] = acc[i][j][v];
        }
      }
    }
    wait_loads<0>();  // no load into LDS outlives the workgroup
    return;
  }
  // ---- epilogue.  Lane: token r16 of a 16-token group, weight rows 4 g + v
  // of a group: scales, bias, activation and gate in place; then, through LDS
  // in fp32, rows of 8 columns a lane: the residual and whole 16-byte stores.
  constexpr int LPR = OC * 2, RP = 64 / LPR, PS = 16 / RP;  // lanes a row, rows a pass, passes
  const int er = lane / LPR, ec = n0 + wn * OC * 16 + (lane % LPR) * 8;
  const int tw = t0 + wm * TM * 16;  // the wave's first token
  // residual rows, four groups ahead of their stores (out may be the
  // residual: a lane reads and writes the same places)
  constexpr int RD = TM < 4 ? TM : 4;
  uint4 rr[RD][PS];
  const bool whole = ec + 8 <= P.N && G.vec_out && (G.vec_res || !P.res);
  auto load_res = [&](int i) __attribute__((always_inline)) {
    if (P.res && whole) {
#pragma unroll
      for (int p = 0; p < PS; ++p) {
        const int t = tw + i * 16 + p * RP, rows = t_end - t;  // uniform
        if (rows > 0)
          rr[i % RD][p] = *reinterpret_cast<const uint4*>(P.res + (int64_t)t * P.ldr +
                                                          (uint32_t)(min(er, rows - 1) * (int)P.ldr + ec));
      }
    }
  };
#pragma unroll
  for (int i = 0; i < RD; ++i) load_res(i);
  wait_loads<0>();
  lds_sync();  // nothing reads or fills the ring any more: its memory takes the staging rows
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const float4 b4 = *reinterpret_cast<const float4*>(s_bias + (wn * TN + j) * 16 + 4 * g);
    const float bj[4] = {b4.x, b4.y, b4.z, b4.w};
    float wj[4] = {1.f, 1.f, 1.f, 1.f};
    if constexpr (QM == MOE_Q_FP8) {
      const float4 w4 = *reinterpret_cast<const float4*>(s_ws + (wn * TN + j) * 16 + 4 * g);
      wj[0] = w4.x, wj[1] = w4.y, wj[2] = w4.z, wj[3] = w4.w;
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      float xs = 1.f;
      if constexpr (QM == MOE_Q_FP8) xs = s_xs[(wm * TM + i) * 16 + r16];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        if constexpr (QM == MOE_Q_FP8) acc[i][j][v] = fmaf(acc[i][j][v], xs * wj[v], bj[v]);
        else acc[i][j][v] += bj[v];
      }
    }
  }
  auto activate = [&](int i, auto fc) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < TN; j += GATED ? 2 : 1)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][j][v] = act_of<decltype(fc)::value>(acc[i][j][v]);
  };
  float* stg = reinterpret_cast<float*>(ring) + wave * 16 * SR;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    switch (P.fn) {
      case MOE_FN_SILU: activate(i, std::integral_constant<int, MOE_FN_SILU>{}); break;
      case MOE_FN_GELU_TANH: activate(i, std::integral_constant<int, MOE_FN_GELU_TANH>{}); break;
      case MOE_FN_GELU_ERF: activate(i, std::integral_constant<int, MOE_FN_GELU_ERF>{}); break;
      case MOE_FN_RELU: activate(i, std::integral_constant<int, MOE_FN_RELU>{}); break;
      default: break;
    }
#pragma unroll
    for (int o = 0; o < OC; ++o) {
      float y[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) y[v] = GATED ? acc[i][2 * o][v] * acc[i][2 * o + 1][v] : acc[i][o][v];
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
          const uint4 q = rr[i % RD][p];
          const uint32_t d[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[2 * e] += __uint_as_float(d[e] << 16);
            y[2 * e + 1] += __uint_as_float(d[e] & 0xFFFF0000u);
          }
        }
        const int64_t ob = (int64_t)(tw + i * 16 + p * RP) * P.ldo;  // uniform
        const uint32_t ol = (uint32_t)(er * (int)P.ldo + ec);
        if (P.out_f32) {
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(P.out) + ob + ol);
          o[0] = make_float4(y[0], y[1], y[2], y[3]);
          o[1] = make_float4(y[4], y[5], y[6], y[7]);
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.out) + ob + ol) = make_uint4(
              bf16x2_rne(y[0], y[1]), bf16x2_rne(y[2], y[3]), bf16x2_rne(y[4], y[5]), bf16x2_rne(y[6], y[7]));
        }
      } else if (t < t_end) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (ec + e < P.N)
            put(P, t, ec + e, P.res ? y[e] + bf16_to_f32(P.res[(int64_t)t * P.ldr + ec + e]) : y[e]);
      }
    }
    asm volatile("" ::: "memory");
    if (i + RD < TM) load_res(i + RD);
  }
}

// The tiles of the linear product (linear_tile.hip).
template <int QM, bool GATED, bool EXACT, int WM, int WN, int TM, int TN, int S>
__global__ __launch_bounds__(64 * WM* WN) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_linear_tile(LinParams P,
                                                                                                        LinTiles G) {
  tile_product<QM, GATED, EXACT, false, WM, WN, TM, TN, S>(P, G, nullptr);
}

// Those with a scale per block of 128, dense and grouped (linear_block_tile.hip).
template <bool GATED, bool EXACT, bool GROUPED, int WM, int WN, int TM, int TN, int S>
__global__ __launch_bounds__(64 * WM* WN) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_block_tile(BlockParams B,
                                                                                                       LinTiles G) {
  tile_product<MOE_Q_FP8_BLOCK, GATED, EXACT, GROUPED, WM, WN, TM, TN, S>(B.L, G, &B);
}

// The outputs of a split K: the runs' sums added in order, then the
// epilogue.  One thread a column of a token.
template <int QM, bool GATED>
__global__ __launch_bounds__(256) void k_linear_join(LinParams P, const float* __restrict__ part, int splits) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)P.T * P.N) return;
  const int t = (int)(i / P.N), n = (int)(i - (int64_t)t * P.N);
  const float* p = part + (int64_t)t * P.R + n;
  const int64_t run = (int64_t)P.T * P.R;
  float a = 0.f, u = 0.f;
  Epilogue<QM, GATED> e;
  e.load(P, t, n);
  for (int s0 = 0; s0 < splits; s0 += 4) {
    float v[4], w[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const float* q = p + min(s0 + s, splits - 1) * run;
      v[s] = q[0];
      if (GATED) w[s] = q[P.N];
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s0 + s < splits) {
        a += v[s];
        if (GATED) u += w[s];
      }
    }
  }
  put(P, t, n, e.finish(P, a, u));
}

}  // namespace moe
