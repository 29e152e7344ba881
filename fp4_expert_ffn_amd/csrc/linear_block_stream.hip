// The FP8 product with a scale per block of 128 for many tiles of short rows
// of work (the experts' row blocks): 128 rows x 128 weight rows, four waves of
// 64 x 64, two workgroups a CU that walk their tiles without a pause.
//
// Bound: the way into LDS (32 KiB a step of 512 matrix cycles), the latency of
// weights that come from HBM and, with a workgroup a tile, each tile's start:
// its place among the experts, its rows, its first loads.  Here the load side
// runs two steps ahead of the compute side across the tiles' borders, so that
// a tile's first stages land while the one before is finished; the tiles'
// places are looked up once, at the start, and their row numbers ride in the
// ring's loads.
//
// 4096 tokens by 8 of 128 experts: 2 x 768 x 2048 175 us (198 with a workgroup a
// tile), 2048 x 768 112 (149).  Matrix cores 0.34 busy, texture unit 0.68, L2
// hits 0.66, 692 MB fetched of 411 read once: a band of four row tiles takes in
// several experts, some 170 passes over an expert's weights for 128 of them; a
// quarter of the matrix instructions is for empty rows of last tiles.  With
// weights that the L2 holds already 23 us less.
//
// One step in four parts as in linear_block_big.hip, part i the wave's i-th 16
// rows.  When a step starts, its weights and the first half of its x are in
// every wave's registers: their places take those of step s + 2 (parts 0 and
// 1), those of the other half of x the rest (parts 2 and 3).  A load has a
// step to a step and a half to land.
#include <algorithm>
#include <type_traits>

#include "linear_block.h"
#include "linear_block_epilogue.h"
#include "linear_block_plan.h"

namespace moe {

namespace {

struct __align__(16) Tile {  // read in one 16-byte piece
  int t0, end, n0, slot;
};

template <bool GATED, bool GROUPED>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_block_stream(BlockParams B, LinTiles G) {
  constexpr int WM = 2, WN = 2, TM = 4, TN = 4, BM = 128, BN = 128;
  constexpr int BO = GATED ? BN / 2 : BN;
  constexpr uint32_t kHalf = 128 * 128, kStage = 2 * kHalf;  // x rows, weight rows of a step
  constexpr uint32_t kScales = 3 * 256;                      // a step's scales: 128 rows, 8 groups of weight rows
  constexpr int kRows = 4;                                   // tiles whose row numbers are held
  __shared__ __align__(1024) uint8_t ring[2 * kStage];
  __shared__ __align__(256) uint8_t s_sc[3 * kScales];
  __shared__ __align__(256) int s_rows[GROUPED ? kRows : 1][BM];
  __shared__ __align__(16) float s_stage[4 * 16 * 36];
  __shared__ Tile s_tile[kStreamTiles];
  const LinParams P = B.L;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN, r16 = lane & 15, g = lane >> 4, lr = lane >> 3;

  // ---- this workgroup's tiles.  The list and its eighths for the XCDs are
  // those of tile_product; the workgroups of an XCD deal its eighth out.
  int mt = G.mt, *prefix = reinterpret_cast<int*>(ring);
  if constexpr (GROUPED) {
    // row blocks up to and with each expert's, in the ring's memory
    if (wave == 0) {
      int before = 0;
      for (int e0 = 0; e0 < B.E; e0 += 64) {
        const int e = e0 + lane;
        const int lo = B.offsets[min(e, B.E)], hi = B.offsets[min(e + 1, B.E)];
        const int sum = before + wave_scan((max(hi - lo, 0) + BM - 1) / BM);
        if (e < B.E) prefix[e] = sum;
        before = __builtin_amdgcn_readlane(sum, 63);
      }
    }
    __syncthreads();
    mt = prefix[B.E - 1];
  }
  const int total = mt * G.nt, per = (total + 7) / 8;
  const int xcd = (int)(blockIdx.x % 8), w0 = (int)(blockIdx.x / 8), dealt = (int)(gridDim.x / 8);
  const int mine = min(per, total - xcd * per) - w0;
  // at most kStreamTiles by the host's choice, whatever the offsets hold
  const int n = __builtin_amdgcn_readfirstlane(mine <= 0 ? 0 : min((mine + dealt - 1) / dealt, kStreamTiles));
  if (n == 0) return;  // whole workgroups leave
  if (tid < n) {
    const int L = xcd * per + w0 + tid * dealt;
    const int band = L / (4 * G.nt), in_band = L - band * 4 * G.nt, bh = min(4, mt - 4 * band);
    const int b = 4 * band + in_band % bh;
    Tile t{b * BM, P.T, (in_band / bh) * BO, 0};
    if constexpr (GROUPED) {
      int lo = 0, hi = B.E - 1;  // the first expert whose blocks pass b
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] > b) hi = mid;
        else lo = mid + 1;
      }
      t.t0 = B.offsets[lo] + (b - (lo ? prefix[lo - 1] : 0)) * BM;
      t.end = min(B.offsets[lo + 1], P.T);
      t.slot = B.slot ? B.slot[lo] : lo;
      if (t.t0 >= t.end) t.t0 = t.end = 0;  // rows past the last of out: none
    }
    s_tile[tid] = t;
  }
  __syncthreads();

  const int steps = B.steps;
  const uint32_t ring0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)ring;
  const uint32_t sc0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)s_sc;
  const uint32_t rows0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)&s_rows[0][0];
  auto tile_at = [&](int k) __attribute__((always_inline)) {
    const int4 v = *reinterpret_cast<const int4*>(&s_tile[k]);
    return Tile{__builtin_amdgcn_readfirstlane(v.x), __builtin_amdgcn_readfirstlane(v.y),
                __builtin_amdgcn_readfirstlane(v.z), __builtin_amdgcn_readfirstlane(v.w)};
  };

  // ---- load side: chunks of 8 rows, piece (l % 8) ^ (row bits 3:1).  Weights: chunk 4 wave + u; x: chunks u < 2
  // hold rows of the waves' first two row groups, the others rows of the last two.
  auto a_chunk = [&](int u) {
    const int c = wave * 2 + (u & 1);
    return c / 4 * 8 + c % 4 + (u >> 1) * 4;
  };
  auto piece = [&](int c) { return (lane & 7) ^ ((4 * (c & 1) + (lr >> 1)) & 7); };
  uint32_t aoff[4], boff[4], soff = 0;
  const uint8_t *pa = nullptr, *pb = nullptr, *ps = nullptr;
  const int sc = wave % 3;
  const int64_t sstep = sc < 2 ? (int64_t)B.X * 4 : 4;
  const int64_t up = GATED ? (int64_t)P.N * P.ldw : 0;
  const bool by_rows = GROUPED && B.rows;
  // the row numbers of tile k, 64 by two waves each
  auto load_rows = [&](int k) __attribute__((always_inline)) {
    const Tile t = tile_at(k);
    const int h = wave & 1;
    dma4s((uint32_t)min(64 * h + lane, max(t.end - 1 - t.t0, 0)) * 4u, reinterpret_cast<const uint8_t*>(B.rows + t.t0),
          rows0 + (uint32_t)(k % kRows) * (BM * 4) + h * 256);
  };
  auto row_of = [&](const Tile& t, int k, int i) __attribute__((always_inline)) {  // of x, for the tile's row i
    const int j = min(i, max(t.end - 1 - t.t0, 0));
    if (!GROUPED) return (uint32_t)(t.t0 + j);
    const uint32_t r = by_rows ? (uint32_t)s_rows[k % kRows][j] / (uint32_t)B.div : (uint32_t)(t.t0 + j);
    return r < (uint32_t)B.X ? r : (uint32_t)(B.X - 1);
  };
  // the load side goes to tile k's first step
  auto to_tile = [&](int k) __attribute__((always_inline)) {
    const Tile t = tile_at(k);
    const uint32_t first = GROUPED ? 0u : (uint32_t)t.t0;  // dense: 32-bit offsets inside the tile
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = a_chunk(u);
      aoff[u] = (row_of(t, k, 8 * c + lr) - first) * (uint32_t)P.ldx + piece(c) * 16;
    }
    pa = P.x + (int64_t)first * P.ldx;
    if (sc < 2) {
      soff = row_of(t, k, 64 * sc + lane) * 4u;
      ps = static_cast<const uint8_t*>(P.xs);
    } else {
      const int q = min(lane, BN / 16 - 1);
      const int c = min(t.n0 + (GATED ? (q >> 1) * 16 : q * 16), P.N - 1) >> 7;
      soff = (uint32_t)((GATED && (q & 1) ? B.nb : 0) + c) * (uint32_t)steps * 4u;
      ps = static_cast<const uint8_t*>(P.ws) + (GROUPED ? t.slot * B.ws_stride * 4 : 0);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = 4 * wave + u, j = 8 * c + lr;
      const int col = GATED ? (j >> 5) * 16 + (j & 15) : j;
      boff[u] = (uint32_t)min(col, P.N - 1 - t.n0) * (uint32_t)P.ldw + piece(c) * 16;
    }
    pb = P.w + (GROUPED ? t.slot * B.w_stride : 0) + (int64_t)t.n0 * P.ldw;
  };
  uint32_t at_a = 0, at_b = kHalf, at_s = 0;  // where the next loads go
  auto load_w = [&](int u) __attribute__((always_inline)) {
    const int c = 4 * wave + u;
    dma16s(boff[u], pb + (GATED && ((c >> 1) & 1) ? up : 0), ring0 + at_b + c * 1024);
  };
  auto load_x = [&](int u) __attribute__((always_inline)) { dma16s(aoff[u], pa, ring0 + at_a + a_chunk(u) * 1024); };
  auto load_s = [&]() __attribute__((always_inline)) { dma4s(soff, ps, sc0 + at_s + sc * 256); };
  auto next_w = [&]() __attribute__((always_inline)) {
    at_b ^= kStage;
    pb += 128;
  };
  auto next_x = [&]() __attribute__((always_inline)) {
    at_a ^= kStage;
    at_s = at_s == 2 * kScales ? 0 : at_s + kScales;
    pa += 128;
    ps += sstep;
  };
  if (by_rows) {
    load_rows(0);
    if (n > 1) load_rows(1);
    wait_loads<0>();
    lds_sync();
  }
  to_tile(0);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int u = 0; u < 4; ++u) load_w(u);
    next_w();
#pragma unroll
    for (int u = 0; u < 4; ++u) load_x(u);
    load_s();
    next_x();
  }

  // ---- compute side
  lf32x4_t acc[TM][TN], late[TN];
  float late_f[TN];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      late[j] = lf32x4_t{0.f, 0.f, 0.f, 0.f};
      late_f[j] = 0.f;
#pragma unroll
      for (int i = 0; i < TM; ++i) acc[i][j] = lf32x4_t{0.f, 0.f, 0.f, 0.f};
    }
  };
  const uint32_t rd = r16 * 128 + ((g ^ (r16 >> 1)) << 4);
  const uint32_t rda = wm * TM * 2048 + rd, rdb = kHalf + wn * TN * 2048 + rd;
  const uint32_t rsa = (wm * TM * 16 + r16) * 4, rsb = (BM + wn * TN) * 4;
  Frag fw[TN], fx[TM];
  float bx[TM], bw[2], nw[2];
  auto read_w = [&](uint32_t st, uint32_t sp, int j) __attribute__((always_inline)) {
    fw[j].a = *reinterpret_cast<const uint4*>(ring + st + rdb + j * 2048);
    fw[j].b = *reinterpret_cast<const uint4*>(ring + st + (rdb ^ 64) + j * 2048);
    if (j < 2) nw[j] = *reinterpret_cast<const float*>(s_sc + sp + rsb + j * 4);
  };
  auto read_x = [&](uint32_t st, uint32_t sp, int i) __attribute__((always_inline)) {
    fx[i].a = *reinterpret_cast<const uint4*>(ring + st + rda + i * 2048);
    fx[i].b = *reinterpret_cast<const uint4*>(ring + st + (rda ^ 64) + i * 2048);
    bx[i] = *reinterpret_cast<const float*>(s_sc + sp + rsa + i * 64);
  };
  wait_loads<0>();  // steps 0 and 1
  lds_sync();
#pragma unroll
  for (int j = 0; j < TN; ++j) read_w(0, 0, j);
  read_x(0, 0, 0);
  read_x(0, 0, 1);
  bw[0] = nw[0];
  bw[1] = nw[1];
  uint32_t at = 0, sp = 0;  // stage and scale place of the step
  auto step = [&]() __attribute__((always_inline)) {
    const uint32_t nx = at ^ kStage, nsp = sp == 2 * kScales ? 0 : sp + kScales;
    auto part = [&](auto ic) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value;
      if constexpr (i == 0) {
        wait_loads<9>();  // the step's other half of x; every wave has its weights and first half
        lds_sync();
      }
      if constexpr (i == 2) {
        wait_loads<6>();  // the next step's weights, scales and first half of x; every wave has this step's x
        lds_sync();
      }
      if constexpr (i < 2) read_x(at, sp, i + 2);
      else read_x(nx, nsp, i - 2);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[(i + 3) & 3][j][v] = fmaf(late[j][v], late_f[j], acc[(i + 3) & 3][j][v]);
        __builtin_amdgcn_sched_barrier(0);
        late[j] = mma_fp8<0, 0>(fw[j], fx[i], lf32x4_t{0.f, 0.f, 0.f, 0.f}, 0x7F7F7F7F, 0x7F7F7F7F);
        late_f[j] = bx[i] * bw[GATED ? j & 1 : 0];
        __builtin_amdgcn_sched_barrier(0);
        // evenly, in the order that the waits count: 2 weights, 2 weights, 2 of x's first half, scales and 2 of the other
        if (j == 0 || j == 2) {
          if constexpr (i < 2) load_w(2 * i + j / 2);
          else if constexpr (i == 2) load_x(j / 2);
          else load_x(2 + j / 2);
        }
        if constexpr (i == 2) {
          if (j == 3) load_s();
        }
        if constexpr (i == 3) read_w(nx, nsp, j);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (i == 1) next_w();
    };
    part(std::integral_constant<int, 0>{});
    part(std::integral_constant<int, 1>{});
    part(std::integral_constant<int, 2>{});
    part(std::integral_constant<int, 3>{});
    next_x();
    bw[0] = nw[0];
    bw[1] = nw[1];
    at = nx;
    sp = nsp;
  };
  // the sums stay where they are: no matrix instruction moves past this
  auto pin = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      asm volatile("" : "+v"(late[j]));
#pragma unroll
      for (int i = 0; i < TM; ++i) asm volatile("" : "+v"(acc[i][j]));
    }
  };
  for (int k = 0; k < n; ++k) {
    clear();
#pragma unroll 1
    for (int s = 2; s < steps; ++s) step();
    // The load side, two steps ahead, goes to the next tile; behind the last it starts that again, since the
    // counted waits need the same loads every step.  Row numbers are asked for a tile ahead: the waits of
    // the two steps from here to their turn cover them.
    pin();
    to_tile(min(k + 1, n - 1));
    if (by_rows && k + 2 < n) load_rows(k + 2);
    step();
    step();
    pin();
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[TM - 1][j][v] = fmaf(late[j][v], late_f[j], acc[TM - 1][j][v]);
    const Tile t = tile_at(k);
    LinParams E = P;
    if constexpr (GROUPED) {
      E.res = nullptr;
      if (E.bias) E.bias += (int64_t)t.slot * P.R;
    }
    block_epilogue<GATED, WM, WN, TM, TN, 2>(E, G, acc, s_stage, t.t0, t.end, t.n0, lane, wave);
  }
  wait_loads<0>();  // no load into LDS outlives the workgroup
}

template <bool GATED, bool GROUPED>
void launch_one(const BlockParams& B, const LinTiles& G, hipStream_t s) {
  launch(k_block_stream<GATED, GROUPED>, dim3(2 * kCus), dim3(256), 0, s, B, G);
}

}  // namespace

void launch_block_stream(const BlockParams& B, hipStream_t s) {
  const LinParams& P = B.L;
  LinTiles G{};
  G.mt = (P.T + 127) / 128;
  G.nt = P.gated ? (P.N + 63) / 64 : (P.N + 127) / 128;
  G.vec_out = ((uintptr_t)P.out & 15) == 0 && (P.ldo * 2) % 16 == 0;
  G.vec_res = ((uintptr_t)P.res & 15) == 0 && P.ldr % 8 == 0;
  G.splits = 1;
  if (B.offsets) P.gated ? launch_one<true, true>(B, G, s) : launch_one<false, true>(B, G, s);
  else P.gated ? launch_one<true, false>(B, G, s) : launch_one<false, false>(B, G, s);
}

}  // namespace moe
