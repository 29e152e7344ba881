// The FP8 product with a scale per block of 128 for long batches: tiles of 256
// rows x 256 weight rows, eight waves of 128 x 64.
//
// Bound: the matrix cores (a step is 32 instructions of 32 cycles a wave, two
// waves a SIMD) and the way from the L2 into LDS.  The largest tile moves the
// fewest bytes: 64 KiB a step of 2048 matrix cycles, 32 a cycle, of about 50
// that a CU's loads to LDS reach; a 128 x 128 tile needs 64.
//
// One step of 128 columns in eight parts, part i the wave's i-th 16 rows of x
// against its four fragments of weights:
//   - each instruction starts from zero; beside it the four FMA that add what
//     the instruction four before left, times its scales' product.
//   - fragments of x are read two parts ahead, four in registers; those of the
//     next step's weights as the last part uses up this one's.
//   - after part 0 every wave has the step's weights in registers: their
//     place takes the weights of step s + 2 (parts 2 to 5).  Before part 6
//     every wave has read the step's rows of x: their place takes those of step
//     s + 2 (parts 6 and 7, and 0 and 1 of the next step), and the same barrier
//     says that step s + 1 has landed.
// So a load has from five parts to a step and a half to land in two stages,
// the loads go out evenly, and each barrier stands where no wave waits for its
// own reads.
//
// 4096 x (2 x 2048) x 7168, SwiGLU: 98.5 us, 2.44 PFLOP/s (a library product of
// 8192^3 reaches 3.09); 128 x 128 tiles, a workgroup each, 184 with the sums
// scaled at once and 126 scaled late, walked 121.  Matrix cores 0.54 busy, texture
// unit 0.41, L2 hits 0.81, 179 MB fetched of 60 read once.  Operands of zeros take
// 77 us where real ones, in the same run, take 104: what is left is their power.
#include <algorithm>
#include <type_traits>

#include "linear_block.h"
#include "linear_block_epilogue.h"
#include "linear_block_plan.h"

namespace moe {

namespace {

template <bool GATED>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_block_big(BlockParams B, LinTiles G) {
  constexpr int WM = 2, WN = 4, TM = 8, TN = 4, BM = 256, BN = 256;
  constexpr int BO = GATED ? BN / 2 : BN;
  constexpr uint32_t kHalf = 256 * 128, kStage = 2 * kHalf;  // x rows, weight rows of a step
  constexpr uint32_t kScales = 5 * 256;                      // a step's scales: 256 rows, 16 groups of weight rows
  __shared__ __align__(1024) uint8_t ring[2 * kStage];
  __shared__ __align__(256) uint8_t s_sc[3 * kScales];
  const LinParams P = B.L;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN, r16 = lane & 15, g = lane >> 4, lr = lane >> 3;

  // the tile: as in tile_product
  const int mt = G.mt;
  const int total = mt * G.nt, per = (total + 7) / 8;
  if ((int)(blockIdx.x / 8) >= per) return;
  const int L = (int)(blockIdx.x % 8) * per + (int)(blockIdx.x / 8);
  if (L >= total) return;
  const int band = L / (4 * G.nt), in_band = L - band * 4 * G.nt, bh = min(4, mt - 4 * band);
  const int n0 = (in_band / bh) * BO;
  const int t0 = (4 * band + in_band % bh) * BM, t_end = P.T;
  const int steps = B.steps;
  const uint32_t ring0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)ring;
  const uint32_t sc0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)s_sc;

  // ---- load side: chunk 4 wave + u of 8 rows, piece (l % 8) ^ (row bits 3:1)
  auto piece = [&](int c) { return (lane & 7) ^ ((4 * (c & 1) + (lr >> 1)) & 7); };
  uint32_t aoff[4], boff[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int c = 4 * wave + u, j = 8 * c + lr;
    const int i = min(j, t_end - 1 - t0);
    aoff[u] = (uint32_t)i * (uint32_t)P.ldx + piece(c) * 16;
    const int col = GATED ? (j >> 5) * 16 + (j & 15) : j;
    boff[u] = (uint32_t)min(col, P.N - 1 - n0) * (uint32_t)P.ldw + piece(c) * 16;
  }
  const int64_t up = GATED ? (int64_t)P.N * P.ldw : 0;
  const int sc = wave % 5;
  uint32_t soff;
  const uint8_t* ps;
  int64_t sstep;
  if (sc < 4) {
    const int t = min(t0 + 64 * sc + lane, t_end - 1);
    soff = (uint32_t)t * 4u;
    ps = static_cast<const uint8_t*>(P.xs);
    sstep = (int64_t)B.X * 4;
  } else {
    const int q = min(lane, BN / 16 - 1);
    const int c = min(n0 + (GATED ? (q >> 1) * 16 : q * 16), P.N - 1) >> 7;
    soff = (uint32_t)((GATED && (q & 1) ? B.nb : 0) + c) * (uint32_t)steps * 4u;
    ps = static_cast<const uint8_t*>(P.ws);
    sstep = 4;
  }
  const uint8_t* pa = P.x + (int64_t)t0 * P.ldx;
  const uint8_t* pb = P.w + (int64_t)n0 * P.ldw;
  // steps fa (x and scales) and fb (weights) are loaded next, into stage f % 2
  // and scale place f % 3; past the end the last step again
  int fa = 0, fb = 0;
  uint32_t at_a = 0, at_b = kHalf, at_s = 0;
  auto load_w = [&](int u) __attribute__((always_inline)) {
    const int c = 4 * wave + u;
    dma16s(boff[u], pb + (GATED && ((c >> 1) & 1) ? up : 0), ring0 + at_b + c * 1024);
  };
  auto load_x = [&](int u) __attribute__((always_inline)) {
    dma16s(aoff[u], pa, ring0 + at_a + (4 * wave + u) * 1024);
  };
  auto load_s = [&]() __attribute__((always_inline)) { dma4s(soff, ps, sc0 + at_s + sc * 256); };
  auto next_w = [&]() __attribute__((always_inline)) {
    if (++fb < steps) pb += 128;
    at_b ^= kStage;
  };
  auto next_x = [&]() __attribute__((always_inline)) {
    if (++fa < steps) {
      pa += 128;
      ps += sstep;
    }
    at_a ^= kStage;
    at_s = at_s == 2 * kScales ? 0 : at_s + kScales;
  };
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int u = 0; u < 4; ++u) load_w(u);
    next_w();
    load_x(0);
    load_x(1);
    if (s == 0) {  // the rest of step 1's: in step 0
      load_x(2);
      load_x(3);
      load_s();
      next_x();
    }
  }
  // ---- compute side
  lf32x4_t acc[TM][TN], late[TN];
  float late_f[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    late[j] = lf32x4_t{0.f, 0.f, 0.f, 0.f};
    late_f[j] = 0.f;
#pragma unroll
    for (int i = 0; i < TM; ++i) acc[i][j] = lf32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  // fragment row r16 of a 16-row group: pieces g and 4 + g (64 bytes apart in the permuted row too)
  const uint32_t rd = r16 * 128 + ((g ^ (r16 >> 1)) << 4);
  const uint32_t rda = wm * TM * 2048 + rd, rdb = kHalf + wn * TN * 2048 + rd;
  const uint32_t rsa = (wm * TM * 16 + r16) * 4, rsb = (BM + wn * TN) * 4;
  Frag fw[TN], fx[4];
  float bx[4], bw[2], nw[2];
  auto read_w = [&](uint32_t st, uint32_t sp, int j) __attribute__((always_inline)) {
    fw[j].a = *reinterpret_cast<const uint4*>(ring + st + rdb + j * 2048);
    fw[j].b = *reinterpret_cast<const uint4*>(ring + st + (rdb ^ 64) + j * 2048);
    if (j < 2) nw[j] = *reinterpret_cast<const float*>(s_sc + sp + rsb + j * 4);
  };
  auto read_x = [&](uint32_t st, uint32_t sp, int i) __attribute__((always_inline)) {
    fx[i & 3].a = *reinterpret_cast<const uint4*>(ring + st + rda + i * 2048);
    fx[i & 3].b = *reinterpret_cast<const uint4*>(ring + st + (rda ^ 64) + i * 2048);
    bx[i & 3] = *reinterpret_cast<const float*>(s_sc + sp + rsa + i * 64);
  };
  wait_loads<6>();  // step 0
  lds_sync();
#pragma unroll
  for (int j = 0; j < TN; ++j) read_w(0, 0, j);
  read_x(0, 0, 0);
  read_x(0, 0, 1);
  bw[0] = nw[0];
  bw[1] = nw[1];
  uint32_t at = 0, sp = 0;  // stage and scale place of the step
#pragma unroll 1
  for (int s = 0; s < steps; ++s) {
    const uint32_t nx = at ^ kStage, nsp = sp == 2 * kScales ? 0 : sp + kScales;
    auto part = [&](auto ic) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value;
      if constexpr (i == 6) {
        wait_loads<4>();  // step s + 1, all but the weights of s + 2
        lds_sync();
      }
      if constexpr (i < 6) read_x(at, sp, i + 2);
      else read_x(nx, nsp, i - 6);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[(i + 7) & 7][j][v] = fmaf(late[j][v], late_f[j], acc[(i + 7) & 7][j][v]);
        __builtin_amdgcn_sched_barrier(0);
        late[j] = mma_fp8<0, 0>(fw[j], fx[i & 3], lf32x4_t{0.f, 0.f, 0.f, 0.f}, 0x7F7F7F7F, 0x7F7F7F7F);
        late_f[j] = bx[i & 3] * bw[GATED ? j & 1 : 0];
        __builtin_amdgcn_sched_barrier(0);
        // one load a part: together they would hold back every wave's instructions behind the texture unit
        if (j == 1) {
          if constexpr (i < 2) load_x(i + 2);
          else if constexpr (i < 6) load_w(i - 2);
          else load_x(i - 6);
        }
        if constexpr (i == 1) {
          if (j == 3) load_s();
        }
        if constexpr (i == 7) read_w(nx, nsp, j);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (i == 0) lds_sync();  // every wave has the step's weights
      if constexpr (i == 1) next_x();
      if constexpr (i == 5) next_w();
    };
    part(std::integral_constant<int, 0>{});
    part(std::integral_constant<int, 1>{});
    part(std::integral_constant<int, 2>{});
    part(std::integral_constant<int, 3>{});
    part(std::integral_constant<int, 4>{});
    part(std::integral_constant<int, 5>{});
    part(std::integral_constant<int, 6>{});
    part(std::integral_constant<int, 7>{});
    bw[0] = nw[0];
    bw[1] = nw[1];
    at = nx;
    sp = nsp;
  }
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[TM - 1][j][v] = fmaf(late[j][v], late_f[j], acc[TM - 1][j][v]);
  wait_loads<0>();
  lds_sync();  // nothing reads or fills the ring any more: its memory takes the staging rows
  block_epilogue<GATED, WM, WN, TM, TN, GATED ? TN / 2 : TN>(P, G, acc, reinterpret_cast<float*>(ring), t0, t_end, n0, lane,
                                                             wave);
}

template <bool GATED>
void launch_one(const BlockParams& B, const LinTiles& G, hipStream_t s) {
  const int64_t grid = ((int64_t)G.mt * G.nt + 7) / 8 * 8;
  launch(k_block_big<GATED>, dim3((unsigned)grid), dim3(512), 0, s, B, G);
}

}  // namespace

void launch_block_big(const BlockParams& B, hipStream_t s) {
  const LinParams& P = B.L;
  LinTiles G{};
  G.mt = (P.T + 255) / 256;
  G.nt = P.gated ? (P.N + 127) / 128 : (P.N + 255) / 256;
  G.vec_out = ((uintptr_t)P.out & 15) == 0 && (P.ldo * 2) % 16 == 0;
  G.vec_res = ((uintptr_t)P.res & 15) == 0 && P.ldr % 8 == 0;
  G.splits = 1;
  P.gated ? launch_one<true>(B, G, s) : launch_one<false>(B, G, s);
}

}  // namespace moe
