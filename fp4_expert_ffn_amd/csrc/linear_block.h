// Shared by the kernels of the FP8 product with a scale per block of 128,
// dense and grouped over the experts' rows (linear_block*.hip).
#pragma once
#include "linear.h"

namespace moe {

// What LinParams does not say: the scales' layouts and the groups.
// LinParams: T rows of out, kb = K, xs fp32 [steps][X], ws fp32 [row
// blocks][steps] of slot 0 (a row block: 128 rows; gated: the gate's nb, then
// the up's).
struct BlockParams {
  LinParams L;
  int X;      // rows of x
  int steps;  // K / 128
  int nb;     // ceil(N / 128)
  // grouped
  int E, div;
  const int32_t* offsets;  // null: dense
  const int32_t* rows;
  const int32_t* slot;
  int64_t w_stride, ws_stride;  // bytes, floats
};

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
  return v;
}

// Row block b of the experts' rows in blocks of BM: expert, its first row and
// its end; e < 0 past the last block.  Wave-uniform; every lane of the wave
// takes part.
struct RowBlock {
  int e, t0, end;
};
template <int BM>
__device__ __forceinline__ RowBlock find_row_block(const BlockParams& B, int b) {
  const int lane = threadIdx.x & 63;
  RowBlock r{-1, 0, 0};
  int before = 0;  // row blocks of the experts looked at so far
  for (int e0 = 0; e0 < B.E; e0 += 64) {
    const int e = e0 + lane;
    const int lo = B.offsets[min(e, B.E)], hi = B.offsets[min(e + 1, B.E)];  // past the last expert: no rows
    const int n = (max(hi - lo, 0) + BM - 1) / BM;
    const int sum = before + wave_scan(n);
    const uint64_t past = __ballot(sum > b);
    if (past) {
      const int l = __builtin_ctzll(past);
      r.e = e0 + l;
      const int first = __builtin_amdgcn_readlane(sum - n, l);
      r.t0 = __builtin_amdgcn_readlane(lo, l) + (b - first) * BM;
      r.end = min(__builtin_amdgcn_readlane(hi, l), B.L.T);
      return r;
    }
    before = __builtin_amdgcn_readlane(sum, 63);
  }
  return r;
}

// Row blocks of BM rows of all experts.
template <int BM>
__device__ __forceinline__ int count_row_blocks(const BlockParams& B) {
  int n = 0;
  for (int e = threadIdx.x & 63; e < B.E; e += 64) n += (max(B.offsets[e + 1] - B.offsets[e], 0) + BM - 1) / BM;
  return __builtin_amdgcn_readlane(wave_scan(n), 63);
}

// Row of x that row p of the product reads.
__device__ __forceinline__ int x_row(const BlockParams& B, int p) {
  const uint32_t r = B.rows ? (uint32_t)B.rows[p] / (uint32_t)B.div : (uint32_t)p;
  return (int)min(r, (uint32_t)(B.X - 1));
}

// The expert's weights, scales and bias in place of slot 0's.
__device__ __forceinline__ void to_slot(const BlockParams& B, int e, LinParams& P) {
  const int64_t s = B.slot ? B.slot[e] : e;
  P.w += s * B.w_stride;
  P.ws = static_cast<const float*>(P.ws) + s * B.ws_stride;
  if (P.bias) P.bias += s * P.R;
}

struct TilePlan;
// The tile kernel (linear_block_tile.hip).  False: the call's strides do not fit it.
bool block_tile_fits(const BlockParams& B);
void launch_block_tile(const BlockParams& B, const TilePlan& pl, void* workspace, hipStream_t s);
// Tiles of 256 x 256 (linear_block_big.hip): dense, bf16 outputs, K not split.
void launch_block_big(const BlockParams& B, hipStream_t s);
// Tiles of 128 x 128 walked by two workgroups a CU (linear_block_stream.hip):
// bf16 outputs, K not split and at least two blocks, at most kStreamTiles tiles a workgroup.
void launch_block_stream(const BlockParams& B, hipStream_t s);

size_t linear_block_workspace(int T, int N, int K, bool gated, bool out_f32);
void launch_linear_block(const BlockParams& B, void* workspace, hipStream_t s);

}  // namespace moe
