// Internal header of libmoe (not installed): the routing of a cache's layers
// by a router of their own.  The cache calls it through a pointer, so that its
// host code links without the kernels.
#pragma once
#include <algorithm>

#include "host_common.h"

namespace moe {

constexpr int kScoredMaxK = 16;              // experts a token
constexpr int kScoredMaxRows = 1 << 17;      // tokens x experts a token of a permutation

// The most experts a token can be given by *r (checked) over E: those of the groups it may take.
inline int router_most(const moe_router& r, int E) { return std::min(r.topk_group * (E / r.n_group), kScoredMaxK); }

// moe_route_scored_permute; with host_counts set, the counts copied there
// (host-mapped) and `seq` published in *flag behind every output.
typedef moe_status (*RouteHook)(const moe_router* r, const float* logits, int T, int E, int k, int32_t* topk_ids,
                                float* topk_w, int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* inv,
                                int32_t* host_counts, uint32_t* flag, uint32_t seq, hipStream_t s);

// Layer `layer` (-1: every layer) of the cache routes by *r through `hook`;
// r null: by moe_route again.
void cache_shape(const moe_cache* c, int* num_layers, int* num_experts);
void cache_set_router(moe_cache* c, int layer, const moe_router* r, RouteHook hook);

}  // namespace moe
