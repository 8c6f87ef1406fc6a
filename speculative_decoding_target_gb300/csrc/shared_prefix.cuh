// Verify attention of requests that share cached prefixes (shared_prefix.cu,
// prefix_attention.cu): launch parameters and the plan of the shared part.
//
// A group is a run of consecutive requests whose page tables start with the
// same pages.  Its shared part, the first `eff` tokens (a multiple of
// kPrefixTile that every row of every live request sees whole), is attended
// once for all rows of the group; each request's remaining tokens are attended
// by the ordinary split kernels from kv_begin on.  Both write fp32 partials
// (normalised rows and base-2 log-sum-exps), which one kernel merges.
//
// Plan of the shared part.  The rows of (group n, KV head g), all requests'
// block rows that read head g, are cut into tiles of kPrefixRows; a
// (n, g, tile) is a segment of eff / kPrefixTile units, charged kPrefixCost
// units in front as in common.cuh.  Segments lie end to end, CTA pair c takes
// the c-th even share of the line, and the partial of segment k from pair c
// goes to slot c + k.
#pragma once

#include "common.cuh"

namespace specv {

constexpr int kPrefixTile = 128;   // tokens per tile
constexpr int kPrefixRows = 256;   // rows per CTA pair
constexpr int kPrefixCost = 4;     // plan units a segment's start costs
constexpr int kPrefixMinUnits = 2; // least share of a CTA pair
constexpr int kMaxGroups = kMaxBatch;

// One entry per group, plus the totals at [groups].
struct GroupPlan {
  long long unit0;   // virtual units before this group
  int seg0;          // segments before this group
  int tiles;         // row tiles per KV head (0: nothing is shared)
  int eff;           // shared tokens attended once
  int start;         // first request
  int count;         // requests
  int lead;          // the live request whose page table is read
};

struct SharedParams {
  AttnParams a;               // the tails' call; kv_begin and group_of set
  const int32_t* starts;      // [groups + 1]
  const int32_t* shared_lens; // [groups]
  int groups;
  GroupPlan* plan;            // [groups + 1]
  int32_t* kv_begin;          // [B]
  int32_t* group_of;          // [B]: group with a shared part, or -1
  float* pre_o;               // [slots, kPrefixRows, 256]
  float* pre_lse;             // [slots, kPrefixRows]
  int pairs;                  // CTA pairs of the prefix kernel
};

__device__ __forceinline__ int prefix_units(const GroupPlan& g) {
  return g.eff / kPrefixTile + kPrefixCost;
}

// The totals as a plan over the pairs.
__device__ __forceinline__ Plan prefix_plan(const SharedParams& p) {
  Plan pl;
  pl.U = p.plan[p.groups].unit0;
  const long long want = (pl.U + kPrefixMinUnits - 1) / kPrefixMinUnits;
  pl.P = want < p.pairs ? (int)want : p.pairs;
  return pl;
}

cudaError_t launch_shared_plan(const SharedParams& p, cudaStream_t s);
cudaError_t launch_prefix_attention(const SharedParams& p,
                                    const CUtensorMap& tm_k,
                                    const CUtensorMap& tm_v, cudaStream_t s);
cudaError_t launch_shared_merge(const SharedParams& p, cudaStream_t s);
int prefix_attention_pairs(bool fp8);

}  // namespace specv
