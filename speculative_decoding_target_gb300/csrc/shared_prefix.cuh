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
// block rows that read head g, are cut into tiles of kPrefixRows, and the
// group's shared tokens into `splits` even runs of 128-token tiles.  A piece is
// one row tile over one run; pieces are numbered by (group, head, run, row
// tile), pair c of P takes pieces c, c + P, ..., and piece i writes its partial
// to slot i.  Pieces that read the same tokens are neighbours, so they run at
// the same time and share their tiles in L2.  The run length is the one of
// kPlans candidates around the even share that ends first, counting each
// piece's fixed cost as kPrefixCost tiles (charges of 1, 4 and 12 measure alike
// within 0.5 us on calls of 30 to 180 us).
#pragma once

#include "common.cuh"

namespace specv {

constexpr int kPrefixTile = 128;   // tokens per tile
constexpr int kPrefixRows = 256;   // rows per CTA pair
constexpr int kPrefixCost = 4;     // tiles' time that a piece's start and end cost
constexpr int kPlans = 32;         // run lengths tried, a warp each
constexpr int kMaxGroups = kMaxBatch;

// One entry per group; [groups].piece0 is the number of pieces.
struct GroupPlan {
  int piece0;   // first piece
  int tiles;    // row tiles per KV head (0: nothing is shared)
  int splits;   // runs of tokens
  int eff;      // shared tokens attended once
  int start;    // first request
  int count;    // requests
  int lead;     // the live request whose page table is read
  int pad;
};

struct SharedParams {
  AttnParams a;               // the tails' call; kv_begin and group_of set
  const int32_t* starts;      // [groups + 1]
  const int32_t* shared_lens; // [groups]
  int groups;
  GroupPlan* plan;            // [groups + 1]
  int32_t* kv_begin;          // [B]
  int32_t* group_of;          // [B]: group with a shared part, or -1
  float* pre_o;               // [pieces, kPrefixRows, 256]
  float* pre_lse;             // [pieces, kPrefixRows]
  int pairs;                  // CTA pairs of the prefix kernel
};

// First 128-token tile of run c of a group's shared part (c <= splits).
__device__ __forceinline__ int run_start(const GroupPlan& g, int c) {
  return (int)((long long)c * (g.eff / kPrefixTile) / g.splits);
}

// Most pieces a plan makes, for `tiles` row tiles in all: the shortest run
// tried is above half the even share, and each segment rounds up by one.
inline long long max_pieces(int pairs, long long segments) {
  return 2LL * pairs + segments;
}

cudaError_t launch_shared_plan(const SharedParams& p, cudaStream_t s);
cudaError_t launch_prefix_attention(const SharedParams& p,
                                    const CUtensorMap& tm_k,
                                    const CUtensorMap& tm_v, cudaStream_t s);
cudaError_t launch_shared_merge(const SharedParams& p, cudaStream_t s);
int prefix_attention_pairs(bool fp8);

}  // namespace specv
