// Attention of a chunk of new tokens over the paged cache (chunk_plan.cu, and
// the causal instance of the kernel in prefix_attention.cu): launch parameters
// and the plan.
//
// The rows of (request b, KV head g) are its new tokens' query heads that read
// g, token by token: row R is token R / group of the chunk.  They are cut into
// tiles of kPrefixRows; tile m attends the first t 128-token tiles of the cache
// that its last row sees.  A piece is a row tile over a run of those.
//
// Pieces of a whole row tile are sorted by t (in kChunkBuckets steps, longest
// first; in a step by head, so that pieces that read the same tokens run at the
// same time and share them in L2) and dealt to the CTA pairs in rounds, every
// other round backwards.  What does not fill a round, the rest, is laid end to
// end and cut into one run of tiles per pair, so long that all pairs end
// together: only there are row tiles cut, into partials that a merge joins.  A
// rest that costs no more when dealt whole is dealt whole.
#pragma once

#include "shared_prefix.cuh"

namespace specv {

constexpr int kChunkBuckets = 64;

struct ChunkHead {
  int rounds;  // whole rounds of the pairs
  int rest;    // pieces after them, < pairs
  int split;   // whether the rest is cut into runs
  int pad;
};

struct ChunkParams {
  AttnParams a;       // rows, grid, part_o and part_lse unused
  ChunkHead* head;
  int4* pieces;       // (request, row tile, KV head, tiles of tokens), in order
  int* rest_units;    // [pairs + 1]: tiles before each piece of the rest
  int* ranges;        // [pairs + 1]: each pair's run of the rest's tiles
  float* pre_o;       // [2 pairs, kPrefixRows, 256]
  float* pre_lse;     // [2 pairs, kPrefixRows]
  int pairs;
};

// A request's rows: of its w new tokens the last `live` are in the cache (all,
// unless it is longer than its cache); they are block rows first .. w - 1.
struct ChunkRows {
  int len, live, first, rows;
};
__device__ __forceinline__ ChunkRows chunk_rows(const AttnParams& p, int b) {
  ChunkRows r;
  const int w = block_rows(p, b);
  r.len = clamp_len(p.seq_lens[b], p.max_tokens);
  r.live = min(w, r.len);
  r.first = w - r.live;
  r.rows = r.live * p.group;
  return r;
}
__device__ __forceinline__ int chunk_row_tiles(const ChunkRows& r) {
  return (r.rows + kPrefixRows - 1) / kPrefixRows;
}
// Tokens that row R sees.
__device__ __forceinline__ int chunk_limit(const ChunkRows& r, int R, int group) {
  return r.len - r.live + R / group + 1;
}
// Tiles of tokens of row tile m.
__device__ __forceinline__ int chunk_tiles(const ChunkRows& r, int m, int group) {
  const int R = min(m * kPrefixRows + kPrefixRows, r.rows) - 1;
  return (chunk_limit(r, R, group) + kPrefixTile - 1) / kPrefixTile;
}

cudaError_t launch_chunk_plan(const ChunkParams& p, cudaStream_t s);
cudaError_t launch_chunk_attention(const ChunkParams& p, const CUtensorMap& tm_k,
                                   const CUtensorMap& tm_v, cudaStream_t s);
cudaError_t launch_chunk_merge(const ChunkParams& p, int sms, cudaStream_t s);
int chunk_attention_pairs(bool fp8);

}  // namespace specv
