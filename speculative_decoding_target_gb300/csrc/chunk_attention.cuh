// Attention of a chunk of new tokens over the paged cache (chunk_plan.cu, and
// the causal instance of the kernel in prefix_attention.cu): launch parameters
// and the plan.
//
// The rows of (request b, KV head g) are its new tokens' query heads that read
// g, token by token: row R is token R / group of the chunk.  They are cut into row
// tiles of 2 cta_rows, half for each CTA of a pair: as many whole tokens as fit
// into 128 rows, so that one tensor copy brings a CTA's queries, or 128 rows where
// whole tokens would leave more than three of them empty.  Row tile m attends
// the first t 128-token tiles of the cache that its last row sees.  A piece is a
// row tile over a run of those.
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

// A row tile of a request and KV head.
struct __align__(16) ChunkPiece {
  int b, g, row0, tiles;         // tiles of tokens
  int rows, first, limit, last;  // the request's rows, block row of row 0, tokens
                                 // that row 0 sees, last cached token
};
// A pair's run of the rest: its first piece, the tile it starts at, its tiles, and
// the partial slot of that first piece if it does not start it.
struct __align__(16) ChunkRun {
  int piece, from, tiles, slot;
};

struct ChunkParams {
  AttnParams a;       // rows, grid, part_o and part_lse unused
  ChunkHead* head;
  ChunkPiece* pieces; // in order
  ChunkRun* runs;     // [pairs]
  int2* rest;         // [pairs]: a rest's piece's first partial slot, and partials
                      // (1: whole)
  float* pre_o;       // [2 pairs, kPrefixRows, 256]
  float* pre_lse;     // [2 pairs, kPrefixRows]
  int pairs;
  int cta_rows;       // rows of a CTA: q_tokens * group, or 128
  int q_tokens;       // tokens of a tensor copy of queries; 0: no such copies
};

// Tokens whose rows fill a CTA well enough (of 128 rows no more than 3 empty).
// Whole tokens against 128 rows that threads copy, 22 to 50 query heads, us:
//   rows a CTA          300 tokens   4,096 tokens   700 behind   2,048 behind
//                       into empty   into empty     12,000       32,768
//   126 (groups of 6)   19 / 20.5    145 / 153      149 / 150    1,010 / 996
//   125 (25)            22.5 / 25    312 / 347      277 / 273    2,074 / 2,008
//   121 (11)            21.5 / 23    164 / 156      146 / 144    912 / 833
//   120 (20)            22.5 / 24.5  288 / 281      242 / 216    1,752 / 1,631
// Short calls gain 1.5 us either way; long ones lose the empty rows' share.
inline int chunk_q_tokens(int group) {
  const int n = group <= 128 ? 128 / group : 0;
  return n * group >= 125 ? n : 0;
}

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
__device__ __forceinline__ int chunk_row_tiles(const ChunkRows& r, int cta_rows) {
  return (r.rows + 2 * cta_rows - 1) / (2 * cta_rows);
}
// Tokens that row R sees.
__device__ __forceinline__ int chunk_limit(const ChunkRows& r, int R, int group) {
  return r.len - r.live + R / group + 1;
}
// Tiles of tokens of row tile m.
__device__ __forceinline__ int chunk_tiles(const ChunkRows& r, int m, int group,
                                           int cta_rows) {
  const int R = min((m + 1) * 2 * cta_rows, r.rows) - 1;
  return (chunk_limit(r, R, group) + kPrefixTile - 1) / kPrefixTile;
}

// Row tiles of a request with `rows` rows, at most.
inline long long chunk_tiles_of(long long rows, int cta_rows) {
  return (rows + 2 * cta_rows - 1) / (2 * cta_rows);
}

cudaError_t launch_chunk_plan(const ChunkParams& p, cudaStream_t s);
cudaError_t launch_chunk_attention(const ChunkParams& p, const CUtensorMap& tm_k,
                                   const CUtensorMap& tm_v,
                                   const CUtensorMap& tm_q, cudaStream_t s);
cudaError_t launch_chunk_merge(const ChunkParams& p, int sms, cudaStream_t s);
int chunk_attention_pairs(bool fp8);

}  // namespace specv
