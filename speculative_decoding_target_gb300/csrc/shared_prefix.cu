// Verify attention of requests that share cached prefixes: the plan of the
// shared parts, and the merge of their partials with those of the requests'
// own tails.  (The shared parts are attended in prefix_attention.cu, the tails
// by the ordinary split kernels from kv_begin on.)
#include <algorithm>
#include <climits>

#include "shared_prefix.cuh"
#include "spec_verify.h"

namespace specv {
namespace {

constexpr int kPlanThreads = 1024;   // at most: kMaxBatch, kMaxGroups
static_assert(kPlanThreads >= kMaxBatch && kPlanThreads >= kMaxGroups, "");

// One CTA: thread b looks at request b, thread n at group n.  A group's shared
// part is cut to what every row of every live request sees and to whole tiles
// of tokens; with fewer than two live requests, or less than a tile, nothing
// is shared and the tails hold everything.  Group borders that run backwards
// or out of the batch share nothing at all.
__global__ void __launch_bounds__(kPlanThreads)
    shared_plan_kernel(const SharedParams p) {
  __shared__ int s_start[kMaxGroups + 1];
  __shared__ int s_seen[kMaxGroups];   // tokens that every live row sees
  __shared__ int s_lead[kMaxGroups];
  __shared__ int s_live[kMaxGroups];
  __shared__ int s_rows[kMaxGroups];   // row tiles over all KV heads
  __shared__ int s_kv[kMaxGroups];     // 128-token tiles
  __shared__ int s_pieces[2][kMaxGroups];
  __shared__ long long s_plan[kPlans]; // (time, pieces) of a candidate
  __shared__ int s_run[kPlans];
  __shared__ unsigned long long s_work;
  __shared__ int s_bad;
  const int tid = threadIdx.x, G = p.groups;
  const AttnParams& a = p.a;
  // the prefix kernel may set itself up now; it waits for this grid
  tc_grid_launch_dependents();
  if (tid == 0) {
    s_bad = 0;
    s_work = 0;
  }
  for (int n = tid; n <= G; n += blockDim.x) s_start[n] = p.starts[n];
  if (tid < G) {
    s_seen[tid] = INT_MAX;
    s_lead[tid] = INT_MAX;
    s_live[tid] = 0;
  }
  __syncthreads();
  if (tid < G && (s_start[tid] < 0 || s_start[tid] > s_start[tid + 1] ||
                  s_start[tid + 1] > a.batch))
    s_bad = 1;
  __syncthreads();
  const bool bad = s_bad;
  if (bad && tid == 0 && a.status) atomicOr(a.status, SPEC_STATUS_BAD_GROUPS);

  int mine = -1, width = 0, len = 0;
  if (tid < a.batch) {
    width = block_rows(a, tid);
    len = clamp_len(a.seq_lens[tid], a.max_tokens);
    if (!bad && G > 0 && tid >= s_start[0] && tid < s_start[G]) {
      int lo = 0, hi = G - 1;  // the last group that starts at or before b
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_start[mid] <= tid) lo = mid; else hi = mid - 1;
      }
      mine = lo;
    }
    if (mine >= 0 && width > 0) {
      // the block's first row sees len - width + 1 tokens, itself included
      atomicMin(&s_seen[mine], len - width);
      atomicMin(&s_lead[mine], tid);
      atomicAdd(&s_live[mine], 1);
    }
  }
  __syncthreads();
  GroupPlan gp{};
  if (tid < G) {
    if (!bad) {
      gp.start = s_start[tid];
      gp.count = s_start[tid + 1] - gp.start;
      if (s_live[tid] >= 2) {
        const int eff = min(p.shared_lens[tid], s_seen[tid]);
        if (eff >= kPrefixTile) {
          gp.eff = eff / kPrefixTile * kPrefixTile;
          gp.lead = s_lead[tid];
          gp.tiles = (gp.count * a.rows + kPrefixRows - 1) / kPrefixRows;
        }
      }
    }
    s_seen[tid] = gp.eff;  // each thread reads and writes its own entry
    s_rows[tid] = a.hkv * gp.tiles;
    s_kv[tid] = gp.eff / kPrefixTile;
    if (gp.eff)
      atomicAdd(&s_work, (unsigned long long)s_rows[tid] * s_kv[tid]);
  }
  __syncthreads();
  // candidate run lengths, 1.6 down to 0.53 of the even share, a warp each
  const int warp = tid >> 5, lane = tid & 31;
  for (int cand = warp; cand < kPlans; cand += blockDim.x >> 5) {
    const float share = (float)s_work / (float)p.pairs;
    // (no run is longer than the 2^23 tiles of the longest cache)
    const float tiles = ceilf(1.6f * share * __powf(0.965f, cand));
    const int run = (int)fminf(fmaxf(tiles, 1.f), 8388608.f);
    int pieces = 0, longest = 0;
    for (int n = lane; n < G; n += 32) {
      if (!s_kv[n]) continue;
      const int splits = (s_kv[n] + run - 1) / run;
      pieces += s_rows[n] * splits;
      longest = max(longest, (s_kv[n] + splits - 1) / splits);
    }
    pieces = __reduce_add_sync(0xffffffffu, pieces);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) {
      const long long waves = (pieces + p.pairs - 1) / p.pairs;
      s_plan[cand] = waves * (longest + kPrefixCost) << 24 |
                     min(pieces, (1 << 24) - 1);
      s_run[cand] = run;
    }
  }
  __syncthreads();
  int pick = 0;
  for (int j = 1; j < kPlans; ++j)
    if (s_plan[j] < s_plan[pick]) pick = j;
  const int run = s_run[pick];
  // pieces per group, and their prefix sums
  int mine_pieces = 0;
  if (tid < G && gp.eff) {
    gp.splits = (s_kv[tid] + run - 1) / run;
    mine_pieces = s_rows[tid] * gp.splits;
  }
  if (tid < G) s_pieces[0][tid] = mine_pieces;
  __syncthreads();
  int from = 0;
  for (int o = 1; o < G; o <<= 1, from ^= 1) {
    if (tid < G)
      s_pieces[from ^ 1][tid] =
          s_pieces[from][tid] + (tid >= o ? s_pieces[from][tid - o] : 0);
    __syncthreads();
  }
  if (tid < G) {
    gp.piece0 = s_pieces[from][tid] - mine_pieces;
    p.plan[tid] = gp;
  }
  if (tid == 0) {
    GroupPlan end{};
    end.piece0 = s_pieces[from][G - 1];
    p.plan[G] = end;
  }
  if (tid < a.batch) {
    const bool shares = !bad && mine >= 0 && width > 0 && s_seen[mine] > 0;
    p.group_of[tid] = shares ? mine : -1;
    // an idle request attends nothing
    p.kv_begin[tid] = width == 0 ? (len + 127) / 128 * 128
                                 : (shares ? s_seen[mine] : 0);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// out = sum_s 2^(lse_s - lse) o_s over a row's partials, those of its tail
// and those of its group's shared part.  One warp per output row, lane l
// channels 8l .. 8l+7, kBatch partials in flight with a running maximum: 20 for
// few rows, which are cut into many runs (one round of loads instead of three
// or four), 6 for many, where registers cost residency (4 single-token requests
// over 4K tokens: 30.5 us a call with 20, 31.6 with 6; 32 blocks of 8 over 32K:
// 189 us with 20, 179.4 with 6).  A merge of 6,144 rows of 5 to 7 partials
// takes 14 us, mostly from L2.
constexpr int kMergeWarps = 8;

template <int kBatch>
__global__ void __launch_bounds__(kMergeWarps * 32)
    shared_merge_kernel(const SharedParams p) {
  __shared__ int s_pre[kMaxBatch + 1];
  const AttnParams& a = p.a;
  // a following attention call's split kernel may be scheduled now
  tc_grid_launch_dependents();
  // The prefix kernel releases its dependents only after the plan kernel is
  // complete, so the plan may be read already.
  plan_prefix(a, s_pre);
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  const long long per = (long long)a.q_len * a.hq;
  if (w >= a.batch * per) return;  // uniform per warp
  const int b = (int)(w / per);
  const int rem = (int)(w - b * per);
  const int i = rem / a.hq, h = rem - i * a.hq, g = h / a.group;
  const int r = i * a.group + (h - g * a.group);
  const bool live = i < block_rows(a, b);
  // the tail's partials
  const Plan pl = make_plan(a, (long long)a.hkv * s_pre[a.batch]);
  const int ntv = s_pre[b + 1] - s_pre[b], nt = ntv - a.piece_cost;
  const long long s0 =
      (long long)a.hkv * s_pre[b] + (long long)g * ntv + a.piece_cost;
  const int n_tail = live && nt > 0 ? seg_splits(pl, s0, nt) : 0;
  long long tail_row = 0, pre_row = 0, pre_step = 0;
  if (n_tail)
    tail_row = (long long)partial_slot(chunk_of(pl, s0), b * a.hkv + g) *
                   a.rows + r;
  // the shared part's
  int n_pre = 0;
  const int n = live ? p.group_of[b] : -1;
  if (n >= 0) {
    const GroupPlan gp = p.plan[n];
    const int R = (b - gp.start) * a.rows + r;
    n_pre = gp.splits;
    pre_step = (long long)gp.tiles * kPrefixRows;
    pre_row = ((long long)gp.piece0 + (long long)g * gp.splits * gp.tiles +
               R / kPrefixRows) * kPrefixRows + R % kPrefixRows;
  }
  // the partials are read only once the kernels before are done
  tc_grid_dependency_wait();
  const int S = n_tail + n_pre;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float den = 0.f, mx = -INFINITY;
  for (int sb = 0; sb < S; sb += kBatch) {
    float lv[kBatch];
    float4 x0[kBatch], x1[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int s = sb + j;
      lv[j] = -INFINITY;
      x0[j] = x1[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < S) {
        const bool tail = s < n_tail;
        const long long row =
            tail ? tail_row + (long long)s * a.rows
                 : pre_row + (s - n_tail) * pre_step;
        const float* o =
            (tail ? a.part_o : p.pre_o) + row * kHeadDim + lane * 8;
        lv[j] = (tail ? a.part_lse : p.pre_lse)[row];
        x0[j] = *reinterpret_cast<const float4*>(o);
        x1[j] = *reinterpret_cast<const float4*>(o + 4);
      }
    }
    float bm = lv[0];
#pragma unroll
    for (int j = 1; j < kBatch; ++j) bm = fmaxf(bm, lv[j]);
    if (bm == -INFINITY) continue;  // no partial of this batch saw a key
    if (bm > mx) {
      const float c = exp2f(mx - bm);  // 0 while nothing was summed
      den *= c;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] *= c;
      mx = bm;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (lv[j] == -INFINITY) continue;  // an empty partial's row is not data
      const float wt = exp2f(lv[j] - mx);
      den += wt;
      acc[0] += wt * x0[j].x; acc[1] += wt * x0[j].y;
      acc[2] += wt * x0[j].z; acc[3] += wt * x0[j].w;
      acc[4] += wt * x1[j].x; acc[5] += wt * x1[j].y;
      acc[6] += wt * x1[j].z; acc[7] += wt * x1[j].w;
    }
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  uint4 v;
  v.x = pack_bf16(acc[0] * inv, acc[1] * inv);
  v.y = pack_bf16(acc[2] * inv, acc[3] * inv);
  v.z = pack_bf16(acc[4] * inv, acc[5] * inv);
  v.w = pack_bf16(acc[6] * inv, acc[7] * inv);
  *reinterpret_cast<uint4*>(
      a.out + (((long long)b * a.q_len + i) * a.hq + h) * kHeadDim + lane * 8) = v;
}

}  // namespace

cudaError_t launch_shared_plan(const SharedParams& p, cudaStream_t s) {
  // a thread for every request and group; a small block's barriers are cheaper
  const int need = (std::max(p.a.batch, p.groups) + 31) / 32 * 32;
  shared_plan_kernel<<<1, std::max(need, 256), 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_shared_merge(const SharedParams& p, cudaStream_t s) {
  const long long rows = (long long)p.a.batch * p.a.q_len * p.a.hq;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3((unsigned)((rows + kMergeWarps - 1) / kMergeWarps)),
                 dim3(kMergeWarps * 32), 0, s, attr);
  return rows <= (long long)kMergeWarps * 2 * p.pairs
             ? cudaLaunchKernelEx(&cfg, shared_merge_kernel<20>, p)
             : cudaLaunchKernelEx(&cfg, shared_merge_kernel<6>, p);
}

}  // namespace specv
