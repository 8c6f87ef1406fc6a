// Attention of a chunk of new tokens: the plan (chunk_attention.cuh), the merge
// of the row tiles that it cuts, and the zeros of rows that hold no token.
#include <climits>

#include "chunk_attention.cuh"

namespace specv {
namespace {

// At most: a thread for each request and each pair.  Few of both, and of row
// tiles, take a block of kFew, whose barriers are cheaper (with it and without:
// 50 tokens behind 4,096 29.5 and 31.2 us, 300 behind 2,000 40.1 and 41.8, twelve
// requests of 40 24.5 and 26.1).
constexpr int kThreads = 1024;
constexpr int kFew = 128;
constexpr int kWarps = kThreads / 32;
static_assert(kThreads >= kMaxBatch, "");
static_assert(kChunkBuckets == 64, "two a lane");
constexpr int kHeld = 4096;  // pieces whose tile counts shared memory holds
// A run of the rest is at least this long, in 128-token tiles, and one that
// would start or end as close as kSnap to a piece's border starts or ends there
// (a piece costs as much as kPrefixCost tiles).
constexpr int kMinRun = 2;
constexpr int kSnap = 2;

// Inclusive scan over the block; `total` for every thread.  s: kWarps values.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* s, T* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  __syncthreads();  // s is free
  if (lane == 31) s[w] = v;
  __syncthreads();
  if (w == 0) {
    T x = lane < (int)(blockDim.x >> 5) ? s[lane] : T(0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T n = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += n;
    }
    s[lane] = x;
  }
  __syncthreads();
  *total = s[(blockDim.x >> 5) - 1];
  return v + (w ? s[w - 1] : T(0));
}

// The last i in [0, n) with at[i] <= x (at[0] <= x).
__device__ __forceinline__ int last_at_most(const int* at, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// One CTA.  Ranks and sums are of whole numbers in a fixed order, so the plan,
// and with it every rounding of the result, is the same on every run.
__global__ void __launch_bounds__(kThreads) chunk_plan_kernel(const ChunkParams p) {
  __shared__ int s_tile0[kMaxBatch + 1];
  __shared__ int s_count[kChunkBuckets], s_base[kChunkBuckets];
  __shared__ int s_run[kChunkBuckets];
  __shared__ int s_warp[kWarps][kChunkBuckets];
  __shared__ int s_scan[kWarps];
  __shared__ long long s_scan64[kWarps];
  __shared__ int s_units[kThreads + 1], s_ranges[kThreads + 1];
  __shared__ int s_before[kThreads];  // runs that are not empty, before each
  __shared__ int s_tiles[kHeld];      // of the pieces, when they are few
  __shared__ int s_longest, s_load;
  const AttnParams& a = p.a;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int nt = blockDim.x, nw = nt >> 5;
  // the attention kernel may set itself up now; it waits for this grid
  tc_grid_launch_dependents();
  if (tid == 0) s_longest = s_load = 0;
  if (tid < kChunkBuckets) s_count[tid] = s_run[tid] = 0;
  __syncthreads();
  int tiles = 0;
  if (tid < a.batch) {
    const ChunkRows r = chunk_rows(a, tid);
    tiles = chunk_row_tiles(r, p.cta_rows);
    if (tiles) atomicMax(&s_longest, (r.len + kPrefixTile - 1) / kPrefixTile);
  }
  int T;
  const int upto = block_scan(tiles, s_scan, &T);
  if (tid < a.batch) s_tile0[tid + 1] = upto;
  if (tid == 0) s_tile0[0] = 0;
  __syncthreads();
  const int longest = s_longest;
  const bool held = (long long)T * a.hkv <= kHeld;
  auto tile_at = [&](int i, int* b, int* m) {
    *b = last_at_most(s_tile0, a.batch, i);
    *m = i - s_tile0[*b];
    return chunk_tiles(chunk_rows(a, *b), *m, a.group, p.cta_rows);
  };
  // 0 the longest
  auto bucket_of = [&](int t) {
    return kChunkBuckets - 1 -
           (int)((long long)t * kChunkBuckets / (longest + 1));
  };
  for (int i = tid; i < T; i += nt) {
    int b, m;
    atomicAdd(&s_count[bucket_of(tile_at(i, &b, &m))], 1);
  }
  __syncthreads();
  if (w == 0) {  // two buckets a lane
    const int c0 = s_count[2 * lane], c1 = s_count[2 * lane + 1];
    int n = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += up;
    }
    s_base[2 * lane] = n - c0 - c1;
    s_base[2 * lane + 1] = n - c1;
  }
  // places in a bucket, in the tiles' order
  for (int i0 = 0; i0 < T; i0 += nt) {
    for (int k = tid; k < nw * kChunkBuckets; k += nt)
      (&s_warp[0][0])[k] = 0;
    __syncthreads();
    const int i = i0 + tid;
    int b = 0, m = 0, t = 0, bucket = -1;
    if (i < T) {
      t = tile_at(i, &b, &m);
      bucket = bucket_of(t);
    }
    const unsigned same = __match_any_sync(0xffffffffu, bucket);
    const int before = __popc(same & ((1u << lane) - 1));
    if (bucket >= 0 && before == 0) s_warp[w][bucket] = __popc(same);
    __syncthreads();
    if (tid < kChunkBuckets) {
      int n = s_run[tid];
      for (int k = 0; k < nw; ++k) {
        const int c = s_warp[k][tid];
        s_warp[k][tid] = n;
        n += c;
      }
      s_run[tid] = n;
    }
    __syncthreads();
    if (i < T) {
      ChunkPiece* to = p.pieces + (long long)s_base[bucket] * a.hkv +
                       s_warp[w][bucket] + before;
      const ChunkRows r = chunk_rows(a, b);
      for (int g = 0; g < a.hkv; ++g, to += s_count[bucket]) {
        if (held) s_tiles[to - p.pieces] = t;
        *to = ChunkPiece{b,      g,       m * 2 * p.cta_rows,   t,
                         r.rows, r.first, r.len - r.live + 1, r.len - 1};
      }
    }
    __syncthreads();
  }
  // rounds, and the rest
  const int P = p.pairs, N = T * a.hkv, rounds = N / P, rest = N - rounds * P;
  auto tiles_of = [&](long long i) {
    return held ? s_tiles[i] : p.pieces[i].tiles;
  };
  long long dealt = 0;  // of pair tid
  if (tid < P) {
#pragma unroll 4
    for (int r = 0; r < rounds; ++r)
      dealt += tiles_of((long long)r * P + (r & 1 ? P - 1 - tid : tid)) +
               kPrefixCost;
  }
  int R;
  const int units = block_scan(
      tid < rest ? tiles_of((long long)rounds * P + tid) : 0, s_scan, &R);
  s_units[tid + 1] = units;
  if (tid == 0) s_units[0] = 0;
  long long sum;
  block_scan(dealt, s_scan64, &sum);
  // few tiles go to few pairs
  const int takers = rounds ? P : max(1, min(P, R / kMinRun));
  const long long target =
      (sum + R + (long long)kPrefixCost * (rest + takers) + takers - 1) / takers;
  if (tid < P) {
    const int mine = rounds & 1 ? P - 1 - tid : tid;
    const long long whole =
        dealt + (mine < rest ? s_units[mine + 1] - s_units[mine] + kPrefixCost : 0);
    atomicMax(&s_load, (int)min(whole, (long long)INT_MAX));
  }
  __syncthreads();
  const bool split = rest && s_load > target + target / 64 + 1;
  // a pair's share of the rest
  const long long share =
      tid < takers ? max(0LL, target - dealt - kPrefixCost) : 0;
  long long all;
  const long long end = block_scan(share, s_scan64, &all);
  if (tid < P) {
    int u = all ? (int)((double)R * (double)end / (double)all) : R;
    if (tid == P - 1) u = R;
    if (rest) {
      const int i = last_at_most(s_units, rest, min(u, R - 1));
      if (u - s_units[i] <= kSnap) u = s_units[i];
      else if (s_units[i + 1] - u <= kSnap) u = s_units[i + 1];
    }
    if (tid == P - 1) u = R;
    s_ranges[tid + 1] = u;
    if (tid == 0) {
      s_ranges[0] = 0;
      *p.head = ChunkHead{rounds, rest, split, 0};
    }
  }
  __syncthreads();
  // a cut piece's partials have neighbouring slots, in the order of its runs
  const int n = tid < P ? s_ranges[tid + 1] - s_ranges[tid] : 0;
  int sum_n;
  const int filled = block_scan(n ? 1 : 0, s_scan, &sum_n) - (n ? 1 : 0);
  if (tid < P) s_before[tid] = filled;
  __syncthreads();
  int first = 0, parts = 0;
  if (tid < rest) {
    first = s_before[last_at_most(s_ranges, P, s_units[tid])];
    parts = s_before[last_at_most(s_ranges, P, s_units[tid + 1] - 1)] + 1 - first;
  }
  const int slots = parts > 1 ? parts : 0;
  const int slot = block_scan(slots, s_scan, &sum_n) - slots;
  __syncthreads();
  if (tid < rest) {
    p.rest[tid] = make_int2(slot, parts);
    s_tiles[tid] = slot - first;  // (a rest is shorter than kHeld)
  }
  __syncthreads();
  if (tid < P) {
    const int i = n ? last_at_most(s_units, rest, s_ranges[tid]) : 0;
    p.runs[tid] =
        ChunkRun{i, s_ranges[tid] - s_units[i], n, n ? s_tiles[i] + filled : 0};
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Rows of cut tiles: out = sum_s 2^(lse_s - lse) o_s over the runs.  One warp
// per row, lane l channels 8l .. 8l+7.  Then the rows without a token.
constexpr int kMergeWarps = 8;
constexpr int kBatch = 8;  // partials in flight

__global__ void __launch_bounds__(kMergeWarps * 32)
    chunk_merge_kernel(const ChunkParams p) {
  const AttnParams& a = p.a;
  const int lane = threadIdx.x & 31;
  // the call that follows may set itself up
  tc_grid_launch_dependents();
  // Block rows in front of and behind the live ones, which no other kernel of the
  // call writes (the attention has waited for whatever wrote them before).
  const long long vecs = (long long)a.hq * (kHeadDim / 8);  // 16 bytes, a token
  for (int b = 0; b < a.batch; ++b) {
    const ChunkRows cr = chunk_rows(a, b);
    if (cr.live == a.q_len) continue;
    uint4* o = reinterpret_cast<uint4*>(a.out) + (long long)b * a.q_len * vecs;
    const long long front = cr.first * vecs, from = (cr.first + cr.live) * vecs;
    const long long n = front + a.q_len * vecs - from;
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n;
         i += (long long)gridDim.x * blockDim.x)
      o[i < front ? i : from + (i - front)] = make_uint4(0, 0, 0, 0);
  }
  tc_grid_dependency_wait();
  const ChunkHead h = *p.head;
  if (h.split) {
    for (int w = blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
         w < h.rest * kPrefixRows; w += gridDim.x * kMergeWarps) {
      const int i = w / kPrefixRows, r = w % kPrefixRows;
      const int2 at = p.rest[i];
      const ChunkPiece e = p.pieces[(long long)h.rounds * p.pairs + i];
      if (at.y <= 1) continue;  // whole
      const int half = r / 128, in = r - half * 128;
      const int R = e.row0 + half * p.cta_rows + in;
      if (in >= p.cta_rows || R >= e.rows) continue;
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      float den = 0.f, mx = -INFINITY;
      for (int c = 0; c < at.y; c += kBatch) {
        float lv[kBatch];
        float4 x0[kBatch], x1[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          lv[j] = -INFINITY;
          x0[j] = x1[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c + j < at.y) {
            const long long row = (long long)(at.x + c + j) * kPrefixRows + r;
            const float* o = p.pre_o + row * kHeadDim + lane * 8;
            lv[j] = p.pre_lse[row];
            x0[j] = *reinterpret_cast<const float4*>(o);
            x1[j] = *reinterpret_cast<const float4*>(o + 4);
          }
        }
        float bm = lv[0];
#pragma unroll
        for (int j = 1; j < kBatch; ++j) bm = fmaxf(bm, lv[j]);
        if (bm > mx) {
          const float k = exp2f(mx - bm);  // 0 while nothing was summed
          den *= k;
#pragma unroll
          for (int e8 = 0; e8 < 8; ++e8) acc[e8] *= k;
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
      const int tok = R / a.group;
      const long long to = ((long long)e.b * a.q_len + e.first + tok) * a.hq +
                           e.g * a.group + (R - tok * a.group);
      *reinterpret_cast<uint4*>(a.out + to * kHeadDim + lane * 8) = v;
    }
  }
}

}  // namespace

cudaError_t launch_chunk_plan(const ChunkParams& p, cudaStream_t s) {
  const long long tiles =
      p.a.batch * chunk_tiles_of((long long)p.a.q_len * p.a.group,
                                   p.cta_rows);
  const bool few = p.a.batch <= kFew && p.pairs <= kFew && tiles <= 4 * kFew;
  chunk_plan_kernel<<<1, few ? kFew : kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_chunk_merge(const ChunkParams& p, int sms, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(sms * 4), dim3(kMergeWarps * 32), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, chunk_merge_kernel, p);
}

}  // namespace specv
