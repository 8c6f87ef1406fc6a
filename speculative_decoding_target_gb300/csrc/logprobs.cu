// Log probabilities of given tokens, the entropy of their distributions and the
// most likely alternatives, in one pass over the logits.
//
// With z_v = x_v / T, S = sum_v e^(z_v - max z):
//   log p(v) = z_v - max z - ln S,   H = ln S - sum_v e^(z_v - max z)
//                                                     (z_v - max z) / S,
// and the alternatives are the first `top` tokens by (x descending, id
// ascending).  4 or 2 bytes a token against about five instructions: HBM bounds
// it as long as the sums keep up.
//
// A cluster of CTAs takes a row; a thread takes every 512th 16-byte vector of
// its CTA's part.  In base 2, with t = (x - ref) log2(e) / T:
//   s = sum 2^t,  h = sum 2^t t
// against a reference of the thread's own, its first batch's largest value; a
// batch that exceeds it by 2^kRebase moves it (the sums stay far inside fp32's
// range, so nothing has to follow each new maximum).  A batch is summed by
// itself before it joins the sums: beside a weight of one, single small weights
// would be lost.  Threads' sums join in fp32 inside a warp and in fp64 beyond.
// Values below ref - kLow T / log2(e) weigh nothing in fp32 and are raised to
// that, -inf and NaN among them, so that t stays a number.
//
// Alternatives.  Each thread keeps its largest value and the vector that holds
// it (the first, of equals).  The `top` best tokens of a CTA lie in the vectors'
// threads with the `top` best (value, vector); a thread of rank r among them
// holds at most top - r of them.  So a warp reads each winner's values once more
// (from L1 or L2), and takes out its best until one falls below the last
// winner's: one or two each on real rows, and a bounded number on any row.
#include <cuda_bf16.h>

#include <atomic>

#include "common.cuh"
#include "logprobs.cuh"
#include "pair_ptx.cuh"

namespace specv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 4;          // 16-byte vectors of a batch
constexpr int kMaxCluster = 16;
constexpr float kRebase = 8.f;    // log2
constexpr float kLow = 160.f;     // log2
constexpr int kTop = kLogprobMaxTop;
constexpr int kGroups = 64;       // groups of 8 threads
// what winners of ranks 0 .. top - 1 may hand in; also a cluster's lists
constexpr int kCands = kTop * (kTop + 1) / 2;
static_assert(kCands >= kMaxCluster * kTop, "");
constexpr float kMaxFinite = 3.402823466e+38f;
typedef unsigned long long u64;

__device__ __forceinline__ u64 pack2(float lo, float hi) {
  u64 v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ float2 unpack2(u64 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// NaN counts as -inf, +inf as the type's largest value.
template <typename T>
__device__ __forceinline__ constexpr float most_of() {
  return sizeof(T) == 2 ? 3.38953139e+38f : kMaxFinite;
}
template <typename T>
__device__ __forceinline__ float clean(float x) {
  return fminf(fmaxf(x, -INFINITY), most_of<T>());
}

template <typename T>
struct Vec {
  static constexpr int kN = 16 / sizeof(T);
};
__device__ __forceinline__ void widen(uint4 v, float (&x)[8], __nv_bfloat16*) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = __uint_as_float(w[k] << 16);
    x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen(uint4 v, float (&x)[4], float*) {
  x[0] = __uint_as_float(v.x);
  x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z);
  x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Largest of a vector (-inf for one of NaN).
__device__ __forceinline__ float largest(uint4 v, __nv_bfloat16*) {
  const uint32_t m =
      max_bf16x2(max_bf16x2(v.x, v.y), max_bf16x2(v.z, v.w));
  return fmaxf(fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u)),
               -INFINITY);
}
__device__ __forceinline__ float largest(uint4 v, float*) {
  return fmaxf(fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                     fmaxf(__uint_as_float(v.z), __uint_as_float(v.w))),
               -INFINITY);
}
// A vector's values, those below `low` (and NaN) raised to it.
__device__ __forceinline__ void widen_from(uint4 v, float low, float (&x)[8],
                                           __nv_bfloat16* t) {
  // `low` rounded down
  const uint32_t l = (__float_as_uint(low) + (low < 0.f ? 0xffffu : 0u)) &
                     0xffff0000u;
  const uint32_t l2 = l | l >> 16;
  v.x = max_bf16x2(v.x, l2);
  v.y = max_bf16x2(v.y, l2);
  v.z = max_bf16x2(v.z, l2);
  v.w = max_bf16x2(v.w, l2);
  widen(v, x, t);
}
__device__ __forceinline__ void widen_from(uint4 v, float low, float (&x)[4],
                                           float* t) {
  widen(v, x, t);
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = fmaxf(x[k], low);
}

// Larger value first, then the smaller number.
__device__ __forceinline__ bool better(float a, int ia, float b, int ib) {
  return a > b || (a == b && ia < ib);
}

struct Shared {
  float max[kWarps];
  double s[kWarps], h[kWarps];
  // a CTA's results, read by the cluster's first
  float row_max;
  double row_s, row_h;
  float top_v[kTop];
  int top_i[kTop];
  // selection
  __align__(16) float group[kGroups];
  float bound;
  int listed, cands;
  float list_v[kThreads];
  int list_vec[kThreads], list_t[kThreads];
  int winner[kTop];
  float cand_v[kCands];
  int cand_i[kCands];
};

// A CTA's part of a row: vectors [begin, end) from the first 16-byte boundary
// on; the tokens in front of that and behind the last vector, at most 7 each,
// are the first CTA's, one a thread (the thread's "odd" token).
template <typename T>
struct Part {
  const T* x;
  int head;          // tokens in front of the first vector
  int begin, end;
  int odd;           // this thread's odd token, or -1
  __device__ Part(const T* x, int vocab, int rank, int csize) : x(x) {
    constexpr int kN = Vec<T>::kN;
    const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    head = min((kN - off) % kN, vocab);
    const int nv = (vocab - head) / kN;
    begin = (int)((long long)nv * rank / csize);
    end = (int)((long long)nv * (rank + 1) / csize);
    odd = odd_of(threadIdx.x, vocab, rank, nv);
  }
  __device__ __forceinline__ int odd_of(int t, int vocab, int rank, int nv) const {
    if (rank) return -1;
    if (t < head) return t;
    const int tail = head + nv * Vec<T>::kN + t - 8;
    return t >= 8 && tail < vocab ? tail : -1;
  }
  __device__ __forceinline__ const uint4* vec(int v) const {
    return reinterpret_cast<const uint4*>(x + head) + v;
  }
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) {
  return __bfloat162float(x);
}

// A thread's sums against ref, its largest value and where it is.
struct Sums {
  float ref, low, s, h, max;
  int vec;
};

// Moves the reference to `ref`, a finite value.
template <typename T>
__device__ __forceinline__ void rebase(Sums& a, float ref, float c) {
  if (a.ref > -INFINITY) {
    const float d = (a.ref - ref) * c, k = ex2(d);
    a.h = (a.h + fmaxf(d, -kLow) * a.s) * k;
    a.s *= k;
  }
  a.ref = ref;
  // below ref by more than its rounding
  a.low = fmaxf(ref - fmaxf(kLow / c, fabsf(ref) * 4.8e-7f), -most_of<T>());
}

// A batch of vectors v0, v0 + kThreads, .. joins the sums.
template <typename T>
__device__ __forceinline__ void join(Sums& a, const uint4 (&raw)[kVecs], int v0,
                                     float c) {
  constexpr int kN = Vec<T>::kN;
  float most = -INFINITY;
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    const float m = largest(raw[u], static_cast<T*>(nullptr));
    most = fmaxf(most, m);
    const float fine = fminf(m, most_of<T>());
    if (fine > a.max) {
      a.max = fine;
      a.vec = v0 + u * kThreads;
    }
  }
  if (most == -INFINITY) return;  // nothing that weighs
  const bool endless = most == INFINITY;
  most = fminf(most, most_of<T>());
  if (!((most - a.ref) * c <= kRebase)) rebase<T>(a, most, c);
  if (endless || a.ref < -1e38f) {  // no number to raise to, or none below
    float s = 0.f, h = 0.f;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      float x[kN];
      widen(raw[u], x, static_cast<T*>(nullptr));
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const float t = fmaxf((clean<T>(x[k]) - a.ref) * c, -kLow), e = ex2(t);
        s += e;
        h = fmaf(e, t, h);
      }
    }
    a.s += s;
    a.h += h;
    return;
  }
  const u64 c2 = pack2(c, c), r2 = pack2(-a.ref, -a.ref);
  u64 s = 0, h = 0;  // two zeros each
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    float x[kN];
    widen_from(raw[u], a.low, x, static_cast<T*>(nullptr));
#pragma unroll
    for (int k = 0; k < kN; k += 2) {
      const u64 t = mul2(add2(pack2(x[k], x[k + 1]), r2), c2);
      const float2 tf = unpack2(t);
      const u64 e = pack2(ex2(tf.x), ex2(tf.y));
      s = add2(s, e);
      h = fma2(e, t, h);
    }
  }
  const float2 sf = unpack2(s), hf = unpack2(h);
  a.s += sf.x + sf.y;
  a.h += hf.x + hf.y;
}

template <typename T>
__device__ __forceinline__ Sums stream(const Part<T>& part, float c) {
  Sums a{-INFINITY, 0.f, 0.f, 0.f, -INFINITY, 0};
  const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -inf
  const uint4 empty = make_uint4(none, none, none, none);
  int v = part.begin + (int)threadIdx.x;
  uint4 raw[kVecs];
  auto load = [&](int at) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int w = at + u * kThreads;
      raw[u] = empty;
      if (w < part.end) raw[u] = __ldg(part.vec(w));
    }
  };
  load(v);
  for (; v < part.end; v += kVecs * kThreads) {
    uint4 now[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) now[u] = raw[u];
    load(v + kVecs * kThreads);
    join<T>(a, now, v, c);
  }
  if (part.odd >= 0) {
    const float x = clean<T>(to_float(part.x[part.odd]));
    // before every vector, or behind them
    const int at = part.odd < part.head ? -1 : 1 << 30;
    if (x > a.max || (x == a.max && at < a.vec && x > -INFINITY)) {
      a.max = x;
      a.vec = at;
    }
    if (x > -INFINITY) {
      if (!((x - a.ref) * c <= kRebase)) rebase<T>(a, x, c);
      const float t = fmaxf((x - a.ref) * c, -kLow), e = ex2(t);
      a.s += e;
      a.h = fmaf(e, t, a.h);
    }
  }
  return a;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// The CTA's best `top` tokens into sh.top_v / top_i (-inf and -1 behind the
// last finite one).  Called by the whole CTA; ends with a barrier.
template <typename T>
__device__ void select(Shared& sh, const Part<T>& part, const Sums& a, int vocab,
                       int rank, int top) {
  constexpr int kN = Vec<T>::kN;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  // a bound: the top-th largest of 64 groups' maxima
  float g = a.max;
#pragma unroll
  for (int o = 4; o; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
  if ((lane & 7) == 0) sh.group[tid >> 3] = g;
  if (tid == 0) sh.listed = sh.cands = 0;
  if (tid < kTop) {
    sh.top_v[tid] = -INFINITY;
    sh.top_i[tid] = -1;
  }
  __syncthreads();
  if (tid < kGroups) {
    const float mine = sh.group[tid];
    int rank_g = 0;
#pragma unroll 8
    for (int k = 0; k < kGroups; ++k)
      rank_g += better(sh.group[k], k, mine, tid);
    if (rank_g == top - 1) sh.bound = mine;
  }
  __syncthreads();
  // the threads at or above it, in any order
  const bool in = a.max >= sh.bound && a.max > -INFINITY;
  const unsigned who = __ballot_sync(0xffffffffu, in);
  int at = 0;
  if (lane == 0 && who) at = atomicAdd(&sh.listed, __popc(who));
  at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1));
  if (in) {
    sh.list_v[at] = a.max;
    sh.list_vec[at] = a.vec;
    sh.list_t[at] = tid;
  }
  __syncthreads();
  const int n = sh.listed;
  if (tid < n) {
    const float v = sh.list_v[tid];
    const int vec = sh.list_vec[tid];
    const int key_t = sh.list_t[tid];  // odd tokens: in the threads' order
    int r = 0;
    for (int k = 0; k < n; ++k) {
      const float kv = sh.list_v[k];
      const int kvec = sh.list_vec[k];
      r += kv > v || (kv == v && (kvec < vec ||
                                  (kvec == vec && sh.list_t[k] < key_t)));
    }
    if (r < top) sh.winner[r] = key_t;
    if (r == top - 1) sh.bound = v;
  }
  __syncthreads();
  const int winners = min(n, top);
  const float bound = n >= top ? sh.bound : -INFINITY;
  const int nv = (vocab - part.head) / kN;
  for (int r = w; r < winners; r += kWarps) {
    const int t = sh.winner[r];
    constexpr int kHold = kLogprobMaxVocab / kThreads / 32;  // 32 values a lane
    float x[kHold];
    const int v0 = part.begin + t + lane * kThreads;
#pragma unroll
    for (int q = 0; q < kHold / kN; ++q) {
      const int v = v0 + q * 32 * kThreads;
      float y[kN];
#pragma unroll
      for (int k = 0; k < kN; ++k) y[k] = -INFINITY;
      if (v < part.end) widen(__ldg(part.vec(v)), y, static_cast<T*>(nullptr));
#pragma unroll
      for (int k = 0; k < kN; ++k) x[q * kN + k] = clean<T>(y[k]);
    }
    // the odd token, lane 31's only
    float odd_x = -INFINITY;
    const int odd = part.odd_of(t, vocab, rank, nv);
    if (lane == 31 && odd >= 0) odd_x = clean<T>(to_float(part.x[odd]));
    for (int left = top - r; left; --left) {
      float best = odd_x;
      int id = odd_x > -INFINITY ? odd : 0x7fffffff;
#pragma unroll
      for (int k = 0; k < kHold; ++k) {
        const int i = part.head + (v0 + k / kN * 32 * kThreads) * kN + k % kN;
        if (x[k] > -INFINITY && better(x[k], i, best, id)) {
          best = x[k];
          id = i;
        }
      }
      float wb = best;
      int wi = id;
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const float ov = __shfl_xor_sync(0xffffffffu, wb, o);
        const int oi = __shfl_xor_sync(0xffffffffu, wi, o);
        if (better(ov, oi, wb, wi)) {
          wb = ov;
          wi = oi;
        }
      }
      if (wb == -INFINITY || wb < bound) break;  // uniform
      if (lane == 0) {
        const int c = atomicAdd(&sh.cands, 1);
        sh.cand_v[c] = wb;
        sh.cand_i[c] = wi;
      }
      // taken out
      if (wi == odd) odd_x = -INFINITY;
#pragma unroll
      for (int k = 0; k < kHold; ++k)
        if (part.head + (v0 + k / kN * 32 * kThreads) * kN + k % kN == wi)
          x[k] = -INFINITY;
    }
  }
  __syncthreads();
  const int cands = sh.cands;
  for (int j = tid; j < cands; j += kThreads) {
    const float v = sh.cand_v[j];
    const int i = sh.cand_i[j];
    int r = 0;
    for (int k = 0; k < cands; ++k) r += better(sh.cand_v[k], sh.cand_i[k], v, i);
    if (r < top) {
      sh.top_v[r] = v;
      sh.top_i[r] = i;
    }
  }
  __syncthreads();
}

template <typename V>
__device__ __forceinline__ V peer_load(const V* p, uint32_t rank) {
  const uint32_t at = tc::map_to(tc::smem_u32(p), rank);
  V v;
  if constexpr (sizeof(V) == 8) {
    u64 r;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(r) : "r"(at));
    v = *reinterpret_cast<const V*>(&r);
  } else {
    uint32_t r;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(r) : "r"(at));
    v = *reinterpret_cast<const V*>(&r);
  }
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
    logprobs_kernel(const LogprobParams p, int csize) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / csize, rank = blockIdx.x - row * csize;
  const T* x = static_cast<const T*>(p.logits) + row * p.row_stride;
  const float temp = p.temperature ? p.temperature[row] : 1.f;
  const int token = p.token ? p.token[row] : 0;
  const long long out = (long long)row * p.top;
  if (token < 0 || token >= p.vocab || !(temp >= 0.f && temp <= kMaxFinite)) {
    if (rank) return;  // an idle row
    if (tid == 0 && p.logprob) p.logprob[row] = 0.f;
    if (tid == 0 && p.entropy) p.entropy[row] = 0.f;
    if (tid < p.top) {
      p.top_ids[out + tid] = -1;
      p.top_logprobs[out + tid] = -INFINITY;
    }
    return;
  }
  const bool one = temp == 0.f;  // all the mass on the first of the largest
  const int top = one ? max(p.top, 1) : p.top;
  // 1 / T stays inside fp32's range
  const float c =
      one ? 1.f
          : fminf(fmaxf(__fdiv_rn(1.4426950408889634f, temp), 1e-37f), 1e37f);
  float given = 0.f;
  if (tid == 0) given = clean<T>(to_float(x[token]));
  const Part<T> part(x, p.vocab, rank, csize);
  const Sums a = stream(part, c);
  // the CTA's sums
  const float wm = warp_max(a.max);
  if (lane == 0) sh.max[w] = wm;
  __syncthreads();
  float m = sh.max[lane & (kWarps - 1)];
  m = warp_max(m);
  float s = 0.f, h = 0.f;
  if (a.ref > -INFINITY) {
    const float d = fmaxf((a.ref - m) * c, -kLow), k = ex2(d);
    s = a.s * k;
    h = fmaf(d, s, a.h * k);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    h += __shfl_xor_sync(0xffffffffu, h, o);
  }
  if (lane == 0) {
    sh.s[w] = s;
    sh.h[w] = h;
  }
  __syncthreads();
  if (tid == 0) {
    double ss = 0., hh = 0.;
    for (int k = 0; k < kWarps; ++k) {
      ss += sh.s[k];
      hh += sh.h[k];
    }
    sh.row_max = m;
    sh.row_s = ss;
    sh.row_h = hh;
  }
  if (top) select(sh, part, a, p.vocab, rank, top);
  if (csize > 1) {
    tc::cluster_sync();
    if (rank == 0) {
      if (w == 0) {  // sums, a lane for each CTA
        float pm = -INFINITY;
        double ps = 0., ph = 0.;
        if (lane < csize) {
          pm = peer_load(&sh.row_max, lane);
          ps = peer_load(&sh.row_s, lane);
          ph = peer_load(&sh.row_h, lane);
        }
        const float all = warp_max(pm);
        if (pm > -INFINITY) {
          const float d = fmaxf((pm - all) * c, -kLow), k = ex2(d);
          ph = (ph + (double)d * ps) * k;
          ps *= k;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          ps += __shfl_xor_sync(0xffffffffu, ps, o);
          ph += __shfl_xor_sync(0xffffffffu, ph, o);
        }
        __syncwarp();
        if (lane == 0) {
          sh.max[0] = all;
          sh.s[0] = ps;
          sh.h[0] = ph;
        }
      }
      const int n = csize * top;
      for (int j = tid; j < n; j += kThreads) {
        const int from = j / top, k = j - from * top;
        sh.cand_v[j] = peer_load(&sh.top_v[k], from);
        sh.cand_i[j] = peer_load(&sh.top_i[k], from);
      }
    }
    tc::cluster_sync();  // no CTA leaves while the first reads
    if (rank) return;
    const int n = csize * top;
    for (int j = tid; j < n; j += kThreads) {
      const float v = sh.cand_v[j];
      const int i = sh.cand_i[j];
      int r = 0;
      for (int k = 0; k < n; ++k)
        r += better(sh.cand_v[k], sh.cand_i[k], v, i);
      if (r < top && i >= 0) {
        sh.top_v[r] = v;
        sh.top_i[r] = i;
      }
      if (r < top && i < 0) {
        sh.top_v[r] = -INFINITY;
        sh.top_i[r] = -1;
      }
    }
    __syncthreads();
    m = sh.max[0];
  } else {
    if (tid == 0) {
      sh.s[0] = sh.row_s;
      sh.h[0] = sh.row_h;
    }
    __syncthreads();
  }
  const double ln2 = 0.69314718055994530942;
  const bool none = m == -INFINITY;  // no finite logit
  const double sum = sh.s[0];
  const double log2s = none ? 0. : log2(sum);
  auto logprob = [&](float v, bool first) {
    if (one) return first ? 0.f : -INFINITY;
    if (none || v == -INFINITY) return -INFINITY;
    return (float)((((double)v - m) * c - log2s) * ln2);
  };
  if (tid == 0) {
    if (p.logprob)
      p.logprob[row] = logprob(given, token == sh.top_i[0]);
    if (p.entropy)
      p.entropy[row] =
          one || none ? 0.f : fmaxf((float)((log2s - sh.h[0] / sum) * ln2), 0.f);
  }
  if (tid < p.top) {
    const int i = sh.top_i[tid];
    p.top_ids[out + tid] = i;
    p.top_logprobs[out + tid] = i < 0 ? -INFINITY : logprob(sh.top_v[tid], tid == 0);
  }
}

template <typename T>
cudaError_t launch(const LogprobParams& p, int csize, cudaStream_t s) {
  // once per device (an attribute call per launch costs microseconds)
  static std::atomic<uint64_t> ready{0};
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(logprobs_kernel<T>,
                             cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.rows * csize);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = csize;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, p, csize);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams& p, bool bf16, int sms,
                            cudaStream_t s) {
  int csize = 1;
  const int batch = kThreads * kVecs * (bf16 ? 8 : 4);  // tokens
  while (csize < kMaxCluster && (long long)p.rows * csize < 2 * sms &&
         p.vocab > csize * batch)
    csize *= 2;
  return bf16 ? launch<__nv_bfloat16>(p, csize, s) : launch<float>(p, csize, s);
}

}  // namespace specv
