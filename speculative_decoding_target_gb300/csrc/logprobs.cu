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
// A CTA a row: 256 threads, four CTAs an SM, so that one row's reductions and
// selection run under the others' loads, and the hardware deals the rows out.
// (1,024 bf16 rows of 248,320 with top 20: 90.7 us, 5.6 TB/s; 512 threads 90.6, but
// 6,000 rows of 33,000 with top 5 then take 186 us instead of 110.  Resident CTAs that start on
// their next row under the last one's selection: 103 and 223 us.  Equal runs of
// slices that cut rows, joined by a second kernel: 112 us, and 256 rows 44 instead
// of 32.  Such runs dealt out by a counter, shorter ones last: 121 to 150 us.)
//
// While that leaves SMs idle, a cluster a row, of a size that puts up to two CTAs on
// an SM: 100 rows of 33,000 11.1 us with two CTAs a row, 12.2 with four; 64 fp32
// rows of 248,320 17.8 with four and 20.1 with eight; 152 rows 31.5 with two and 35.2
// with four, and 153, with one, 30.7.  (Sizes that are no power of two leave parts of
// the GPU's groups of SMs empty: 100 rows 26 us with three, 20 with two.)
//
// A thread takes every 256th 16-byte vector of its CTA's part of a row.  In
// base 2, with t = (x - ref) log2(e) / T:
//   s = sum 2^t,  h = sum 2^t t
// against a reference of the thread's own, its first batch's largest value; a
// batch that exceeds it by 2^kRebase moves it (the sums stay far inside fp32's
// range, so nothing has to follow each new maximum).  A batch is summed by
// itself before it joins the sums: beside a weight of one, single small weights
// would be lost.
// t is one fused step on the logit, x c - fl(ref c); what that product was
// rounded by (delta) is put right where the threads' sums join.  A batch with
// values that are not finite makes h NaN or infinite; it, and one whose ref c is
// too large to be rounded so, is summed from (x - ref) c, where -inf and NaN
// weigh nothing.  (Rows with banned tokens, 1,024 bf16 rows of 248,320, top 20: one
// in a thousand 113 us, half of them 132, all in one half of the row 109.)
//
// Alternatives.  Each thread keeps its largest value, the vector that holds it
// (the first, of equals) and the largest value of its other vectors.  The `top`
// best tokens of a CTA lie in the threads with the `top` best (value, vector); a
// thread of rank r among them holds at most top - r of them.  Each of these
// winners reads that one vector again (on its way while they are ranked) and hands
// in what is not below the last winner's value.  A winner whose other vectors hold
// such values too, as with many equals, is read by a warp as a whole, and its best
// top - r are taken out.  Values are compared without flushing subnormal ones, or
// as whole numbers of the same order.  (1,024 bf16 rows: top 20 takes 11 us more than none;
// reading all values of every winner took 38.)
#include <cuda_bf16.h>

#include <atomic>

#include "common.cuh"
#include "logprobs.cuh"
#include "packed.cuh"
#include "pair_ptx.cuh"

namespace specv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroup = kThreads / 32;  // threads of a group of the bound
constexpr int kCtasPerSm = 4;
constexpr int kVecs = 4;          // 16-byte vectors of a batch
constexpr int kSlice = 4096;      // tokens of a CTA of a cluster, at least
constexpr int kMaxCluster = 16;
constexpr int kClusterCtas = 2;   // of clusters on an SM, at most
constexpr float kRebase = 8.f;    // log2
constexpr float kLow = 160.f;     // log2
constexpr float kLargeRef = 1048576.f;
constexpr int kTop = kLogprobMaxTop;
// what winners of ranks 0 .. top - 1 may hand in
// (a vector of 8 even for the last of them)
constexpr int kCands = kTop * (kTop + 1) / 2 + 28;
constexpr float kMaxFinite = 3.402823466e+38f;
constexpr float kTempMin = 7.8886091e-31f, kTempMax = 1.2676506e+30f;  // 2^-100, 2^100

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What orders the logits keeps subnormal ones apart, which fmaxf, fminf and the
// comparison operators flush here.
__device__ __forceinline__ float max_of(float a, float b) {
  float d;
  asm("max.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_of(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min_of(float a, float b) {
  float d;
  asm("min.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// The larger of the two, and its place if that is m.
__device__ __forceinline__ void rise(float& max, int& at, float m, int place) {
  asm("{\n\t.reg .pred p;\n\tsetp.gt.f32 p, %2, %0;\n\t"
      "selp.b32 %1, %3, %1, p;\n\tmax.f32 %0, %0, %2;\n\t}"
      : "+f"(max), "+r"(at)
      : "f"(m), "r"(place));
}
// (false for NaN)
__device__ __forceinline__ bool at_least(float a, float b) {
  int d;
  asm("{\n\t.reg .pred p;\n\tsetp.ge.f32 p, %1, %2;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(d)
      : "f"(a), "f"(b));
  return d;
}

// NaN counts as -inf, +inf as the type's largest value.
template <typename T>
__device__ __forceinline__ constexpr float most_of() {
  return sizeof(T) == 2 ? 3.38953139e+38f : kMaxFinite;
}
template <typename T>
__device__ __forceinline__ float clean(float x) {
  return min_of(max_of(x, -INFINITY), most_of<T>());
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
  return max_of(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u),
                -INFINITY);
}
__device__ __forceinline__ float largest(uint4 v, float*) {
  return max_of(max_of(__uint_as_float(v.x), __uint_as_float(v.y),
                       __uint_as_float(v.z)),
                __uint_as_float(v.w), -INFINITY);
}
// A value as a whole number of the same order.
__device__ __forceinline__ uint32_t order_of(float v) {
  uint32_t b = __float_as_uint(v);
  if (b == 0x80000000u) b = 0;  // -0 as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// A token as one number: larger value first, then the smaller place (its own, or
// its vector's first token's).  0 is no token.
__device__ __forceinline__ u64 key_of(float v, int place) {
  return (u64)order_of(v) << 32 | (0xffffffffu - (uint32_t)place);
}
__device__ __forceinline__ float value_of(u64 key) {
  const uint32_t o = (uint32_t)(key >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int place_of(u64 key) {
  return (int)(0xffffffffu - (uint32_t)key);
}

struct Shared {
  float max[32], s[kWarps], h[kWarps];  // largest of every kGroup threads; sums
  // selection: keys, in pairs
  __align__(16) u64 list[kThreads + 2];
  __align__(16) u64 cands[kCands + 2];
  u64 bound;
  int listed, found, deep;
  uint16_t deep_t[kTop], deep_r[kTop];
  u64 top[kTop];
};

// A CTA's part of a row: vectors [begin, end) from the first 16-byte boundary
// on, slices [q0, q1) of `slices`.  The tokens in front of that and behind the
// last vector, at most 7 each, go with slice 0, one a thread (the thread's "odd"
// token).
template <typename T>
struct Part {
  const T* x;
  int head;          // tokens in front of the first vector
  int begin, end;
  int odds;          // odd tokens behind the last vector start here; -1: none here
  int odd;           // this thread's odd token, or -1
  int vocab;
  __device__ Part(const T* x, int vocab, int rank, int size)
      : x(x), vocab(vocab) {
    constexpr int kN = Vec<T>::kN;
    const int off = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    head = min((kN - off) % kN, vocab);
    const int nv = (vocab - head) / kN;
    begin = (int)((long long)nv * rank / size);
    end = (int)((long long)nv * (rank + 1) / size);
    odds = rank ? -1 : head + nv * kN;
    odd = odd_of(threadIdx.x);
  }
  __device__ __forceinline__ int odd_of(int t) const {
    if (odds < 0) return -1;
    if (t < head) return t;
    return t >= 8 && odds + t - 8 < vocab ? odds + t - 8 : -1;
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
  float ref, rc, s, h;   // rc = fl(ref c)
  float max, next;       // the largest value, and that of all other vectors
  int vec;               // where the largest is (-1: the odd token)
};

// What ref c was rounded by; 0 where that is no small number any more, and t is
// taken from the difference of the logits.
__device__ __forceinline__ float delta_of(float ref, float c) {
  const float rc = ref * c;
  return fabsf(rc) <= kLargeRef ? fmaf(ref, c, -rc) : 0.f;
}

// Moves the reference to `ref`, a finite value.
__device__ __forceinline__ void rebase(Sums& a, float ref, float c) {
  if (a.ref > -INFINITY) {
    const float d = fmaxf(
        fmaf(a.ref - ref, c, delta_of(ref, c) - delta_of(a.ref, c)), -kLow);
    const float k = ex2(d);
    a.h = (a.h + d * a.s) * k;
    a.s *= k;
  }
  a.ref = ref;
  a.rc = ref * c;
}

// A batch of vectors v0, v0 + kThreads, .. joins the sums; `refill` is called
// with a number that all of the batch went into.
template <typename T, typename F>
__device__ __forceinline__ void join(Sums& a, const uint4 (&raw)[kVecs], int v0,
                                     float c, F refill) {
  constexpr int kN = Vec<T>::kN;
  float m[kVecs], most = -INFINITY;
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    m[u] = largest(raw[u], static_cast<T*>(nullptr));
    most = max_of(most, m[u]);
  }
  if (most == INFINITY) {  // the type's largest, of which the first counts
    most = most_of<T>();
#pragma unroll
    for (int u = 0; u < kVecs; ++u) m[u] = min_of(m[u], most);
  }
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    a.next = max_of(a.next, min_of(m[u], a.max));
    rise(a.max, a.vec, m[u], v0 + u * kThreads);
  }
  refill(most);
  if (!((most - a.ref) * c <= kRebase)) {  // (also without a reference)
    if (most == -INFINITY) return;         // nothing so far that weighs
    rebase(a, most, c);
  }
  const u64 c2 = pack2(c, c), r2 = pack2(-a.rc, -a.rc);
  u64 s2 = 0, h2 = 0;  // two zeros each
#pragma unroll
  for (int u = 0; u < kVecs; ++u) {
    float x[kN];
    widen(raw[u], x, static_cast<T*>(nullptr));
#pragma unroll
    for (int k = 0; k < kN; k += 2) {
      const u64 t = fma2(pack2(x[k], x[k + 1]), c2, r2);
      const float2 tf = unpack2(t);
      const u64 e = pack2(ex2(tf.x), ex2(tf.y));
      s2 = add2(s2, e);
      h2 = fma2(e, t, h2);
    }
  }
  const float2 sf = unpack2(s2), hf = unpack2(h2);
  float s = sf.x + sf.y, h = hf.x + hf.y;
  if (!(fabsf(h) <= kMaxFinite && fabsf(a.rc) <= kLargeRef)) {
    const float delta = delta_of(a.ref, c);
    s = h = 0.f;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      float x[kN];
      widen(raw[u], x, static_cast<T*>(nullptr));
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const float t = fmaxf(fmaf(clean<T>(x[k]) - a.ref, c, delta), -kLow);
        const float e = ex2(t);
        s += e;
        h = fmaf(e, t, h);
      }
    }
  }
  a.s += s;
  a.h += h;
}

// A thread's own ring of batches in shared memory: it copies its vectors there
// and reads them back, so no thread waits for another.
// (Three batches; six where few CTAs share an SM: 256 fp32 rows 47.1 us, not 44.1.)
constexpr int kStages = 3;
constexpr int kStep = kVecs * kThreads;
constexpr int kRingBytes = kStages * kStep * 16;

struct Ring {
  uint32_t base;  // this thread's first place
  uint32_t at;    // and that of the next batch
  __device__ __forceinline__ explicit Ring(const void* smem)
      : base((uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16),
        at(base) {}
  __device__ __forceinline__ uint32_t behind(uint32_t place) const {
    place += kStep * 16;
    return place == base + kRingBytes ? base : place;
  }
  // A batch of vectors from v on, `left` of them in the part.  `after`: what
  // has to be known before (what was read from the place).
  __device__ __forceinline__ void load(const uint4* from, int left, uint32_t to,
                                       float after) {
    if (left >= kStep) {  // (uniform)
#pragma unroll
      for (int u = 0; u < kVecs; ++u) copy(from, u, to, after);
    } else {
#pragma unroll
      for (int u = 0; u < kVecs; ++u)
        if ((int)threadIdx.x + u * kThreads < left) copy(from, u, to, after);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  static __device__ __forceinline__ void copy(const uint4* from, int u,
                                              uint32_t to, float after) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     to + u * kThreads * 16),
                 "l"(from + u * kThreads), "f"(after)
                 : "memory");
  }
  // The first batches of a part.
  template <typename T>
  __device__ __forceinline__ void start(const Part<T>& part) {
    const uint4* from = part.vec(part.begin + (int)threadIdx.x);
    uint32_t to = at;
#pragma unroll
    for (int k = 0; k < kStages; ++k, from += kStep, to = behind(to))
      load(from, part.end - part.begin - k * kStep, to, 0.f);
  }
};

// The sums of a part that the ring has started.
template <typename T>
__device__ __forceinline__ Sums stream(const Part<T>& part, Ring& ring, float c) {
  Sums a{-INFINITY, 0.f, 0.f, 0.f, -INFINITY, -INFINITY, 0};
  int v = part.begin + (int)threadIdx.x;
  int left = part.end - part.begin;
  const uint4* ahead = part.vec(v + kStages * kStep);
  uint4 raw[kVecs];
  auto get = [&]() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(raw[u].x), "=r"(raw[u].y), "=r"(raw[u].z),
                     "=r"(raw[u].w)
                   : "r"(ring.at + u * kThreads * 16)
                   : "memory");
  };
#pragma unroll 1
  for (; left >= kStep; left -= kStep, v += kStep, ahead += kStep) {
    get();
    join<T>(a, raw, v, c, [&](float most) {
      ring.load(ahead, left - kStages * kStep, ring.at, most);
    });
    ring.at = ring.behind(ring.at);
  }
  if (left > 0) {  // the last batch, -inf behind the last vector
    get();
    const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
      if ((int)threadIdx.x + u * kThreads >= left)
        raw[u] = make_uint4(none, none, none, none);
    join<T>(a, raw, v, c, [&](float) {
      asm volatile("cp.async.commit_group;" ::: "memory");
    });
    ring.at = ring.behind(ring.at);
  }
  if (part.odd >= 0) {
    const float x = clean<T>(to_float(part.x[part.odd]));
    a.next = max_of(a.next, min_of(x, a.max));
    // in front of every vector, or behind them
    if (!at_least(a.max, x) ||
        (at_least(x, a.max) && part.odd < part.head && x > -INFINITY)) {
      a.max = x;
      a.vec = -1;
    }
    if (x > -INFINITY) {
      if (!((x - a.ref) * c <= kRebase)) rebase(a, x, c);
      const float t =
          fmaxf(fmaf(x - a.ref, c, delta_of(a.ref, c)), -kLow);
      const float e = ex2(t);
      a.s += e;
      a.h = fmaf(e, t, a.h);
    }
  }
  return a;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = max_of(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// How many of the n keys beat `mine` (behind the last stands a 0).
__device__ __forceinline__ int rank_in(const u64* keys, int n, u64 mine) {
  int r = 0;
#pragma unroll 4
  for (int k = 0; k < n; k += 2) {
    const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(keys + k);
    r += (two.x > mine) + (two.y > mine);
  }
  return r;
}

__device__ __forceinline__ void warp_sum(float& s, float& h) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    h += __shfl_xor_sync(0xffffffffu, h, o);
  }
}

// The CTA's best `top` tokens into sh.top (0 behind the last finite one).
// Called by the whole CTA; ends with a barrier.
template <typename T>
__device__ void select(Shared& sh, const Part<T>& part, const Sums& a,
                       int top) {
  constexpr int kN = Vec<T>::kN;
  const int tid = threadIdx.x, lane = tid & 31;
  // a bound: the top-th largest of 32 groups' maxima
  const uint32_t group = order_of(sh.max[lane]);
  int ahead = 0;
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const uint32_t other = __shfl_sync(0xffffffffu, group, k);
    ahead += other > group || (other == group && k < lane);
  }
  const unsigned last_group = __ballot_sync(0xffffffffu, ahead == top - 1);
  const uint32_t low = __shfl_sync(0xffffffffu, group, __ffs(last_group) - 1);
  // the threads at or above it, in any order, and their vectors
  const bool in = order_of(a.max) >= low && a.max > -INFINITY;
  uint4 raw = make_uint4(0u, 0u, 0u, 0u);
  if (in && a.vec >= 0) raw = __ldg(part.vec(a.vec));
  const u64 mine =
      in ? key_of(a.max, a.vec < 0 ? part.odd : part.head + a.vec * kN) : 0;
  const unsigned who = __ballot_sync(0xffffffffu, in);
  if (who) {
    int at = 0;
    if (lane == 0) at = atomicAdd(&sh.listed, __popc(who));
    at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1));
    if (in) sh.list[at] = mine;
  }
  __syncthreads();
  const int n = sh.listed;
  if (tid == 0) sh.list[n] = 0;
  if (n & 1) __syncthreads();  // uniform
  int rank = top;
  if (in) {
    rank = rank_in(sh.list, n, mine);
    if (rank == top - 1) sh.bound = mine;
  }
  __syncthreads();
  // the last winner's value: what lies below it is no candidate
  const float bound =
      n >= top ? max_of(value_of(sh.bound), -kMaxFinite) : -kMaxFinite;
  if (rank < top) {
    if (at_least(a.next, bound)) {
      const int at = atomicAdd(&sh.deep, 1);
      sh.deep_t[at] = (uint16_t)tid;
      sh.deep_r[at] = (uint16_t)rank;
    } else if (a.vec < 0) {
      sh.cands[atomicAdd(&sh.found, 1)] = mine;
    } else {
      float x[kN];
      widen(raw, x, static_cast<T*>(nullptr));
#pragma unroll
      for (int k = 0; k < kN; ++k)
        if (at_least(x[k], bound))
          sh.cands[atomicAdd(&sh.found, 1)] =
              key_of(clean<T>(x[k]), part.head + a.vec * kN + k);
    }
  }
  __syncthreads();
  const int deep = sh.deep;
  // a warp each
  for (int d = tid >> 5; d < deep; d += kWarps) {
    const int t = sh.deep_t[d], r = sh.deep_r[d];
    // this lane's vectors of the thread, every 32nd, a bit for each value that
    // is a candidate
    constexpr int kStride = 32 * kThreads;
    const int v0 = part.begin + t + lane * kThreads;
    static_assert(kLogprobMaxVocab / kThreads / 32 <= 64, "");
    u64 hit = 0;
    int bit = 0;
    for (int v = v0; v < part.end; v += 4 * kStride) {
      uint4 raw[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
        raw[q] = make_uint4(none, none, none, none);
        if (v + q * kStride < part.end) raw[q] = __ldg(part.vec(v + q * kStride));
      }
      uint32_t bits = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float x[kN];
        widen(raw[q], x, static_cast<T*>(nullptr));
#pragma unroll
        for (int k = 0; k < kN; ++k)
          if (at_least(x[k], bound)) bits |= 1u << (q * kN + k);
      }
      hit |= (u64)bits << bit;
      bit += 4 * kN;
    }
    const int odd = part.odd_of(t);
    const float odd_x =
        lane == 31 && odd >= 0 ? clean<T>(to_float(part.x[odd])) : -INFINITY;
    const bool odd_hit = at_least(odd_x, bound);
    int hits = __popcll(hit) + odd_hit;
#pragma unroll
    for (int o = 16; o; o >>= 1) hits += __shfl_xor_sync(0xffffffffu, hits, o);
    // the key of the value at a bit
    auto key_at = [&](int b) {
      const int place = part.head + (v0 + b / kN * kStride) * kN + b % kN;
      return key_of(clean<T>(to_float(part.x[place])), place);
    };
    if (hits <= top - r) {
      if (odd_hit) sh.cands[atomicAdd(&sh.found, 1)] = key_of(odd_x, odd);
      for (; hit; hit &= hit - 1)
        sh.cands[atomicAdd(&sh.found, 1)] = key_at(__ffsll(hit) - 1);
    } else {
      // many equals, or many large values: the first top - r of them
      u64 last = ~0ull;
      for (int n_left = top - r; n_left; --n_left) {
        u64 best = odd_hit ? key_of(odd_x, odd) : 0;
        if (best >= last) best = 0;
        for (u64 h = hit; h; h &= h - 1) {
          const u64 key = key_at(__ffsll(h) - 1);
          if (key < last && key > best) best = key;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          const u64 other = __shfl_xor_sync(0xffffffffu, best, o);
          best = other > best ? other : best;
        }
        last = best;
        if (lane == 0) sh.cands[atomicAdd(&sh.found, 1)] = best;
      }
    }
  }
  if (deep) __syncthreads();  // uniform
  const int found = sh.found;
  if (tid == 0) sh.cands[found] = 0;
  if (found & 1) __syncthreads();
  for (int j = tid; j < found; j += kThreads) {
    const u64 key = sh.cands[j];
    const int r = rank_in(sh.cands, found, key);
    if (r < top) sh.top[r] = key;
  }
  __syncthreads();
}

// Natural logarithm of S >= 1 (below 2^24), within 2^-22 of itself: S = m 2^e with m
// within a factor sqrt(2) of 1, ln m = 2 artanh((m - 1) / (m + 1)).
__device__ __forceinline__ float ln_of(float S) {
  int e = (int)((__float_as_uint(S) - 0x3f3504f3u) >> 23);
  const float m = __uint_as_float(__float_as_uint(S) - ((uint32_t)e << 23));
  const float z = __fdiv_rn(m - 1.f, m + 1.f), z2 = z * z;
  float p = fmaf(z2, 1.f / 11.f, 1.f / 9.f);
  p = fmaf(p, z2, 1.f / 7.f);
  p = fmaf(p, z2, 1.f / 5.f);
  p = fmaf(p, z2, 1.f / 3.f);
  const float lm = fmaf(2.f * z, p * z2, 2.f * z);
  return fmaf((float)e, 0.693147180559945f, lm);
}

// A row's inputs.
struct Row {
  float temp, c;
  int token;
  bool live, one;  // one: all the mass on the first of the largest
};
__device__ __forceinline__ Row row_of(const LogprobParams& p, int row) {
  Row r;
  r.token = p.token ? p.token[row] : 0;
  r.temp = p.temperature ? p.temperature[row] : 1.f;
  // by the bits: comparisons take subnormal numbers of either sign as zero
  const uint32_t bits = __float_as_uint(r.temp);
  r.one = bits << 1 == 0;
  r.live = r.token >= 0 && r.token < p.vocab && (bits < 0x7f800000u || r.one);
  // With temperatures inside these bounds 1 / T lies in fp32's range, and
  // logits of T's size are not among the numbers that are flushed.
  r.temp = fminf(fmaxf(r.temp, kTempMin), kTempMax);
  r.c = r.one ? 1.f : __fdiv_rn(1.4426950408889634f, r.temp);
  return r;
}
__device__ __forceinline__ int top_of(const LogprobParams& p, const Row& r) {
  return r.one ? max(p.top, 1) : p.top;
}

// The outputs of a row with largest logit m, sums s and h and its best tokens
// in `top`.  Called by one warp.
template <typename T>
__device__ __forceinline__ void finish(const LogprobParams& p, int row,
                                       const Row& r, float m, float s, float h,
                                       const u64* top) {
  const int lane = threadIdx.x & 31;
  const bool none = m == -INFINITY;  // no finite logit
  // S >= 1, though its roundings may fall short of that: no log p above zero
  const float lns = none ? 0.f : fmaxf(ln_of(s), 0.f);
  auto logprob = [&](float v, bool first) {
    if (r.one) return first ? 0.f : -INFINITY;
    if (none || v == -INFINITY) return -INFINITY;
    return __fdiv_rn(v - m, r.temp) - lns;
  };
  const u64 first = top_of(p, r) ? top[0] : 0;
  if (lane == 0) {
    if (p.logprob) {
      const T* x = static_cast<const T*>(p.logits) + row * p.row_stride;
      p.logprob[row] = logprob(clean<T>(to_float(x[r.token])),
                               first && r.token == place_of(first));
    }
    if (p.entropy)
      p.entropy[row] = r.one || none
                           ? 0.f
                           : fmaxf(fmaf(__fdiv_rn(h, s), -0.693147180559945f,
                                        lns),
                                   0.f);
  }
  if (lane < p.top) {
    const long long out = (long long)row * p.top + lane;
    const u64 key = top[lane];
    p.top_ids[out] = key ? place_of(key) : -1;
    p.top_logprobs[out] = key ? logprob(value_of(key), lane == 0) : -INFINITY;
  }
}

__device__ __forceinline__ void finish_idle(const LogprobParams& p, int row) {
  const int tid = threadIdx.x;
  if (tid == 0 && p.logprob) p.logprob[row] = 0.f;
  if (tid == 0 && p.entropy) p.entropy[row] = 0.f;
  if (tid < p.top) {
    p.top_ids[(long long)row * p.top + tid] = -1;
    p.top_logprobs[(long long)row * p.top + tid] = -INFINITY;
  }
}

// A part of a row: its largest logit, sums (in warp 0) and best tokens (sh.top).
// Called by the whole CTA.
template <typename T>
__device__ __forceinline__ void work_on(Shared& sh, Ring& ring,
                                        const Part<T>& part, float c, int top,
                                        float& m, float& s, float& h) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Sums a = stream(part, ring, c);
  float gm = a.max;
#pragma unroll
  for (int o = kGroup / 2; o; o >>= 1)
    gm = max_of(gm, __shfl_xor_sync(0xffffffffu, gm, o));
  if (threadIdx.x % kGroup == 0) sh.max[threadIdx.x / kGroup] = gm;
  if (threadIdx.x == 0) sh.listed = sh.found = sh.deep = 0;
  if (threadIdx.x < kTop) sh.top[threadIdx.x] = 0;
  __syncthreads();
  m = warp_max(sh.max[lane]);
  s = h = 0.f;
  if (a.ref > -INFINITY) {
    const float d = fmaxf(fmaf(a.ref - m, c, -delta_of(a.ref, c)), -kLow);
    const float k = ex2(d);
    s = a.s * k;
    h = fmaf(d, s, a.h * k);
  }
  warp_sum(s, h);
  if (lane == 0) {
    sh.s[w] = s;
    sh.h[w] = h;
  }
  __syncthreads();
  if (w == 0) {
    s = lane < kWarps ? sh.s[lane] : 0.f;
    h = lane < kWarps ? sh.h[lane] : 0.f;
    warp_sum(s, h);
  }
  if (top) select(sh, part, a, top);
}

template <typename T>
__device__ __forceinline__ const T* row_at(const LogprobParams& p, int row) {
  return static_cast<const T*>(p.logits) + row * p.row_stride;
}

// A row a CTA.
template <typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    logprobs_rows_kernel(const LogprobParams p) {
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ Shared sh;
  const int row = blockIdx.x;
  const Row r = row_of(p, row);
  if (!r.live) return finish_idle(p, row);
  Ring ring(ring_smem);
  const Part<T> part(row_at<T>(p, row), p.vocab, 0, 1);
  ring.start(part);
  float m, s, h;
  work_on(sh, ring, part, r.c, top_of(p, r), m, s, h);
  if (threadIdx.x < 32) finish<T>(p, row, r, m, s, h, sh.top);
}

// The best `top` of `n` keys that beat or equal `low` (0 is none) into sh.top.
// Called by the whole CTA; ends with a barrier.
__device__ __forceinline__ void join_tops(Shared& sh, const u64* keys, int n,
                                          int top, u64 low) {
  static_assert(kMaxCluster * kTop <= kCands, "all of them may be as good");
  const int tid = threadIdx.x;
  if (tid == 0) sh.found = 0;
  if (tid < kTop) sh.top[tid] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const u64 k = keys[i];
    if (k && k >= low) sh.cands[atomicAdd(&sh.found, 1)] = k;
  }
  __syncthreads();
  const int found = sh.found;
  if (tid == 0) sh.cands[found] = 0;
  __syncthreads();
  for (int i = tid; i < found; i += kThreads) {
    const u64 k = sh.cands[i];
    const int at = rank_in(sh.cands, found, k);
    if (at < top) sh.top[at] = k;
  }
  __syncthreads();
}

// A cluster a row, joined through distributed shared memory.
template <typename V>
__device__ __forceinline__ void store_first(V* p, V v) {
  const uint32_t at = tc::map_to(tc::smem_u32(p), 0);
  if constexpr (sizeof(V) == 8)
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
  else
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    logprobs_cluster_kernel(const LogprobParams p, int csize) {
  extern __shared__ __align__(16) uint8_t ring_smem[];
  __shared__ Shared sh;
  __shared__ float c_max[kMaxCluster], c_s[kMaxCluster], c_h[kMaxCluster];
  u64* c_top = reinterpret_cast<u64*>(ring_smem + kRingBytes);  // [csize, top]
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / csize, rank = blockIdx.x - row * csize;
  const Part<T> part(row_at<T>(p, row), p.vocab, rank, csize);
  Ring ring(ring_smem);
  const Row r = row_of(p, row);
  if (!r.live) {  // the whole cluster
    if (rank == 0) finish_idle(p, row);
    return;
  }
  ring.start(part);
  cluster_arrive();  // started
  const int top = top_of(p, r);
  float m, s, h;
  work_on(sh, ring, part, r.c, top, m, s, h);
  cluster_wait();  // every CTA has started
  if (tid == 0) {
    store_first(&c_max[rank], m);
    store_first(&c_s[rank], s);
    store_first(&c_h[rank], h);
  }
  if (tid < top) store_first(&c_top[rank * top + tid], sh.top[tid]);
  cluster_arrive();
  if (rank) return;
  cluster_wait();
  const float pm = lane < csize ? c_max[lane] : -INFINITY;
  m = warp_max(pm);
  s = h = 0.f;
  if (pm > -INFINITY) {
    const float d = fmaxf((pm - m) * r.c, -kLow), k = ex2(d);
    s = c_s[lane] * k;
    h = fmaf(d, s, c_h[lane] * k);
  }
  warp_sum(s, h);
  if (top) {
    // no CTA's last place is above the row's
    u64 last = lane < csize ? c_top[lane * top + top - 1] : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const u64 other = __shfl_xor_sync(0xffffffffu, last, o);
      last = other > last ? other : last;
    }
    join_tops(sh, c_top, csize * top, top, last);
  }
  if (w == 0) finish<T>(p, row, r, m, s, h, sh.top);
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
    const auto smem = cudaFuncAttributeMaxDynamicSharedMemorySize;
    e = cudaFuncSetAttribute(logprobs_rows_kernel<T>, smem, kRingBytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(logprobs_cluster_kernel<T>, smem,
                               kRingBytes + kMaxCluster * kTop * (int)sizeof(u64));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(logprobs_cluster_kernel<T>,
                               cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  if (csize == 1) {
    logprobs_rows_kernel<T><<<p.rows, kThreads, kRingBytes, s>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.rows * csize));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kRingBytes + csize * max(p.top, 1) * sizeof(u64);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = csize;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, logprobs_cluster_kernel<T>, p, csize);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams& p, bool bf16, int sms,
                            cudaStream_t s) {
  int csize = 1;
  while (csize < kMaxCluster && 2ll * csize * p.rows <= kClusterCtas * sms &&
         2 * csize * kSlice <= p.vocab)
    csize *= 2;
  return bf16 ? launch<__nv_bfloat16>(p, csize, s) : launch<float>(p, csize, s);
}

}  // namespace specv
