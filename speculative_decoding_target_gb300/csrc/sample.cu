// The next token from logits with temperature, top-k, top-p and min-p and a
// given uniform, and the distribution that it was drawn from.
//
// With M the row's largest logit and w(v) = 2^(-(M - x_v) log2(e) / T), tokens
// in the order (x descending, id ascending) keep a prefix: the first k (top-k),
// of those the ones before which less than p of their mass lies (top-p), of
// those the ones with w >= m (min-p).  The token is the smallest id whose
// running sum of kept weights, in id order, exceeds u times their sum.
//
// A token is an integer, decided by comparing sums of up to half a million
// weights, so the weights are integers too: w rounded to a multiple of 2^-43
// of the largest (weight_of below).  Integer sums are the same in any order,
// so histograms, reductions and scans need no fixed order to be repeatable,
// and a row's total stays below 2^63.
//
// One cluster of CTAs holds a row in shared memory (a row is read from HBM
// once; several clusters per GPC overlap one row's loads with another's
// passes) and exchanges through distributed shared memory:
//   1. load, largest and smallest logit            one exchange
//   2. per active cut (top-k by count, then top-p by mass), rounds of a
//      512-bin histogram over the candidates, reduced over the cluster and
//      scanned; the bin that holds the border is the next round's range.
//      The first round's bins divide the logits evenly, the next ones the
//      ordered bit patterns (a border is found exactly in at most five
//      rounds, and two or three on real rows)       two exchanges a round
//   3. kept mass per CTA in id order, the CTA, thread and token that hold
//      u W; kept tokens' probabilities              one exchange
#include <cuda_bf16.h>

#include <atomic>

#include "common.cuh"
#include "pair_ptx.cuh"
#include "sample.cuh"

namespace specv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kThreads;       // a thread scans one bin
constexpr int kMaxCluster = 16;
constexpr float kMaxFinite = 3.402823466e+38f;
constexpr uint64_t kOne = 1ull << 43;  // the largest token's weight

typedef unsigned long long u64;

// ---- distributed shared memory ----------------------------------------------
__device__ __forceinline__ u64 peer_load64(const void* p, uint32_t rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];"
               : "=l"(v)
               : "r"(tc::map_to(tc::smem_u32(p), rank))
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t peer_load32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];"
               : "=r"(v)
               : "r"(tc::map_to(tc::smem_u32(p), rank))
               : "memory");
  return v;
}
__device__ __forceinline__ void peer_store64(void* p, uint32_t rank, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(
                   tc::map_to(tc::smem_u32(p), rank)),
               "l"(v)
               : "memory");
}
__device__ __forceinline__ void peer_store32(void* p, uint32_t rank,
                                             uint32_t v) {
  tc::store_cluster(tc::map_to(tc::smem_u32(p), rank), v);
}

// ---- values and their order -------------------------------------------------
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
// NaN counts as -inf, +inf as the largest finite value, -0 as +0.
__device__ __forceinline__ float clean(float x) {
  return x == x ? fminf(x, kMaxFinite) + 0.f : -INFINITY;
}
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// ---- weights ----------------------------------------------------------------
// 2^-(j/32) for j < 32: as an integer multiple of 2^-50 and as two floats.
struct Table {
  u64 fix;
  float hi, lo;
};

struct Row {
  float m;         // largest logit
  float kh, kl;    // log2(e) / T as two floats
};

// round(2^43 2^-y), y = (M - x) log2(e) / T, to about 2^-46 of the largest
// weight.  The difference and the product are carried as two floats; with
// y = n + j/32 + r, |r| <= 1/64, the factor 2^-r = e^t, t = -r ln 2, is
// 1 + t + t^2/2 in two floats and t^3 (1/6 + t/24 + t^2/120) in one (the next
// term is below 2^-48), times the table's 2^-(j/32), as an integer multiple
// of 2^-50 that is shifted by n.  Weights below 2^-28 take exp2 itself: its
// relative error of 2^-22 is below the integers' step there.
__device__ __forceinline__ u64 weight_of(const Row& r, float x,
                                         const Table* tab) {
  const float dh = __fsub_rn(r.m, x);
  const float yh = __fmul_rn(dh, r.kh);
  if (yh > 28.f)
    return yh > 45.f ? 0ull : (u64)__float2uint_rn(exp2f(__fsub_rn(43.f, yh)));
  const float b = __fsub_rn(dh, r.m);
  const float dl = __fsub_rn(__fsub_rn(r.m, __fsub_rn(dh, b)), __fadd_rn(x, b));
  float yl = __fmaf_rn(dh, r.kh, -yh);
  yl = __fmaf_rn(dh, r.kl, yl);
  yl = __fmaf_rn(dl, r.kh, yl);
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
  const float nt = __fmaf_rn(yh, 32.f, kMagic);
  const int ni = __float_as_int(nt) - 0x4B400000;
  const float rh = __fmaf_rn(__fsub_rn(nt, kMagic), -0.03125f, yh);
  constexpr float kLn2H = 0.693147182464599609375f;      // ln 2 in fp32
  constexpr float kLn2L = -1.904654299957767e-09f;       // and the rest
  const float th = __fmul_rn(rh, -kLn2H);
  float tl = __fmaf_rn(rh, -kLn2H, -th);
  tl = __fmaf_rn(rh, -kLn2L, tl);
  tl = __fmaf_rn(yl, -kLn2H, tl);
  const float hh = __fmul_rn(0.5f, th);
  const float sh = __fmul_rn(th, hh);
  float sl = __fmaf_rn(th, hh, -sh);
  sl = __fmaf_rn(th, tl, sl);
  float c = __fmaf_rn(th, 8.333333768e-3f, 4.166666791e-2f);
  c = __fmaf_rn(th, c, 1.666666716e-1f);
  const float cube = __fmul_rn(__fmul_rn(c, th), __fadd_rn(sh, sh));
  const float qh = __fadd_rn(th, sh);
  const float ql = __fadd_rn(__fadd_rn(__fsub_rn(th, qh), sh),
                             __fadd_rn(__fadd_rn(tl, sl), cube));
  const Table t = tab[ni & 31];
  const float g = __fmul_rn(t.hi, qh);
  float gl = __fmaf_rn(t.hi, qh, -g);
  gl = __fmaf_rn(t.hi, ql, gl);
  gl = __fmaf_rn(t.lo, qh, gl);
  const float i1t = __fmaf_rn(g, 67108864.f, kMagic);  // 2^26
  const int i1 = __float_as_int(i1t) - 0x4B400000;
  const float rem = __fadd_rn(
      __fmaf_rn(__fsub_rn(i1t, kMagic), -1.490116119384765625e-08f, g), gl);
  const int i2 = __float2int_rn(__fmul_rn(rem, 1125899906842624.f));  // 2^50
  const long long e =
      (long long)t.fix + ((long long)i1 << 24) + (long long)i2;
  const int n = ni >> 5;
  // y may round to just below zero steps; the largest token has y = 0
  return (u64)(e + (64ll << n)) >> (7 + n);
}

// ---- block and cluster steps ------------------------------------------------
struct Shared {
  Table tab[32];
  u64 hist_m[kBins], red_m[kBins];
  uint32_t hist_c[kBins], red_c[kBins];
  u64 warp_m[kWarps];
  uint32_t warp_c[kWarps];
  u64 x_m[2];         // exchanged: this CTA's value, one buffer per use
  uint32_t x_c[2];
  u64 before_m;       // the border bin and what lies before it
  uint32_t before_c, bin;
  uint32_t lo, hi;    // its range of order distances
  int eq_last;
};

__device__ __forceinline__ u64 shfl_up64(u64 v, int o) {
  return __shfl_up_sync(0xffffffffu, v, o);
}

// Exclusive prefix over the block (thread order) of a mass and a count.
__device__ __forceinline__ void block_scan(Shared& s, u64 m, uint32_t c,
                                           u64* em, uint32_t* ec, u64* tm,
                                           uint32_t* tcnt) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 im = m;
  uint32_t ic = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 a = shfl_up64(im, o);
    const uint32_t b = __shfl_up_sync(0xffffffffu, ic, o);
    if (lane >= o) {
      im += a;
      ic += b;
    }
  }
  __syncthreads();
  if (lane == 31) {
    s.warp_m[warp] = im;
    s.warp_c[warp] = ic;
  }
  __syncthreads();
  u64 bm = 0, allm = 0;
  uint32_t bc = 0, allc = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const u64 a = s.warp_m[w];
    const uint32_t b = s.warp_c[w];
    if (w < warp) {
      bm += a;
      bc += b;
    }
    allm += a;
    allc += b;
  }
  *em = bm + im - m;
  *ec = bc + ic - c;
  *tm = allm;
  *tcnt = allc;
}

// The cluster's histogram from the CTAs' own, in every CTA: thread (bin,
// source) of the CTA's slice of bins reads one value, the sources of a bin are
// summed by shuffles, and each of those lanes stores the sum to one CTA.
__device__ __forceinline__ void reduce_bins(Shared& s, uint32_t rank, int csize) {
  __syncthreads();
  tc::cluster_sync();
  const int tid = threadIdx.x;
  const int bin = (int)rank * (kBins / csize) + tid / csize, src = tid % csize;
  u64 m = peer_load64(&s.hist_m[bin], src);
  uint32_t c = peer_load32(&s.hist_c[bin], src);
  for (int o = 1; o < csize; o <<= 1) {
    m += __shfl_xor_sync(0xffffffffu, m, o);
    c += __shfl_xor_sync(0xffffffffu, c, o);
  }
  peer_store64(&s.red_m[bin], src, m);
  peer_store32(&s.red_c[bin], src, c);
  tc::cluster_sync();
}

struct Cut {
  uint32_t dk;     // order distance of the border value
  uint32_t count;  // how many tokens of that value are kept, lowest ids first
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
    sample_kernel(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t s_raw[];
  __shared__ Shared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = tc::cluster_rank();
  int csize;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(csize));
  const int row = blockIdx.x / csize;
  const int base = (int)rank * p.chunk;
  const int n = max(0, min(p.chunk, p.vocab - base));

  // 1. the chunk into shared memory, at its own offset within 16 bytes, so
  // that whole vectors are copied whatever the row's alignment
  const T* src = static_cast<const T*>(p.logits) + row * p.row_stride + base;
  constexpr int kE = 16 / sizeof(T);
  const int off = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
  T* xs = reinterpret_cast<T*>(s_raw) + off;
  {
    const int head = min(n, (kE - off) % kE);
    const int nv = (n - head) / kE;
    for (int v = tid; v < nv; v += kThreads)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                       tc::smem_u32(xs + head + v * kE)),
                   "l"(src + head + v * kE)
                   : "memory");
    if (tid < head) xs[tid] = src[tid];
    const int tail = head + nv * kE + tid;
    if (tail < n) xs[tail] = src[tail];
  }
  float T0 = p.temperature ? p.temperature[row] : 1.f;
  const float u = p.u[row];
  int k = p.top_k ? p.top_k[row] : 0;
  const float tp = p.top_p ? p.top_p[row] : 1.f;
  const float mp = p.min_p ? p.min_p[row] : 0.f;
  const bool idle = !(T0 >= 0.f);
  if (k <= 0 || k >= p.vocab) k = 0;
  // cuts that leave the first token alone
  const bool one = T0 == 0.f || k == 1 || tp <= 0.f || mp > 1.f;
  if (tid < 32) {
    const double e = exp2(-tid / 32.0);
    Table t;
    t.fix = (u64)__double2ll_rn(e * 1125899906842624.0);
    t.hi = (float)e;
    t.lo = (float)(e - t.hi);
    s.tab[tid] = t;
  }
  s.hist_m[tid] = 0;
  s.hist_c[tid] = 0;
  if (tid == 0) s.eq_last = -1;
  asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
  __syncthreads();

  // the largest logit with its lowest id, and the smallest finite one
  u64 best = 0;
  uint32_t low = 0xffffffffu;
  for (int i = tid; i < n; i += kThreads) {
    const float x = clean(as_float(xs[i]));
    const uint32_t key = key_of(x);
    const u64 v = (u64)key << 32 | (uint32_t)~(uint32_t)(base + i);
    best = v > best ? v : best;
    if (x > -INFINITY) low = min(low, key);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const u64 v = __shfl_xor_sync(0xffffffffu, best, o);
    best = v > best ? v : best;
  }
  low = __reduce_min_sync(0xffffffffu, low);
  if (lane == 0) {
    s.warp_m[warp] = best;
    s.warp_c[warp] = low;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kWarps; ++w) {
      best = s.warp_m[w] > best ? s.warp_m[w] : best;
      low = min(low, s.warp_c[w]);
    }
    s.x_m[0] = best;
    s.x_c[0] = low;
  }
  __syncthreads();
  tc::cluster_sync();
  best = 0;
  low = 0xffffffffu;
  for (int j = 0; j < csize; ++j) {
    const u64 v = peer_load64(&s.x_m[0], j);
    best = v > best ? v : best;
    low = min(low, peer_load32(&s.x_c[0], j));
  }
  const uint32_t mkey = (uint32_t)(best >> 32);
  const int arg = (int)~(uint32_t)best;
  Row r;
  r.m = value_of(mkey);
  const bool none = idle || !(r.m > -INFINITY);

  Cut cut{0xffffffffu, 0u};  // everything
  u64 total = 0;
  int eq_last = -1;          // last kept id (in the chunk) of the border value
  u64 minw = 0;
  if (!none && !one) {
    // log2(e) / T, kept finite and above zero so that 0 k = 0, inf k = inf
    double kd = 1.4426950408889634074 / (double)T0;
    kd = kd > 1e38 ? 1e38 : (kd < 1e-37 ? 1e-37 : kd);
    r.kh = (float)kd;
    r.kl = (float)(kd - r.kh);
    if (mp > 0.f) minw = (u64)ceil((double)mp * (double)kOne);

    // 2. the cuts
    const bool by_p = tp < 1.f;
    // the first round's bins: even steps of the logit over what has weight
    const float span = fminf(__fsub_rn(r.m, value_of(low)), 45.f / r.kh);
    const float step = span > 0.f ? fminf((kBins - 1) / span, kMaxFinite) : 0.f;
    auto bin_of = [&](float x) {
      const float f = __fmul_rn(__fsub_rn(r.m, x), step);
      return f < kBins - 1 ? (uint32_t)f : kBins - 1u;  // NaN: the last
    };
    for (int which = 0; which < 2; ++which) {  // top-k, then top-p
      if (which == 0 ? k == 0 : !by_p) continue;
      const bool mass = which == 1;
      const Cut old = cut;
      u64 want = mass ? 0 : (u64)k;  // the border is where the sum reaches it
      u64 above = 0;
      uint32_t lo = 0, hi = 0xffffffffu;
      for (int round = 0;; ++round) {
        const int shift = max(0, 32 - __clz((int)(hi - lo)) - 9);
        auto digit = [&](uint32_t dk, float x) {
          return round == 0 ? bin_of(x) : (dk - lo) >> shift;
        };
        for (int i = tid; i < n; i += kThreads) {
          const float x = clean(as_float(xs[i]));
          const uint32_t dk = mkey - key_of(x);
          if (dk < lo || dk > hi || dk >= old.dk) continue;
          const uint32_t d = digit(dk, x);
          if (mass) {
            const u64 w = weight_of(r, x, s.tab);
            if (w) atomicAdd(&s.hist_m[d], w);
          } else {
            atomicAdd(&s.hist_c[d], 1u);
          }
        }
        if (mass && rank == 0 && tid == 0 && old.count && old.dk >= lo &&
            old.dk <= hi) {
          // the kept part of the top-k border, as one lump
          const float x = value_of(mkey - old.dk);
          atomicAdd(&s.hist_m[digit(old.dk, x)],
                    old.count * weight_of(r, x, s.tab));
        }
        reduce_bins(s, rank, csize);
        s.hist_m[tid] = 0;
        s.hist_c[tid] = 0;
        const u64 v = mass ? s.red_m[tid] : (u64)s.red_c[tid];
        u64 ex, all;
        uint32_t ec, ac;
        block_scan(s, v, 0u, &ex, &ec, &all, &ac);
        if (round == 0) {
          if (mass) {  // sums before a kept token are below p W
            const double t = ceil((double)tp * (double)all);
            want = t < 1.0 ? 1ull : (u64)t;
            want = want > all ? all : want;
          } else if (want > all) {
            break;  // fewer tokens than k: uniform, every thread has all
          }
        }
        if (tid == 0) s.bin = kBins;
        __syncthreads();
        if (above + ex < want && want <= above + ex + v) {
          s.bin = tid;
          s.before_m = above + ex;
        }
        __syncthreads();
        const uint32_t b = s.bin;
        if (b == kBins) break;  // no mass left: cannot be reached
        above = s.before_m;
        if (round == 0) {
          // the range of order distances that falls into bin b: the digit
          // does not decrease with the distance
          if (tid < 2) {
            uint32_t a = 0, z = 0xffffffffu;  // first distance with digit >= g
            const uint32_t g = b + tid;
            if (g < kBins) {
              while (a < z) {
                const uint32_t mid = a + ((z - a) >> 1);
                // below the smallest value every pattern belongs to the last
                const bool in = mid <= mkey - low &&
                                bin_of(value_of(mkey - mid)) < g;
                if (in) a = mid + 1; else z = mid;
              }
              if (tid == 0) s.lo = a; else s.hi = a - 1;
            } else {
              s.hi = mkey - low;
            }
          }
          __syncthreads();
          lo = s.lo;
          hi = s.hi;
        } else {
          const u64 end = lo + ((u64)(b + 1) << shift) - 1;
          hi = end < hi ? (uint32_t)end : hi;
          lo += b << shift;
        }
        if (lo >= hi) {
          cut.dk = lo;
          if (mass) {
            const u64 w = weight_of(r, value_of(mkey - lo), s.tab);
            cut.count = (uint32_t)((want - above + w - 1) / w);
          } else {
            cut.count = (uint32_t)(want - above);
          }
          break;
        }
        __syncthreads();
      }
      __syncthreads();
    }

    // 3. kept mass, each thread its segment of ids
    const u64 weq =
        cut.count ? weight_of(r, value_of(mkey - cut.dk), s.tab) : 0;
    const uint32_t keep_eq = weq >= minw ? cut.count : 0;
    u64 m = 0;
    uint32_t eq = 0;
    const int i0 = tid * p.seg, i1 = min(n, i0 + p.seg);
    for (int i = i0; i < i1; ++i) {
      const float x = clean(as_float(xs[i]));
      const uint32_t dk = mkey - key_of(x);
      if (dk < cut.dk) {
        const u64 w = weight_of(r, x, s.tab);
        m += w >= minw ? w : 0;
      } else if (dk == cut.dk) {
        ++eq;
      }
    }
    u64 em, am;
    uint32_t ec, ac;
    block_scan(s, m, eq, &em, &ec, &am, &ac);
    if (tid == 0) {
      s.x_m[1] = am;
      s.x_c[1] = ac;
    }
    __syncthreads();
    tc::cluster_sync();
    u64 mine = 0, at = 0;     // kept mass before this CTA and in it
    uint32_t eq_at = 0, eq_before = 0;
    for (int j = 0; j < csize; ++j) {
      const u64 cm = peer_load64(&s.x_m[1], j);
      const uint32_t cc = peer_load32(&s.x_c[1], j);
      const uint32_t kept = min(cc, keep_eq - min(keep_eq, eq_at));
      const u64 w = cm + kept * weq;
      if (j < (int)rank) {
        at += w;
        eq_before += cc;
      }
      if (j == (int)rank) mine = w;
      total += w;
      eq_at += cc;
    }
    u64 t = 0;
    if (u > 0.f) {
      t = (u64)fmin(floor((double)u * (double)total), 9.2e18);
      t = t >= total ? total - 1 : t;
    }
    // kept tokens of the border value before this thread, and its share
    const uint32_t eb = eq_before + ec;
    const uint32_t room = keep_eq - min(keep_eq, eb);
    const uint32_t kept = min(eq, room);
    const uint32_t kept_before =
        min(keep_eq, eb) - min(keep_eq, eq_before);
    const u64 start = at + em + kept_before * weq;
    const bool here = start <= t && t < start + m + kept * weq;
    // every lane of the warp that holds the draw takes a token of that
    // thread's segment
    const unsigned who = __ballot_sync(0xffffffffu, here);
    if (who) {
      const int l = __ffs(who) - 1;
      const int b0 = __shfl_sync(0xffffffffu, i0, l);
      const int b1 = __shfl_sync(0xffffffffu, i1, l);
      u64 run = __shfl_sync(0xffffffffu, start, l);
      uint32_t rm = __shfl_sync(0xffffffffu, room, l);
      for (int e = b0; e < b1; e += 32) {
        const int i = e + lane;
        u64 w = 0;
        bool is_eq = false;
        if (i < b1) {
          const float x = clean(as_float(xs[i]));
          const uint32_t dk = mkey - key_of(x);
          is_eq = dk == cut.dk;
          if (dk < cut.dk) {
            w = weight_of(r, x, s.tab);
            if (w < minw) w = 0;
          }
        }
        const unsigned eqs = __ballot_sync(0xffffffffu, is_eq);
        if (is_eq && __popc(eqs & ((1u << lane) - 1)) < (int)rm) w = weq;
        rm -= min(rm, (uint32_t)__popc(eqs));
        u64 inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const u64 a = shfl_up64(inc, o);
          if (lane >= o) inc += a;
        }
        const unsigned hit =
            __ballot_sync(0xffffffffu, w > 0 && run + inc > t);
        if (hit) {
          if (lane == 0) p.token[row] = base + e + __ffs(hit) - 1;
          break;
        }
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    // the last kept id of the border value, for the distribution
    if (p.probs || p.filtered) {
      if (kept > 0 && (kept < eq || eb + eq >= keep_eq)) {
        // this thread holds the border itself
        uint32_t left = kept;
        for (int i = i0; i < i1 && left; ++i)
          if (mkey - key_of(clean(as_float(xs[i]))) == cut.dk && --left == 0)
            s.eq_last = i;
      } else if (tid == kThreads - 1 && eq_before + ac < keep_eq) {
        s.eq_last = n;  // every one in this chunk is kept
      }
      __syncthreads();
      eq_last = s.eq_last;
    }
  } else if (rank == 0 && tid == 0) {
    p.token[row] = none ? -1 : arg;
  }

  // the distribution
  if (p.probs || p.filtered) {
    const float inv = total ? (float)(8796093022208.0 / (double)total) : 0.f;
    const long long out = (long long)row * p.vocab + base;
    for (int i = tid; i < n; i += kThreads) {
      const float x = clean(as_float(xs[i]));
      bool keep = false;
      float pr = 0.f;
      if (none) {
      } else if (one) {
        keep = base + i == arg;
        pr = keep ? 1.f : 0.f;
      } else {
        const uint32_t dk = mkey - key_of(x);
        keep = x > -INFINITY &&
               (dk < cut.dk || (dk == cut.dk && i <= eq_last));
        if (keep) {
          const u64 w = weight_of(r, x, s.tab);
          keep = w >= minw;
          if (keep) {
            // below 2^-19 the integer has too few digits left for fp32
            pr = (w >> 24) ? __ull2float_rn(w) * 1.13686837721616030e-13f
                           : exp2f(-__fmul_rn(__fsub_rn(r.m, x), r.kh));
            pr *= inv;
          }
        }
      }
      if (p.probs) p.probs[out + i] = pr;
      if (p.filtered) p.filtered[out + i] = keep ? x : -INFINITY;
    }
  }
  tc::cluster_sync();  // no CTA leaves while others read its shared memory
}

template <typename T>
cudaError_t launch(const SampleParams& p, int csize, cudaStream_t s) {
  const size_t smem = (size_t)p.chunk * sizeof(T) + 32;
  // once per device (an attribute call per launch costs microseconds)
  static std::atomic<uint64_t> ready{0};
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(
        sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        kSampleMaxVocab / kMaxCluster * (int)sizeof(T) + 32);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(
          sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.rows * csize);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = csize;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, p);
}

}  // namespace

cudaError_t launch_sample(SampleParams p, bool bf16, int sms, cudaStream_t s) {
  // The smallest cluster whose CTAs hold at most 64 KB of the row, so that
  // more than one fits on an SM; with few rows, more CTAs per row while SMs
  // would stay empty and a CTA keeps a few tokens per thread.
  const size_t esz = bf16 ? 2 : 4;
  int csize = 1;
  while (csize < kMaxCluster && (size_t)p.vocab * esz > (size_t)csize * 65536)
    csize *= 2;
  while (csize < kMaxCluster && (long long)p.rows * csize * 2 <= sms &&
         p.vocab > csize * 4096)
    csize *= 2;
  p.chunk = ((p.vocab + csize - 1) / csize + 7) / 8 * 8;
  p.seg = ((p.chunk + kThreads - 1) / kThreads) | 1;
  return bf16 ? launch<__nv_bfloat16>(p, csize, s) : launch<float>(p, csize, s);
}

}  // namespace specv
