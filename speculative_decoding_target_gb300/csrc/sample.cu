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
// once; clusters share the SMs, so one row's loads overlap another's passes)
// and exchanges through distributed shared memory:
//   1. load, largest and smallest logit                      one exchange
//   2. a histogram over the cluster, 512 bins by count for top-k (for a small k
//      of the threads' own largest logits instead of all), 1,024 by mass for
//      top-p, its bins even steps of the logit: the bin with the border (two
//      exchanges).  Then, by what lies at and above that bin:
//      - at most kList tokens (any usual top-k, any nucleus of a sure model):
//        the first CTA gathers them, and makes every cut and the draw alone;
//      - more, but at most kList in the bin: it finds the border among those,
//        the next cut or step 3 follows;
//      - more than that: the bin is divided by the ordered bit patterns of
//        (logit, id), as many parts a round, until one of the two holds.
//   3. (wide kept sets) kept mass per CTA in id order, then the thread and
//      the token that hold u W                               one exchange
//
// Measured (248,320 tokens): one row with top-k and top-p 19 us, 64 fp32 rows
// with mixed settings 95 us, 224 bf16 rows (top-p over a flat row) with
// their distributions 561 us.  Rows cost instructions and latency, not bytes
// (the last reads and writes 334 MB, 49 us of the copy rate): a flat row's
// weights (about 45 packed fp32 steps a pair of tokens, made once for the bins
// and once more for what is kept) are the largest share, and a row with top-k
// waits on barriers, about 30,000 cycles from its load to its token.
#include <cuda_bf16.h>

#include <atomic>

#include "common.cuh"
#include "pair_ptx.cuh"
#include "sample.cuh"

namespace specv {
namespace {

// (1,024 where a CTA has its SM alone: 64 fp32 rows with top-k 96 us instead of
// 85, flat with top-p 231 instead of 245, one row 22 instead of 19)
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
// Bins of a round over the mass, where fewer tokens in the border's bin save
// gathers and rounds, and of one over counts, which usually ends after the
// first (224 rows of 248,320: bf16, flat, top-p 552 us with 1,024 and 591 with
// 512; fp32, top-k then top-p 331 us with 1,024 for the counts and 325 with
// 512).
constexpr int kMassBits = 10, kCountBits = 9;
constexpr int kBins = 1 << kMassBits;  // a thread scans two bins
static_assert(kBins == 2 * kThreads, "");
constexpr int kBatch = 8;             // values of a thread in flight
constexpr int kMaxCluster = 16;
constexpr int kWideRows = 7;            // rows that may take 16 CTAs each
constexpr int kMaxChunk = 32768;        // tokens of a row, in a CTA
static_assert(kSampleMaxVocab <= kMaxCluster * kMaxChunk, "");
constexpr int kPad = kBatch * kThreads;  // a CTA's values come in whole batches
// a thread's share of a warp's run in the draw (step 3)
constexpr int kPerDraw = kMaxChunk / kWarps / kThreads;
static_assert(kMaxChunk % kPad == 0 && kPerDraw * kWarps * kThreads == kMaxChunk,
              "");
constexpr float kMaxFinite = 3.402823466e+38f;

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
__device__ __forceinline__ void store_float(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_float(__nv_bfloat16* p, float x) {
  *p = __float2bfloat16_rn(x);
}
// NaN counts as -inf, +inf as the type's largest finite value, -0 as +0.
__device__ __forceinline__ float largest(float) { return kMaxFinite; }
__device__ __forceinline__ float largest(__nv_bfloat16) {
  return 3.3895313892515355e+38f;
}
__device__ __forceinline__ float clean(float x, float most) {
  return x == x ? fminf(x, most) + 0.f : -INFINITY;
}
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// ---- weights ----------------------------------------------------------------
// 1.5 * 2^23: an addition of it rounds to an integer, which the sum's low bits
// hold above the constant's.
constexpr float kMagic = 12582912.f;
constexpr uint32_t kMagicBits = 0x4B400000u;
// 2^-(j/32) for j < 32: as an integer multiple of 2^-50, less what kMagicBits
// will add to it (near_weights), and as two floats.
// One 32-bit word of every entry after the other, so that lanes with different
// j read different banks (16-byte entries took about 12 wavefronts a load).
struct Table {
  uint32_t fix_lo[32], fix_hi[32];
  float hi[32], lo[32];
};
__constant__ u64 kPowers[32] = {  // round(2^(50 - j/32))
    0x4000000000000ull, 0x3ea0ecb6dc8a8ull, 0x3d495f454921bull, 0x3bf92e66f736cull,
    0x3ab031b9f7491ull, 0x396e41b9df20dull, 0x383337bb0aa54ull, 0x36feede5f6bc9ull,
    0x35d13f32b5a76ull, 0x34aa07647c4acull, 0x3389230547e12ull, 0x326e6f619b8bdull,
    0x3159ca845541bull, 0x304b1332999c2ull, 0x2f4228e7d6031ull, 0x2e3eebd1d8beeull,
    0x2d413cccfe77aull, 0x2c48fd6074ab1ull, 0x2b560fba90a85ull, 0x2a6856ad3a9f0ull,
    0x297fb5aa6c545ull, 0x289c10c0c3126ull, 0x27bd4c9824684ull, 0x26e34e6e75539ull,
    0x260dfc14636e3ull, 0x253d3bea3fbdcull, 0x2470f4dceac47ull, 0x23a90e62d1735ull,
    0x22e57078faa2full, 0x222603a024b6aull, 0x216ab0d9f3122ull, 0x20b361a62b0afull,
};
__device__ __forceinline__ void fill_table(Table& t, int j) {
  const u64 fix = kPowers[j];
  const float hi = __fmul_rn(__ull2float_rn(fix), 8.8817841970012523e-16f);
  const u64 base = fix - ((u64)kMagicBits << 24);
  t.fix_lo[j] = (uint32_t)base;
  t.fix_hi[j] = (uint32_t)(base >> 32);
  t.hi[j] = hi;  // times 2^-50
  t.lo[j] = __fmul_rn(
      __ll2float_rn((long long)fix -
                    __float2ll_rn(__fmul_rn(hi, 1125899906842624.f))),
      8.8817841970012523e-16f);
}

struct Row {
  float m;         // largest logit
  float kh, kl;    // log2(e) / T as two floats
};

// log2(e) / T: the quotient of the leading part, then what it leaves (exact
// by fma) and the constant's own rest.  Kept finite and above zero, so that
// 0 k = 0 and inf k = inf.
__device__ __forceinline__ void set_scale(Row& r, float T) {
  constexpr float kH = 1.44269502162933349609375f, kL = 1.9259629911e-08f;
  const float q = __fdiv_rn(kH, T);
  r.kh = fminf(fmaxf(q, 1e-37f), 1e38f);
  r.kl = q == r.kh ? __fdiv_rn(__fadd_rn(__fmaf_rn(-q, T, kH), kL), T) : 0.f;
}

// floor(f W) and ceil(f W) (at least 1) for f in [0, 1), exactly: f is a
// 64-bit fraction.
__device__ __forceinline__ u64 floor_part(float f, u64 W) {
  return __umul64hi(__float2ull_rz(__fmul_rn(f, 18446744073709551616.f)), W);
}
__device__ __forceinline__ u64 ceil_part(float f, u64 W) {
  const u64 F = __float2ull_rz(__fmul_rn(f, 18446744073709551616.f));
  const u64 c = __umul64hi(F, W) + (F * W != 0 ? 1 : 0);
  return c ? c : 1;
}

// Packed fp32 steps, spelled out so that none is fused with another.
__device__ __forceinline__ u64 bits2(float2 v) {
  return (u64)__float_as_uint(v.y) << 32 | __float_as_uint(v.x);
}
__device__ __forceinline__ float2 float2_of(u64 v) {
  return make_float2(__uint_as_float((uint32_t)v),
                     __uint_as_float((uint32_t)(v >> 32)));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  u64 d;
  asm("add.rn.ftz.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  u64 d;
  asm("mul.rn.ftz.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
  return float2_of(d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  u64 d;
  asm("fma.rn.ftz.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return float2_of(d);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// The integer of 2^-50 steps from the table's entry, a multiple of 2^24 and a
// rest, rounded to 2^-43 and shifted by n / 32 at once.
__device__ __forceinline__ u64 assemble(const Table& tab, uint32_t n, float i1,
                                        float i2) {
  const int j = n & 31;
  u64 e = (u64)tab.fix_hi[j] << 32 | tab.fix_lo[j];
  asm("mad.wide.s32 %0, %1, 16777216, %0;" : "+l"(e) : "r"(__float_as_int(i1)));
  asm("mad.wide.s32 %0, %1, 1, %0;" : "+l"(e) : "r"(__float2int_rn(i2)));
  return (e >> ((n >> 5) - (kMagicBits >> 5) + 6)) + 1 >> 1;
}

// round(2^43 2^-y), y = (M - x) log2(e) / T, to about 2^-46 of the largest
// weight, of two tokens at once in packed fp32.  The difference and the product
// are carried as two floats; with y = n + j/32 + r, |r| <= 1/64, the factor
// 2^-r = e^t, t = -r ln 2, is 1 + t + t^2/2 in two floats and
// t^3 (1/6 + t/24 + t^2/120) in one, with the t^2/2 that the low part of t adds
// to it (the next term is below 2^-48), times the table's 2^-(j/32), as an
// integer multiple of 2^-50 that is shifted by n.
__device__ __forceinline__ void near_weights(const Row& r, float2 x, float2 dh,
                                             float2 yh, const Table& tab,
                                             u64& w0, u64& w1) {
  // a - b is fma(b, -1, a): packed operands carry no sign of their own
  const float2 one = both(-1.f), m = both(r.m), kh = both(r.kh);
  const float2 magic = both(kMagic), unmagic = both(-kMagic);
  // beyond 28: any value that keeps the steps finite
  const float2 yc = make_float2(fminf(yh.x, 29.f), fminf(yh.y, 29.f));
  const float2 nt = fma2(yc, both(32.f), magic);
  // what m - x and its product leave
  const float2 nb = fma2(dh, one, m);
  const float2 dl = fma2(fma2(nb, one, x), one, fma2(add2(dh, nb), one, m));
  float2 yl = fma2(dh, kh, mul2(yh, one));
  yl = fma2(dh, both(r.kl), yl);
  yl = fma2(dl, kh, yl);
  const float2 rh = fma2(add2(nt, unmagic), both(-0.03125f), yc);
  constexpr float kLn2H = 0.693147182464599609375f;      // ln 2 in fp32
  constexpr float kLn2L = -1.904654299957767e-09f;       // and the rest
  const float2 l2h = both(-kLn2H);
  const float2 th = mul2(rh, l2h);
  float2 tl = fma2(rh, l2h, mul2(th, one));
  tl = fma2(rh, both(-kLn2L), tl);
  tl = fma2(yl, l2h, tl);
  const float2 hh = mul2(both(0.5f), th);
  const float2 sh = mul2(th, hh);
  float2 sl = fma2(th, hh, mul2(sh, one));
  sl = fma2(th, tl, sl);
  float2 c = fma2(th, both(8.333333768e-3f), both(4.166666791e-2f));
  c = fma2(th, c, both(1.666666716e-1f));
  const float2 cube = fma2(sh, tl, mul2(mul2(c, th), add2(sh, sh)));
  const float2 qh = add2(th, sh);
  const float2 ql = add2(add2(fma2(qh, one, th), sh),
                         add2(add2(tl, sl), cube));
  const uint32_t n0 = __float_as_uint(nt.x), n1 = __float_as_uint(nt.y);
  const int j0 = n0 & 31, j1 = n1 & 31;
  const float2 hi = make_float2(tab.hi[j0], tab.hi[j1]);
  const float2 lo = make_float2(tab.lo[j0], tab.lo[j1]);
  const float2 g = mul2(hi, qh);
  float2 gl = fma2(hi, qh, mul2(g, one));
  gl = fma2(hi, ql, gl);
  gl = fma2(lo, qh, gl);
  const float2 i1t = fma2(g, both(67108864.f), magic);  // 2^26
  const float2 rem = add2(
      fma2(add2(i1t, unmagic), both(-1.490116119384765625e-08f), g), gl);
  const float2 i2 = mul2(rem, both(1125899906842624.f));  // 2^50
  w0 = assemble(tab, n0, i1t.x, i2.x);
  w1 = assemble(tab, n1, i1t.y, i2.y);
}

// Weights below 2^-28 take exp2 itself: its relative error of 2^-22 is below
// the integers' step there.
__device__ __forceinline__ u64 far_weight(float yh) {
  return yh > 45.f ? 0ull : (u64)__float2uint_rn(exp2f(__fsub_rn(43.f, yh)));
}

// One token; the same steps, so the same bits.
__device__ __forceinline__ u64 weight_of(const Row& r, float x,
                                         const Table& tab) {
  const float dh = __fsub_rn(r.m, x);
  const float yh = __fmul_rn(dh, r.kh);
  if (yh > 28.f) return far_weight(yh);
  u64 w0, w1;
  near_weights(r, both(x), both(dh), both(yh), tab, w0, w1);
  return w0;
}

// Two tokens, with one branch for the whole warp, which must be converged.
__device__ __forceinline__ void warp_weights(const Row& r, float2 x,
                                             const Table& tab, u64& w0,
                                             u64& w1) {
  const float2 dh = fma2(x, both(-1.f), both(r.m));
  const float2 yh = mul2(dh, both(r.kh));
  w0 = w1 = 0;
  if (__any_sync(0xffffffffu, fminf(yh.x, yh.y) <= 28.f))
    near_weights(r, x, dh, yh, tab, w0, w1);
  if (__any_sync(0xffffffffu, fmaxf(yh.x, yh.y) > 28.f)) {
    if (yh.x > 28.f) w0 = far_weight(yh.x);
    if (yh.y > 28.f) w1 = far_weight(yh.y);
  }
}

// The probability's numerator, 2^-y in fp32 (relative error 2^-22 for the
// exp2, the rounding of y made good).
__device__ __forceinline__ float fast_weight(const Row& r, float x) {
  const float dh = __fsub_rn(r.m, x);
  const float yh = __fmul_rn(dh, r.kh);
  const float b = __fsub_rn(dh, r.m);
  const float dl = __fsub_rn(__fsub_rn(r.m, __fsub_rn(dh, b)), __fadd_rn(x, b));
  float yl = __fmaf_rn(dh, r.kh, -yh);
  yl = __fmaf_rn(dh, r.kl, yl);
  yl = __fmaf_rn(dl, r.kh, yl);
  const float e = exp2f(-yh);
  return e > 0.f ? __fmaf_rn(e, -0.6931471806f * yl, e) : 0.f;
}

// ---- block and cluster steps ------------------------------------------------
constexpr int kList = 2048;      // candidates that one CTA sorts
constexpr int kPerThread = kList / kThreads;
constexpr int kRanked = 256;     // candidates that are sorted, by counting
constexpr int kIdBits = 19;      // ids of kSampleMaxVocab tokens

struct Shared {
  Table tab;
  union {
    struct {
      uint32_t hist_lo[kBins], hist_hi[kBins];  // a bin's mass
      uint32_t hist_c[kBins], red_c[kBins];     // and tokens
      u64 red_m[kBins];
    };
    u64 wts[kRanked];  // the candidates' weights by rank, once no bins are left
  };
  u64 list[kList];    // (order distance, id) of candidates
  int part[256];      // rank_entries
  u64 warp_m[kWarps];
  uint32_t warp_c[kWarps];
  u64 x_m[2];         // exchanged: this CTA's value, one per use
  uint32_t x_c;
  uint32_t n_list;
  u64 cut, total;     // broadcast by the first CTA
  u64 before_m;       // the border bin and what lies before it
  uint32_t before_c, bin, bin_c;
  uint32_t lo, hi;    // its range of order distances
  float u, top_p;     // the row's, kept out of the loops' registers
};

// A 64-bit sum by 32-bit additions: the low word returns what it held, so the
// carry is known, and the high word is touched only by large weights and
// carries.  Measured against 64-bit atomics on shared memory: 902 instead of
// 986 us for 224 rows of 248,320.
__device__ __forceinline__ void add_mass(Shared& s, uint32_t bin, u64 w) {
  const uint32_t lo = (uint32_t)w;
  const uint32_t old = atomicAdd(&s.hist_lo[bin], lo);
  const uint32_t up = (uint32_t)(w >> 32) + (old + lo < old ? 1u : 0u);
  if (up) atomicAdd(&s.hist_hi[bin], up);
}

// Inclusive prefix over a warp's first kN lanes.
template <int kN, typename V>
__device__ __forceinline__ V warp_prefix(V v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < kN; o <<= 1) {
    const V a = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += a;
  }
  return v;
}

// Exclusive prefix over the block (thread order) and the total.
template <typename V>
__device__ __forceinline__ V block_scan(V* warps, V v, V* all) {
  static_assert(kWarps == 16, "");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const V in = warp_prefix<32>(v);
  __syncthreads();
  if (lane == 31) warps[warp] = in;
  __syncthreads();
  const V w = warp_prefix<kWarps>(lane < kWarps ? warps[lane] : V(0));
  const V before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  *all = __shfl_sync(0xffffffffu, w, kWarps - 1);
  return (warp ? before : V(0)) + in - v;
}

// The cluster's histogram from the CTAs' own, in every CTA: thread (bin,
// source) of the CTA's slice of bins reads one value, the sources of a bin are
// summed by shuffles, and each of those lanes stores the sum to one CTA.
__device__ __forceinline__ void reduce_bins(Shared& s, uint32_t rank, int csize,
                                            bool mass, int bins) {
  __syncthreads();
  tc::cluster_sync();
  const int src = threadIdx.x % csize;
  for (int k = threadIdx.x; k < bins; k += kThreads) {
    const int bin = (int)rank * (bins / csize) + k / csize;
    u64 m = 0;
    if (mass)
      m = (u64)peer_load32(&s.hist_hi[bin], src) << 32 |
          peer_load32(&s.hist_lo[bin], src);
    uint32_t c = peer_load32(&s.hist_c[bin], src);
    for (int o = 1; o < csize; o <<= 1) {
      if (mass) m += __shfl_xor_sync(0xffffffffu, m, o);
      c += __shfl_xor_sync(0xffffffffu, c, o);
    }
    if (mass) peer_store64(&s.red_m[bin], src, m);
    peer_store32(&s.red_c[bin], src, c);
  }
  tc::cluster_sync();
}

// Short lists: an entry's place is the number of smaller ones (entries are
// distinct), counted by two threads for half of the list each.
__device__ __forceinline__ void rank_entries(Shared& s, int n) {
  const int tid = threadIdx.x, i = tid & 255, half = (n + 1) / 2;
  const u64 v = i < n ? s.list[i] : 0;
  const int j0 = tid < 256 ? 0 : half, j1 = tid < 256 ? half : n;
  int at = 0;
  if (i < n) {
#pragma unroll 8
    for (int j = j0; j < j1; ++j) at += s.list[j] < v;
    if (tid >= 256) s.part[i] = at;
  }
  __syncthreads();
  if (tid < 256 && i < n) s.list[at + s.part[i]] = v;
  __syncthreads();
}

// The largest of the block's values, in every thread.
__device__ __forceinline__ u64 block_max(u64* warps, u64 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const u64 a = __shfl_xor_sync(0xffffffffu, v, o);
    v = a > v ? a : v;
  }
  __syncthreads();
  if (lane == 0) warps[threadIdx.x >> 5] = v;
  __syncthreads();
  v = warps[lane % kWarps];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) {
    const u64 a = __shfl_xor_sync(0xffffffffu, v, o);
    v = a > v ? a : v;
  }
  return v;
}

// Longer lists are not sorted: the key (all are distinct) at which the running
// sum of the weights, in the keys' order, reaches want, which is above zero and
// at most their sum.  Rounds of a histogram over what is left of the keys'
// range, until one key is; the bins are zero before and after.  (A flat row
// with top-p 43 us; 50 to 63 with a sort of the list, up to 50,000 cycles for
// 1,273 entries.)
__device__ __forceinline__ u64 key_at(Shared& s, const u64 (&key)[kPerThread],
                                   const u64 (&w)[kPerThread], u64 want) {
  const int tid = threadIdx.x;
  u64 lo = 0, hi = 0;
#pragma unroll
  for (int e = 0; e < kPerThread; ++e)
    if (w[e]) {
      hi = key[e] > hi ? key[e] : hi;
      lo = ~key[e] > lo ? ~key[e] : lo;
    }
  hi = block_max(s.warp_m, hi);
  lo = ~block_max(s.warp_m, lo);
  for (;;) {
    const int shift = max(0, 64 - __clzll((long long)(hi - lo)) - kMassBits);
#pragma unroll
    for (int e = 0; e < kPerThread; ++e)
      if (w[e] && key[e] >= lo && key[e] <= hi) {
        const uint32_t d = (uint32_t)((key[e] - lo) >> shift);
        atomicAdd(&s.hist_c[d], 1u);
        add_mass(s, d, w[e]);
      }
    __syncthreads();
    u64 m[2];
    uint32_t c[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int d = 2 * tid + e;
      m[e] = (u64)s.hist_hi[d] << 32 | s.hist_lo[d];
      c[e] = s.hist_c[d];
      s.hist_hi[d] = s.hist_lo[d] = s.hist_c[d] = 0;
    }
    u64 all;
    const u64 before = block_scan(s.warp_m, m[0] + m[1], &all);
    if (before < want && want <= before + m[0] + m[1]) {
      const bool second = want > before + m[0];
      s.bin = 2 * tid + second;
      s.bin_c = second ? c[1] : c[0];
      s.before_m = before + (second ? m[0] : 0);
    }
    __syncthreads();
    want -= s.before_m;
    lo += (u64)s.bin << shift;
    const u64 end = lo + ((1ull << shift) - 1);
    hi = end < hi ? end : hi;
    if (!shift) return lo;
    if (s.bin_c == 1) {
#pragma unroll
      for (int e = 0; e < kPerThread; ++e)
        if (w[e] && key[e] >= lo && key[e] <= hi) s.cut = key[e];
      __syncthreads();
      return s.cut;
    }
  }
}

// The CTAs' lists one after the other in the first CTA, if all fit; returns
// their total in every thread.  Between two cluster barriers.
__device__ __forceinline__ int join_lists(Shared& s, uint32_t rank, int csize) {
  const int lane = threadIdx.x & 31;
  const int mine = (int)s.n_list;
  const int end = warp_prefix<kMaxCluster>(
      lane < csize ? (int)peer_load32(&s.n_list, lane) : 0);
  const int total = __shfl_sync(0xffffffffu, end, kMaxCluster - 1);
  const int at = __shfl_sync(0xffffffffu, end, rank) - mine;
  if (rank && total <= kList)
    for (int i = threadIdx.x; i < mine; i += kThreads)
      peer_store64(&s.list[at + i], 0, s.list[i]);
  return total;
}

// The last kept token, as a value and an id in this CTA's chunk.
struct Border {
  float x;
  int i;
  __device__ __forceinline__ bool holds(float v, int id) const {
    return v > x || (v == x && id <= i);
  }
};
__device__ __forceinline__ Border border_of(u64 cut, uint32_t mkey, int base) {
  if (cut == ~0ull) return {-INFINITY, -1};  // every finite value
  return {value_of(mkey - (uint32_t)(cut >> kIdBits)),
          (int)(cut & ((1u << kIdBits) - 1)) - base};
}

// The draw's target among W: floor(u W), below W.
__device__ __forceinline__ u64 target_of(float u, u64 W) {
  const u64 t = u >= 1.f ? W : (u > 0.f ? floor_part(u, W) : 0);
  return t < W ? t : W - 1;
}

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
  const float T0 = p.temperature ? p.temperature[row] : 1.f;
  const float u = p.u[row];
  int k = p.top_k ? p.top_k[row] : 0;
  const float tp = p.top_p ? p.top_p[row] : 1.f;
  const float mp = p.min_p ? p.min_p[row] : 0.f;
  const bool idle = !(T0 >= 0.f);
  if (k <= 0 || k >= p.vocab) k = 0;
  // cuts that leave the first token alone
  const bool one = T0 == 0.f || k == 1 || tp <= 0.f || mp > 1.f;
  if (tid < 32) fill_table(s.tab, tid);
  for (int i = n + tid; i < p.padded; i += kThreads)
    store_float(xs + i, -INFINITY);
  for (int j = tid; j < kBins; j += kThreads)
    s.hist_lo[j] = s.hist_hi[j] = s.hist_c[j] = 0;
  if (tid == 0) {
    s.n_list = 0;
    s.u = u;
    s.top_p = tp;
  }
  asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory");
  __syncthreads();

  // the largest logit with its lowest id, and the smallest finite one
  const float most = largest(T());
  float top = -INFINITY, least = INFINITY;
  int top_i = tid;
  for (int i0 = tid; i0 < p.padded; i0 += kBatch * kThreads) {
    float x[kBatch];
#pragma unroll
    for (int e = 0; e < kBatch; ++e)
      x[e] = clean(as_float(xs[i0 + e * kThreads]), most);
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int i = i0 + e * kThreads;
      store_float(xs + i, x[e]);  // later passes read clean values
      if (x[e] > top) {           // the first of equals
        top = x[e];
        top_i = i;
      }
      least = fminf(least, x[e] > -INFINITY ? x[e] : INFINITY);
    }
  }
  reinterpret_cast<float*>(s.list)[tid] = top;  // for a small top-k
  u64 best = (u64)key_of(top) << 32 | (uint32_t)~(uint32_t)(base + top_i);
  uint32_t low = least < INFINITY ? key_of(least) : 0xffffffffu;
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
  if (warp == 0) {
    best = lane < kWarps ? s.warp_m[lane] : 0;
    low = lane < kWarps ? s.warp_c[lane] : 0xffffffffu;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
      const u64 v = __shfl_xor_sync(0xffffffffu, best, o);
      best = v > best ? v : best;
    }
    low = __reduce_min_sync(0xffffffffu, low);
    if (lane == 0) {
      s.x_m[0] = best;
      s.x_c = low;
    }
  }
  __syncthreads();
  tc::cluster_sync();
  // one lane per CTA of the cluster, then the same on every lane
  best = peer_load64(&s.x_m[0], lane % csize);
  low = __reduce_min_sync(0xffffffffu, peer_load32(&s.x_c, lane % csize));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const u64 v = __shfl_xor_sync(0xffffffffu, best, o);
    best = v > best ? v : best;
  }
  const uint32_t mkey = (uint32_t)(best >> 32);
  const int arg = (int)~(uint32_t)best;
  Row r;
  r.m = value_of(mkey);
  const bool none = idle || !(r.m > -INFINITY);

  u64 cut = ~0ull;     // (order distance, id) of the last kept token
  u64 total = 0;       // kept mass
  u64 minw = 0;
  bool done = none || one;
  bool leave = false;  // the first CTA finishes alone
  if (done) {
    if (rank == 0 && tid == 0) p.token[row] = none ? -1 : arg;
  } else {
    set_scale(r, T0);
    if (mp > 0.f) minw = __float2ull_ru(__fmul_rn(mp, 8796093022208.f));
    auto place = [&](float x, int i) {  // a token's place in the order
      return (u64)(mkey - key_of(x)) << kIdBits | (uint32_t)(base + i);
    };
    auto weight_at = [&](u64 c) {
      return weight_of(r, value_of(mkey - (uint32_t)(c >> kIdBits)), s.tab);
    };

    // 2. the cuts.  The first round's bins: even steps of the logit over
    // what has weight
    const float span = fminf(__fsub_rn(r.m, value_of(low)), 45.f / r.kh);
    for (int which = 0; which < 2 && !done; ++which) {  // top-k, then top-p
      if (which == 0 ? k == 0 : !(s.top_p < 1.f)) continue;
      const bool mass = which == 1;
      const int bits = mass ? kMassBits : kCountBits, bins = 1 << bits;
      const float step = span > 0.f ? fminf((bins - 1) / span, kMaxFinite) : 0.f;
      auto bin_of = [&](float x) {
        const float f = __fmul_rn(__fsub_rn(r.m, x), step);
        return f < bins - 1 ? (uint32_t)f : (uint32_t)bins - 1;  // NaN: the last
      };
      const u64 old = cut;
      u64 want = mass ? 0 : (u64)k;  // the border is where the sum reaches it
      u64 lo = 0, hi = ~0ull >> 1;
      // The k-th largest of the threads' own maxima is no larger than the row's
      // k-th largest logit: while k is small beside the threads, a round -1
      // counts those maxima instead of all tokens, and what reaches its border
      // holds the k tokens and a few more.  If that is more than a list holds,
      // or fewer threads than k have a finite value, round 0 follows.  (64
      // fp32 rows of 248,320 with top-k of 20 to 200 and top-p: 85 us, 101
      // when round 0 counts all tokens at once.)
      const bool small = !mass && k <= kThreads * csize / 4 && k <= kList / 2;
      if (tid == 0) s.before_m = s.before_c = 0;
      for (int round = small ? -1 : 0;; ++round) {
        const bool quick = round < 0;
        const int shift =
            round > 0 ? max(0, 64 - __clzll((long long)(hi - lo)) - bits) : 0;
        if (quick) {
          const float mine = reinterpret_cast<const float*>(s.list)[tid];
          if (mine > -INFINITY) atomicAdd(&s.hist_c[bin_of(mine)], 1u);
        } else if (round == 0 && !mass) {
          // every finite value, no order beside its bin
          for (int i0 = tid; i0 < p.padded; i0 += kBatch * kThreads) {
            float x[kBatch];
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
              x[e] = as_float(xs[i0 + e * kThreads]);
#pragma unroll
            for (int e = 0; e < kBatch; ++e)
              if (x[e] > -INFINITY) atomicAdd(&s.hist_c[bin_of(x[e])], 1u);
          }
        } else if (round == 0) {
          constexpr int kB = kBatch / 2;
          for (int i0 = tid; i0 < p.padded; i0 += kB * kThreads) {
            float x[kB];
            u64 w[kB];
#pragma unroll
            for (int e = 0; e < kB; ++e) x[e] = as_float(xs[i0 + e * kThreads]);
#pragma unroll
            for (int e = 0; e < kB; e += 2)
            warp_weights(r, make_float2(x[e], x[e + 1]), s.tab, w[e], w[e + 1]);
#pragma unroll
            for (int e = 0; e < kB; ++e) {
              if (!(x[e] > -INFINITY) ||
                  (old != ~0ull && place(x[e], i0 + e * kThreads) > old))
                continue;
              const uint32_t d = bin_of(x[e]);
              atomicAdd(&s.hist_c[d], 1u);
              if (w[e]) add_mass(s, d, w[e]);
            }
          }
        } else {
          for (int i = tid; i < n; i += kThreads) {
            const float x = as_float(xs[i]);
            const u64 c = place(x, i);
            if (x == -INFINITY || c > old || c < lo || c > hi) continue;
            const uint32_t d = (uint32_t)((c - lo) >> shift);
            atomicAdd(&s.hist_c[d], 1u);
            if (mass) {
              const u64 w = weight_of(r, x, s.tab);
              if (w) add_mass(s, d, w);
            }
          }
        }
        reduce_bins(s, rank, csize, mass, bins);
        for (int j = tid; j < bins; j += kThreads)
          s.hist_lo[j] = s.hist_hi[j] = s.hist_c[j] = 0;
        if (tid == 0) s.bin = kBins;
        const u64 above_m = s.before_m;
        const uint32_t above_c = s.before_c;
        const bool two = 2 * tid < bins;
        const uint32_t vc0 = two ? s.red_c[2 * tid] : 0;
        const uint32_t vc1 = two ? s.red_c[2 * tid + 1] : 0;
        const u64 vm0 = mass ? s.red_m[2 * tid] : 0;
        const u64 vm1 = mass ? s.red_m[2 * tid + 1] : 0;
        u64 em = 0, am = 0;
        uint32_t ac;
        const uint32_t ec = block_scan(s.warp_c, vc0 + vc1, &ac);
        if (mass) em = block_scan(s.warp_m, vm0 + vm1, &am);
        if (round <= 0) {
          if (mass) {  // the mass before a kept token is below p W
            want = ceil_part(s.top_p, am);
          } else if (want > ac) {
            if (quick) continue;
            break;  // fewer finite logits than k
          }
        }
        const u64 ex = mass ? above_m + em : (u64)above_c + ec;
        const u64 mid = ex + (mass ? vm0 : (u64)vc0);
        const u64 end = mid + (mass ? vm1 : (u64)vc1);
        if (ex < want && want <= end) {
          const bool second = want > mid;
          s.bin = 2 * tid + second;
          s.bin_c = second ? vc1 : vc0;
          s.before_m = above_m + em + (second ? vm0 : 0);
          s.before_c = above_c + ec + (second ? vc0 : 0);
        }
        __syncthreads();
        const uint32_t b = s.bin;
        if (b == kBins) break;  // cannot be: the sums reach want
        const uint32_t in_bin = s.bin_c;
        const bool finish = quick || s.before_c + in_bin <= kList;
        if (finish || in_bin <= kList) {
          // gather: all up to the bin's end, or the bin
          if (round <= 0) {
            // what lies up to the bin's upper edge is looked at more closely
            // (its edge a little lower: the bins are decided by rounded steps)
            const float reach = __fdiv_rn((float)(b + 1), step);
            const float edge = b < bins - 1 && step > 0.f
                                   ? fmaxf(__fsub_rn(r.m, __fmul_rn(reach, 1.001f)),
                                           -kMaxFinite)
                                   : -kMaxFinite;
            auto append = [&](float x, int i) {
              const u64 c = place(x, i);
              if (c > old) return;
              const uint32_t at = atomicAdd(&s.n_list, 1u);
              if (at < kList) s.list[at] = c;  // more: too many anyway
            };
            if (finish) {
              for (int i0 = tid; i0 < p.padded; i0 += kBatch * kThreads) {
                float x[kBatch];
                bool any = false;
#pragma unroll
                for (int e = 0; e < kBatch; ++e) {
                  x[e] = as_float(xs[i0 + e * kThreads]);
                  any |= x[e] >= edge;
                }
                if (!any) continue;
#pragma unroll
                for (int e = 0; e < kBatch; ++e)
                  if (x[e] >= edge && (quick || bin_of(x[e]) <= b))
                    append(x[e], i0 + e * kThreads);
              }
            } else {
              // within the bin alone, few tokens pass (224 flat bf16 rows 455
              // us; 468 where all above the bin are looked at as well)
              const float inner = __fdiv_rn(__fmul_rn((float)b, 0.999f), step);
              const float upper = step > 0.f ? __fsub_rn(r.m, inner) : kMaxFinite;
              for (int i0 = tid; i0 < p.padded; i0 += kBatch * kThreads) {
                float x[kBatch];
#pragma unroll
                for (int e = 0; e < kBatch; ++e)
                  x[e] = as_float(xs[i0 + e * kThreads]);
#pragma unroll
                for (int e = 0; e < kBatch; ++e)
                  if (x[e] >= edge && x[e] <= upper && bin_of(x[e]) == b)
                    append(x[e], i0 + e * kThreads);
              }
            }
          } else {
            for (int i = tid; i < n; i += kThreads) {
              const float x = as_float(xs[i]);
              const u64 c = place(x, i);
              if (x == -INFINITY || c > old || c > hi) continue;
              const bool take = c < lo ? finish
                                       : (finish ? (c - lo) >> shift <= b
                                                 : (c - lo) >> shift == b);
              if (take) s.list[atomicAdd(&s.n_list, 1u)] = c;
            }
          }
          __syncthreads();
          tc::cluster_sync();
          const int m = join_lists(s, rank, csize);
          tc::cluster_sync();
          if (tid == 0) s.n_list = 0;
          if (m > kList) {  // round -1: more than the maxima showed
            if (tid == 0) s.before_c = 0;
            __syncthreads();
            continue;
          }
          // Without a distribution to write, the first CTA goes on alone; the
          // SMs of the others are free for the next row (64 fp32 rows with
          // top-k 85 -> 67 us; one row 18.6 -> 19.4 for the second barrier).
          leave = finish && !p.probs && !p.filtered;
          constexpr u64 kIdMask = (1ull << kIdBits) - 1;
          if (rank == 0 && m > kRanked) {
            u64 key[kPerThread], w[kPerThread], sum = 0, all;
#pragma unroll
            for (int e = 0; e < kPerThread; ++e) {
              const int q = tid + e * kThreads;
              key[e] = q < m ? s.list[q] : ~0ull;
              w[e] = q < m;
            }
            u64 last = ~0ull - 1;  // the last kept one so far
#pragma unroll 1
            for (int step = 0; step < 3; ++step) {  // top-k, top-p, the draw
              bool need = true;
              u64 to;
              if (step == 0) {
                need = !mass && (!finish || k < m);
                to = finish ? k : want - s.before_c;
              } else if (step == 1) {
                sum = 0;
#pragma unroll
                for (int e = 0; e < kPerThread; ++e) {
                  w[e] = key[e] <= last && (mass || finish) ? weight_at(key[e]) : 0;
                  sum += w[e];
                }
                block_scan(s.warp_m, sum, &all);
                need = mass || (finish && s.top_p < 1.f);
                to = !mass ? ceil_part(s.top_p, all)
                           : finish ? want : want - s.before_m;
              } else {
                if (!finish) break;
                u64 far = 0;
                sum = 0;
#pragma unroll
                for (int e = 0; e < kPerThread; ++e) {
                  const bool keep = key[e] <= last && w[e] >= minw;
                  far = keep && key[e] > far ? key[e] : far;
                  w[e] = keep ? w[e] : 0;
                  sum += w[e];
                  key[e] &= kIdMask;
                }
                last = block_max(s.warp_m, far);
                block_scan(s.warp_m, sum, &all);
                to = target_of(s.u, all) + 1;
              }
              if (!need) continue;
              const u64 at = key_at(s, key, w, to);
              if (step < 2)
                last = at;
              else if (tid == 0)
                p.token[row] = (int32_t)at;
            }
            if (!leave && tid < csize) {  // (the others are gone, else)
              peer_store64(&s.cut, tid, last);
              if (finish) peer_store64(&s.total, tid, all);
            }
          } else if (rank == 0) {
            // an entry a thread, in order
            rank_entries(s, m);
            const int q = tid;
            const bool in = q < m && (!finish || mass || q < k);
            u64 w = in && (mass || finish) ? weight_at(s.list[q]) : 0, all;
            const u64 run = block_scan(s.warp_m, w, &all);
            if (!finish) {
              // the border among the bin's tokens
              const u64 at = s.before_m + run;
              if (q < m && (mass ? at < want && want <= at + w
                                 : (u64)s.before_c + q + 1 == want))
                s.cut = s.list[q];
              __syncthreads();
              // (not finished: every CTA is still here)
              if (tid < csize) peer_store64(&s.cut, tid, s.cut);
            } else {
              // Every remaining cut: a prefix of the ranks, and of those
              // the ones that min-p keeps.  Those need not be a prefix: of
              // two close logits the smaller may have the larger integer, a
              // step of 2^-43 above.  So the ranks go up to the last kept
              // one, and one between that is not kept has no weight.
              u64 limit = mass ? want : ~0ull;
              if (!mass && s.top_p < 1.f) limit = ceil_part(s.top_p, all);
              const bool keep = in && run < limit && w >= minw;
              w = keep ? w : 0;
              if (q < kRanked) s.wts[q] = w;
              block_scan(s.warp_m, w, &all);
              const uint32_t nk =
                  (uint32_t)block_max(s.warp_m, keep ? (u64)q + 1 : 0);
              if (!leave && tid < csize) {
                peer_store64(&s.cut, tid, s.list[nk - 1]);
                peer_store64(&s.total, tid, all);
              }
              __syncthreads();
              // the draw, in id order
              if (q < (int)nk) s.list[q] = (s.list[q] & kIdMask) << 32 | (uint32_t)q;
              __syncthreads();
              rank_entries(s, (int)nk);
              const u64 t = target_of(s.u, all);
              w = q < (int)nk ? s.wts[(uint32_t)s.list[q]] : 0;
              const u64 at = block_scan(s.warp_m, w, &all);
              if (at <= t && t < at + w)
                p.token[row] = (int32_t)(s.list[q] >> 32);
            }
          }
          if (!leave) {
            __syncthreads();
            tc::cluster_sync();
            cut = s.cut;
            if (finish) total = s.total;
          }
          done = finish;
          break;
        }
        // too many in one bin: its range of places is the next round's
        if (round == 0) {
          // order distances in bin b: the digit does not decrease with them
          if (tid < 2) {
            uint32_t a = 0, z = 0xffffffffu;  // first distance with digit >= g
            const uint32_t g = b + tid;
            if (g < bins) {
              while (a < z) {
                const uint32_t mid = a + ((z - a) >> 1);
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
          lo = (u64)s.lo << kIdBits;
          hi = ((u64)s.hi + 1 << kIdBits) - 1;
        } else {
          const u64 end = lo + ((u64)(b + 1) << shift) - 1;
          hi = end < hi ? end : hi;
          lo += (u64)b << shift;
        }
        __syncthreads();
      }
      __syncthreads();
    }

    if (!done) {
      // 3. kept mass, each warp a run of ids
      const Border edge = border_of(cut, mkey, base);
      auto kept = [&](float x, int i) { return edge.holds(x, i); };
      const int run_len = p.padded / kWarps;
      // The weights, most of the time here, are made for full pairs of warps:
      // kept tokens of mixed ones are queued until there are 64 (at most 127,
      // where the lists were), in any order, as the sum is an integer.
      float* queue = reinterpret_cast<float*>(s.list) + warp * 128;
      const uint32_t below = (1u << lane) - 1;
      int queued = 0;
      u64 m = 0;
      auto add_kept = [&](float2 v) {
        u64 w0, w1;
        warp_weights(r, v, s.tab, w0, w1);
        m += (w0 >= minw ? w0 : 0) + (w1 >= minw ? w1 : 0);
      };
      for (int i0 = warp * run_len + lane; i0 < (warp + 1) * run_len;
           i0 += 4 * 32) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = as_float(xs[i0 + 32 * e]);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const bool in0 = kept(x[e], i0 + 32 * e);
          const bool in1 = kept(x[e + 1], i0 + 32 * (e + 1));
          const uint32_t m0 = __ballot_sync(0xffffffffu, in0);
          const uint32_t m1 = __ballot_sync(0xffffffffu, in1);
          if (!(m0 | m1)) continue;
          float2 v = make_float2(x[e], x[e + 1]);
          if ((m0 & m1) != 0xffffffffu) {
            if (in0) queue[queued + __popc(m0 & below)] = v.x;
            queued += __popc(m0);
            if (in1) queue[queued + __popc(m1 & below)] = v.y;
            queued += __popc(m1);
            if (queued < 64) continue;
            queued -= 64;
            __syncwarp();
            v = make_float2(queue[queued + lane], queue[queued + 32 + lane]);
            __syncwarp();
          }
          add_kept(v);
        }
      }
      __syncwarp();
      add_kept(make_float2(
          lane < queued ? queue[lane] : -INFINITY,
          lane + 32 < queued ? queue[lane + 32] : -INFINITY));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
      if (lane == 0) s.warp_m[warp] = m;
      __syncthreads();
      if (tid == 0) {
        u64 all = 0;
        for (int w = 0; w < kWarps; ++w) all += s.warp_m[w];
        s.x_m[1] = all;
      }
      __syncthreads();
      tc::cluster_sync();
      u64 at = 0, mine = 0;  // kept mass before this CTA and in it
      for (int j = 0; j < csize; ++j) {
        const u64 w = peer_load64(&s.x_m[1], j);
        at += j < (int)rank ? w : 0;
        mine = j == (int)rank ? w : mine;
        total += w;
      }
      const u64 t = target_of(s.u, total);
      if (at <= t && t < at + mine) {  // the same for the whole CTA
        int w0 = 0;
        while (at + s.warp_m[w0] <= t) at += s.warp_m[w0++];
        // the run's tokens again, consecutive ones to a thread
        const int per = (run_len + kThreads - 1) / kThreads;
        const int i0 = w0 * run_len + tid * per;
        const int i1 = (w0 + 1) * run_len;
        u64 w[kPerDraw], sum = 0;
#pragma unroll
        for (int e = 0; e < kPerDraw; ++e) {
          w[e] = 0;
          if (e < per && i0 + e < i1) {
            const float x = as_float(xs[i0 + e]);
            if (kept(x, i0 + e)) w[e] = weight_of(r, x, s.tab);
            if (w[e] < minw) w[e] = 0;
          }
          sum += w[e];
        }
        u64 all;
        at += block_scan(s.warp_m, sum, &all);
#pragma unroll
        for (int e = 0; e < kPerDraw; ++e) {
          if (at <= t && t < at + w[e]) p.token[row] = base + i0 + e;
          at += w[e];
        }
      }
    }
  }

  // the distribution
  if (p.probs || p.filtered) {
    const float inv =
        total ? __fdiv_rn(8796093022208.f, __ull2float_rn(total)) : 0.f;
    const long long out = (long long)row * p.vocab + base;
    const Border edge = one ? Border{kMaxFinite, -1} : border_of(cut, mkey, base);
    int i0 = tid;
    if (!p.filtered && !none && !one && !minw) {
      // the usual call: whole batches with nothing else to look at
      float* o = p.probs + out + tid;
      for (; i0 + 3 * kThreads < n; i0 += 4 * kThreads, o += 4 * kThreads) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = as_float(xs[i0 + e * kThreads]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float w = fast_weight(r, x[e]) * inv;
          __stcs(o + e * kThreads, edge.holds(x[e], i0 + e * kThreads) ? w : 0.f);
        }
      }
    }
    for (; i0 < n; i0 += 4 * kThreads) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + e * kThreads;
        x[e] = i < p.padded ? as_float(xs[i]) : -INFINITY;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = i0 + e * kThreads;
        if (i >= n) continue;
        bool keep = !none && (one ? base + i == arg : edge.holds(x[e], i));
        float pr = one && keep ? 1.f : 0.f;
        // beside a cut that already holds it, min-p decides only here
        if (keep && minw) keep = weight_of(r, x[e], s.tab) >= minw;
        if (keep && !one) pr = fast_weight(r, x[e]) * inv;
        if (p.probs) __stcs(p.probs + out + i, pr);
        if (p.filtered) __stcs(p.filtered + out + i, keep ? x[e] : -INFINITY);
      }
    }
  }
  // no CTA leaves while others read its shared memory
  if (!leave) tc::cluster_sync();
}

template <typename T>
cudaError_t launch(const SampleParams& p, int csize, cudaStream_t s) {
  const size_t smem = (size_t)p.padded * sizeof(T) + 32;
  // once per device (an attribute call per launch costs microseconds)
  static std::atomic<uint64_t> ready{0};
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(
        sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        kMaxChunk * (int)sizeof(T) + 32);
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
  // The smallest cluster whose CTAs hold at most 64 KB of the row, two to an
  // SM, but no more than 8 while kMaxChunk tokens each will do: few clusters of
  // 16 are resident at a time (64 fp32 rows of 248,320: 112 us with 8 CTAs a
  // row, 126 with 16; 224 bf16 rows: 772 us with 8, 909 with 4, 1,237 with 16).
  // With few rows, more CTAs per row while SMs would stay empty and a CTA keeps
  // a few tokens per thread; 16 for at most kWideRows rows (of 248,320; top-k
  // and top-p, then top-p alone over a flat row: 7 rows 21.4 and 53 us with 16,
  // 23.0 and 76 with 8; 8 rows, a second wave, 25.8 and 59 against 23.0 and 76;
  // 9 rows 27.9 and 78.5 against 23.8 and 78.5).
  const size_t bytes = (size_t)p.vocab * (bf16 ? 2 : 4);
  int csize = 1;
  while (csize < 8 && bytes > (size_t)csize * 65536) csize *= 2;
  if (p.vocab > csize * kMaxChunk) csize = kMaxCluster;
  while (csize < (p.rows <= kWideRows ? kMaxCluster : 8) &&
         (long long)p.rows * csize * 2 <= sms && p.vocab > csize * 4096)
    csize *= 2;
  p.chunk = ((p.vocab + csize - 1) / csize + 7) / 8 * 8;
  p.padded = (p.chunk + kPad - 1) / kPad * kPad;
  return bf16 ? launch<__nv_bfloat16>(p, csize, s) : launch<float>(p, csize, s);
}

}  // namespace specv
