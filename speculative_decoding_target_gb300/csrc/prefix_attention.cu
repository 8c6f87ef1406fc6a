// Attention of all rows of a group over its shared prefix, on CTA pairs
// (tcgen05 cta_group::2), for bf16 KV and for FP8-E4M3 KV with fp16 scales.
//
// For the rows of one KV head, all requests of the group together, the shared
// prefix is one K and one V: S = Q K^T, O = softmax(S) V with no mask, since
// every row sees every shared token.  With hundreds of rows per KV head the
// work is bound by the tensor cores (4 D flop per row and token against 4 D
// bytes per token), unlike the verify block's 48 rows, which HBM bounds.
//
// A piece of the plan (shared_prefix.cuh) is kPrefixRows = 256 rows, 128 per CTA
// of a pair, over a run of the shared tokens.  Tensor memory, 512 columns
// in each CTA: O [0, 256), two S buffers of 128 columns (one tile of 128
// tokens each) [256, 512); P (16-bit) overwrites its S.  Q lies in shared
// memory.  A measured stream of MMAs takes N / 2 cycles from N = 128 on,
// whether A comes from shared or tensor memory, and 50 instead of 32 at
// N = 64: tiles of 128 tokens run at the full rate, which leaves no tensor
// memory for Q.  A row tile of 128 rows alone would read 64 KB of K and V per
// 1,024 cycles of MMAs, all that an SM takes from L2 (measured 60 bytes per
// cycle); the pair halves that, each CTA loading half the tokens of K and half
// the channels of V.
//
// Warp roles (both CTAs):
//   warps 0, 2  producers of K and of V: TMA boxes of the CTA's halves, [64
//               tokens x 128 channels] twice a tile for each, 128-byte
//               swizzle, into a ring in the order in which the issuer consumes
//               them: K0 K1 V0 K2 V1 ...
//   warp 1      leader: issuer, QK_0, then per tile QK_{j+1}, PV_j, so that
//               the softmax of tile j has a QK and a PV's time to run in
//   warps 1, 3  FP8, the other CTA: relays, see relay_piece
//   warps 4..7  softmax: one thread per row; running maximum and sum in base
//               2 and fp32; O is rescaled only when the maximum grows by 2^8
//               (FP8: 2^4); epilogue (normalised fp32 partial, log-sum-exp)
//   warps 8..15 FP8 only: E4M3 bytes times scale to fp16 slots, two sets of
//               four warps on alternate staging buffers
// With FP8's sixteen warps in different code the instruction cache is what
// limits first: loops are rolled and each step has one call site (with
// everything unrolled and inlined, 3.6 cycles of every issue were spent waiting
// for instructions and a tile took 4,400 cycles).
//
// P is rounded once to the type of V.  bf16: a weight is off by at most 2^-8 of
// itself, whatever its size, as the bf16 output is of its value.  (The verify
// kernel splits P into two bf16 terms, free where HBM is the bound; here it
// would add half again to the MMAs.)  FP8 KV: fp16, off by at most 2^-11 of
// itself down to 2^-14 and by 2^-25 below, where its steps are even; a long
// prefix may hold much of its mass in weights that small beside the largest one.
// So P, O and the sum carry a factor of 2^11: with O rescaled at a growth of 2^4,
// P lies at most at 2^15, and a weight that is w of the largest (or of the
// maximum in use, if that is smaller) is off by 2^-11 w or, below w = 2^-25, by
// 2^-36; a million tokens that small together by 2^-16 of the row.  The factor
// leaves with the division by the sum, and the log-sum-exp's 11.
//
// Measured (24 query heads, 4 KV heads): bf16, 32 requests x 8 rows over 32,768
// shared tokens, 206 Gflop: 121 us, 1.71 Pflop/s, 0.89 of the measured bf16 rate;
// the tensor pipe is busy 81% of the time, DRAM reads 137.5 MB of the prefix's
// 134.2.  What is left is the first and last tile of each piece and the issuer's
// waits on the softmax.  FP8, 64 single tokens over 65,536, 103 Gflop: 117 us, 0.46
// of that rate; the conversion of E4M3 to fp16 through shared memory bounds it
// (issue slots 51% busy, the tensor pipe 53%).
//
// Causal (chunk_attention.cuh), bf16: 4,096 tokens into an empty cache, 206 Gflop,
// 146 us, 136 of them here; 2,048 tokens behind 32,768, 1.70 Pflop, 941 us at full
// clocks, 0.94 of the measured bf16 rate, 1,036 under the power limit.  FP8, six
// ragged requests on 16-token pages, 274 Gflop: 291 us; 2,048 tokens behind 32,768
// 1,250.
//
// Every wait is bounded as in verify_attention_tc.cu.
#include <cuda_fp8.h>

#include <type_traits>

#include "chunk_attention.cuh"
#include "pair_ptx.cuh"
#include "shared_prefix.cuh"
#include "spec_verify.h"
#include "tmem_io.cuh"

namespace specv {
namespace {

constexpr int kT = kPrefixTile;
constexpr int kHalfBytes = 64 * 128 * 2;      // 64 tokens x 128 channels
constexpr int kBlockBytes = 64 * 128;         // its column block of 64
constexpr int kQBytes = 128 * kHeadDim * 2;   // 4 column blocks of 128 rows
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 256;
constexpr int kMaxSlots = 5;
constexpr int kRaw = 3;                       // FP8 staging buffers
constexpr int kRawBytes = 16384 + 1024;       // bytes and scales

template <bool kFp8>
struct Cfg {
  // a slot holds a CTA's share of K or V of one tile
  static constexpr int kSlots = kFp8 ? 3 : 5;
  static constexpr int kSlotBytes = 2 * kHalfBytes;
  static constexpr int kThreads = kFp8 ? 512 : 256;
  static constexpr int kOffRing = kQBytes;
  static constexpr int kOffRaw = kOffRing + kSlots * kSlotBytes;
  static constexpr int kSmem = kOffRaw + (kFp8 ? kRaw * kRawBytes : 0) + 1024;
  static constexpr uint32_t kAB = kFp8 ? 0u : 1u;  // fp16 or bf16 inputs
  // growth of the maximum (log2) that rescales O, and the factor that P and
  // the sum carry (log2); 2^(4 + 11) is fp16's 32,768
  static constexpr float kRescaleLog2 = kFp8 ? 4.f : 8.f;
  static constexpr float kShiftLog2 = kFp8 ? 11.f : 0.f;
  static constexpr uint32_t kIdescQK = (1u << 4) | (kAB << 7) | (kAB << 10) |
                                       ((uint32_t)(kT >> 3) << 17) |
                                       ((uint32_t)(256 >> 4) << 24);
  static constexpr uint32_t kIdescPV = (1u << 4) | (kAB << 7) | (kAB << 10) |
                                       (1u << 16) | ((uint32_t)(256 >> 3) << 17) |
                                       ((uint32_t)(256 >> 4) << 24);
};

struct Bars {
  // bf16, leader: the slot holds both CTAs' halves (TMA); FP8, both: this
  // CTA's half is dequantised, and in the leader the other CTA's too
  uint64_t full[kMaxSlots], peer_full[kMaxSlots];
  uint64_t empty[kMaxSlots];   // both: the slot's MMAs are done
  uint64_t s_full[2];          // both: S_j complete
  uint64_t p_full[2];          // leader: P_j written by both CTAs
  uint64_t pv_done[2];         // both: PV_j complete
  uint64_t q_full;             // leader: Q written by both CTAs
  uint64_t q_land;             // chunk, FP8, own: bf16 queries landed
  uint64_t raw_full[kRaw];     // FP8, own: staged bytes landed
  uint64_t raw_empty[kRaw];    // FP8, own: staged bytes converted
  // chunk, bf16, own: V that needs zeros landed.  One a slot, as with short
  // pieces several such slots may have landed before the first is looked at.
  uint64_t tail_full[kMaxSlots];
  uint64_t drain;              // both: every MMA issued is done
};

struct Ctx {
  Bars* bars;
  volatile int* abort;
  uint32_t peer_abort;         // cluster address of the other CTA's flag
  uint32_t rank;
  const AttnParams* a;
  float* pre_o;
  float* pre_lse;
  const CUtensorMap* tm_q;     // chunk: queries
  int cta_rows, q_tokens;
};

__device__ __forceinline__ void give_up(const Ctx& cx) {
  *cx.abort = 1;
  tc::store_cluster(cx.peer_abort, 1u);
  if (cx.a->status) atomicOr(cx.a->status, SPEC_STATUS_TIMEOUT);
}

// Barriers that carry generic writes of the other CTA (Q, dequantised tiles)
// are waited for at cluster scope; the others carry tensor-memory or TMA
// completions.
template <bool kCluster>
__device__ __noinline__ bool wait_slow(const Ctx& cx, uint32_t a,
                                       uint32_t parity, bool drain) {
  if (!drain && *cx.abort) return false;
  const long long bound = drain ? kDrainWaitCycles : cx.a->wait_cycles;
  const long long t0 = clock64();
  while (true) {
    if (kCluster ? tc::bar_try_wait_cluster(a, parity)
                 : tc::bar_try_wait(a, parity))
      return true;
    if (!drain && *cx.abort) return false;
    if (clock64() - t0 > bound) {
      give_up(cx);
      return false;
    }
  }
}
template <bool kCluster = false>
__device__ __forceinline__ bool wait_bar(const Ctx& cx, uint64_t* bar,
                                         uint32_t parity, bool drain = false) {
  const uint32_t a = tc::smem_u32(bar);
  if (kCluster ? tc::bar_try_wait_cluster(a, parity)
               : tc::bar_try_wait(a, parity))
    return true;
  return wait_slow<kCluster>(cx, a, parity, drain);
}

// A place in a ring of N buffers and the parity of the wait for its current
// use (a consumer's; a producer waits for the use before, of the other one).
// The producers of K and of V, and the two dequantising sets, wait for the
// release of a buffer (`empty`, `raw_empty`) only before their own units and
// step over the others'.  A wait by parity returns at once while the phase
// before the one it means is still open, as the phase before that has the same
// parity.  Before unit i, the wait is for the release of unit i - N, and the
// phase before is that of unit i - 2 N.  Units are released in order, and at
// most 3 lie from one of a waiter's own to the next (V(n-1) K0 K1 V0 across a
// piece border; the sets alternate), so the units up to i - 3 - N are known to
// be released: i - 2 N is among them while N >= 3.
template <int N>
struct Ring {
  static_assert(N >= 3, "a wait could take an earlier phase for its own");
  int at = 0;
  uint32_t parity = 0;
  bool wrapped = false;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      parity ^= 1;
      wrapped = true;
    }
  }
};

// A piece of the plan as one CTA sees it.
struct Piece {
  int lead, start, rows_total;  // page-table row, first request, group rows
  int g, row0;                  // KV head, first row of this CTA's 128
  int tok, n_tiles;
  int slot;                     // partial slot, or -1: straight to the output
  // a chunk's piece
  int last;                     // last cached token of the request
  int first;                    // block row of row 0
  int limit;                    // tokens that row 0 sees
  // Cached tokens of the last tile; behind them its V rows become zeros: their
  // weights are zero, but what lies there may not be a number.
  __device__ __forceinline__ int tail_tokens() const {
    return min(last + 1 - (tok + (n_tiles - 1) * kT), kT);
  }
};

// Behind the cache the page of its last token stands in: the tokens are masked.
template <bool kCausal>
__device__ __forceinline__ int page_id(const AttnParams& p, const Piece& pc,
                                       int t) {
  if (kCausal) t = min(t, pc.last);
  return __ldg(p.page_table + (long long)pc.lead * p.max_pages +
               (t >> p.log2_ps));
}
// Looked at only when the page is used, so that the load of the id runs ahead.
__device__ __forceinline__ int checked_page(const AttnParams& p, int page) {
  if (page < 0 || page >= p.num_pages) {
    if (p.status) atomicOr(p.status, SPEC_STATUS_BAD_PAGE);
    page = 0;  // in bounds; the affected rows are unspecified
  }
  return page;
}

// (The pool has fewer than 2^31 rows.)
__device__ __forceinline__ int pool_row(const AttnParams& p, int page, int g,
                                        int t) {
  return ((page * p.hkv + g) << p.log2_ps) + (t & (p.page_size - 1));
}

// ---- warps 0 and 2: loads -----------------------------------------------------
// A half of 64 tokens is kNb boxes of each column block, of 64 / kNb tokens (one
// with pages of 64 tokens and more).  One thread looks up the pages, a tile
// ahead, and issues the copies, straight-line: with the page ids in other lanes
// and shuffled, pages of 16 tokens set the pace of the kernel (2,048 rows behind
// 32K, bf16: 1,181 us against 956 with pages of 64).
template <bool kFp8>
struct Producer {
  Ring<kFp8 ? kRaw : Cfg<kFp8>::kSlots> ring;
  bool live = true;
};

// bf16: one slot, two halves of two column blocks of 64 channels x 64 tokens:
// K, the CTA's 64 tokens of all channels; V, its 128 channels of all tokens.
// rows: the boxes' pool rows, K's kNb, V's 2 kNb.
template <int kNb, bool kV>
__device__ __forceinline__ void load_slot(const Ctx& cx, Producer<false>& pr,
                                          uint32_t smem, uint32_t full0,
                                          const CUtensorMap* map, bool tail,
                                          const int (&rows)[kV ? 2 * kNb : kNb]) {
  using C = Cfg<false>;
  const int s = pr.ring.at;
  if ((pr.ring.wrapped &&
       !wait_bar(cx, &cx.bars->empty[s], pr.ring.parity ^ 1)) ||
      *cx.abort) {
    pr.live = false;
    return;
  }
  // A tail's bytes count on each CTA's own barrier, for the warps that write
  // its zeros; the issuer learns of them with P.
  uint32_t full = full0 + s * 8;
  if (tail) {
    const uint32_t own = tc::smem_u32(&cx.bars->tail_full[s]);
    tc::bar_arrive_expect_tx(own, C::kSlotBytes);
    if (cx.rank == 0) tc::bar_arrive(tc::smem_u32(&cx.bars->full[s]));
    full = tc::map_to(own, cx.rank);
  } else if (cx.rank == 0) {
    tc::bar_arrive_expect_tx(tc::smem_u32(&cx.bars->full[s]),
                             2 * C::kSlotBytes);
  }
  const uint32_t dst = smem + C::kOffRing + s * C::kSlotBytes;
  const int x0 = kV ? (int)cx.rank * 128 : 0, x1 = kV ? x0 : 128;
#pragma unroll
  for (int b = 0; b < kNb; ++b) {
    const uint32_t d = dst + b * (kBlockBytes / kNb);
    const int y0 = rows[b], y1 = rows[kV ? kNb + b : b];
    tc::tma_load_2d_pair(d, map, full, x0, y0);
    tc::tma_load_2d_pair(d + kBlockBytes, map, full, x0 + 64, y0);
    tc::tma_load_2d_pair(d + kHalfBytes, map, full, x1, y1);
    tc::tma_load_2d_pair(d + kHalfBytes + kBlockBytes, map, full, x1 + 64, y1);
  }
  pr.ring.next();
}

__device__ __forceinline__ void copy_scales(uint32_t dst, const __half* scales,
                                            int row, int rows, uint32_t full) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(reinterpret_cast<const uint8_t*>(scales) + (long long)row * 8),
      "r"(rows * 8), "r"(full)
      : "memory");
}

// FP8: one staging buffer of 16 KB and its scales.  K: two blocks of 128 bytes
// x 64 tokens; V: the CTA's 128 bytes of 128 tokens, the second 64 in the second
// block.
template <int kNb, bool kV>
__device__ __forceinline__ void load_raw(const Ctx& cx, Producer<true>& pr,
                                         uint32_t smem, const CUtensorMap* map,
                                         const __half* scales,
                                         const int (&rows)[kV ? 2 * kNb : kNb]) {
  using C = Cfg<true>;
  constexpr int kBox = 64 / kNb;
  const int s = pr.ring.at;
  // Once a CTA gives up, its dequant warps release buffers that have not
  // landed; the flag is set before that, and arming a barrier whose bytes are
  // still under way is a fault.
  if ((pr.ring.wrapped &&
       !wait_bar(cx, &cx.bars->raw_empty[s], pr.ring.parity ^ 1)) ||
      *cx.abort) {
    pr.live = false;
    return;
  }
  const uint32_t full = tc::smem_u32(&cx.bars->raw_full[s]);
  tc::bar_arrive_expect_tx(full, 16384 + (kV ? 1024 : 512));
  const uint32_t dst = smem + C::kOffRaw + s * kRawBytes;
  const int x = kV ? (int)cx.rank * 128 : 0;
#pragma unroll
  for (int b = 0; b < kNb; ++b) {
    const uint32_t d = dst + b * (kBox * 128), sc = dst + 16384 + b * (kBox * 8);
    tc::tma_load_2d(d, map, full, x, rows[b]);
    tc::tma_load_2d(d + kBlockBytes, map, full, kV ? x : 128,
                    rows[kV ? kNb + b : b]);
    copy_scales(sc, scales, rows[b], kBox, full);
    if (kV) copy_scales(sc + 512, scales, rows[kNb + b], kBox, full);
  }
  pr.ring.next();
}

// One thread loads the K units of the order K0 K1 V0 K2 V1 .., another the V
// units; both step through the whole ring.
template <bool kFp8, bool kCausal, int kNb, bool kV>
__device__ __forceinline__ void produce_piece(const Ctx& cx, const Piece& pc,
                                              Producer<kFp8>& pr, uint32_t smem,
                                              const CUtensorMap* map) {
  const AttnParams& p = *cx.a;
  constexpr int kIds = kV ? 2 * kNb : kNb, kBox = 64 / kNb;
  const uint32_t full0 = tc::map_to(tc::smem_u32(&cx.bars->full[0]), 0);
  const __half* scales = kV ? p.v_scales : p.k_scales;
  // K: this CTA's 64 tokens of a tile; V: all 128, in two halves
  int t = pc.tok + (kV ? 0 : (int)cx.rank * 64);
  int page[kIds];
#pragma unroll
  for (int b = 0; b < kIds; ++b) page[b] = page_id<kCausal>(p, pc, t + b * kBox);
  const bool tails = kCausal && !kFp8 && kV && pc.tail_tokens() < kT;
  if (kV) pr.ring.next();  // K0
  for (int j = 0; j < pc.n_tiles && pr.live; ++j, t += kT) {
    // V: K of the next tile lies before V of this one; K: V of the tile
    // before the last
    if (kV && j + 1 < pc.n_tiles) pr.ring.next();
    int rows[kIds];
#pragma unroll
    for (int b = 0; b < kIds; ++b)
      rows[b] = pool_row(p, checked_page(p, page[b]), pc.g, t + b * kBox);
    if (j + 1 < pc.n_tiles) {
#pragma unroll
      for (int b = 0; b < kIds; ++b)
        page[b] = page_id<kCausal>(p, pc, t + kT + b * kBox);
    }
    if constexpr (kFp8)
      load_raw<kNb, kV>(cx, pr, smem, map, scales, rows);
    else
      load_slot<kNb, kV>(cx, pr, smem, full0, map, tails && j + 1 == pc.n_tiles,
                         rows);
    if (!kV && j > 0) pr.ring.next();  // V of tile j - 1
  }
  if (!kV) pr.ring.next();  // V of the last tile
}

template <bool kFp8, bool kCausal, bool kV>
__device__ void produce(const Ctx& cx, const Piece& pc, Producer<kFp8>& pr,
                        uint8_t* smem, const CUtensorMap* map) {
  const uint32_t base = tc::smem_u32(smem);
  switch (cx.a->box_rows) {
    case 64: return produce_piece<kFp8, kCausal, 1, kV>(cx, pc, pr, base, map);
    case 32: return produce_piece<kFp8, kCausal, 2, kV>(cx, pc, pr, base, map);
    case 16: return produce_piece<kFp8, kCausal, 4, kV>(cx, pc, pr, base, map);
    default: return produce_piece<kFp8, kCausal, 8, kV>(cx, pc, pr, base, map);
  }
}

// ---- warps 8..15 (FP8): staged bytes to fp16 slots ---------------------------
// A staging buffer makes a slot, two halves of 64 tokens x 128 channels.
// Thread t converts 16-byte chunk c = t & 7 (16 channels) of tokens
// (t >> 3) + 16 e; the two 16-byte stores of lanes c and c + 4 fall into the
// same banks of two column blocks, so the upper half stores its pair in the
// other order.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t pair16, __half2 sc) {
  const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
      static_cast<__nv_fp8x2_storage_t>(pair16), __NV_E4M3);
  const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&hr), sc);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Whether unit k of a piece's K0 K1 V0 K2 V1 .. V(n-1) is a V.
__device__ __forceinline__ bool is_v_unit(int k, int units) {
  return k > 0 && (!(k & 1) || k == units - 1);
}

struct Dequant {
  Ring<kRaw> raw;
  Ring<Cfg<true>::kSlots> slot;
  int turn = 0;  // staging buffers so far
};

// `tokens`: those of the unit that are cached (chunk: the others become zeros).
template <bool kCausal>
__device__ __forceinline__ void dequant_unit(const Ctx& cx, uint8_t* smem,
                                             Dequant& dq, bool is_v,
                                             int tokens) {
  using C = Cfg<true>;
  const int tid = (threadIdx.x - 256) & 127, lane = threadIdx.x & 31;
  const int c = tid & 7, tok0 = tid >> 3;
  const int r = dq.raw.at, s = dq.slot.at;
  // Both sets see every buffer land and release it, the set that converts it
  // after its last read: with two waiters that each look at every other use
  // only, one a lap ahead would take the phase before for its own.  One lane
  // polls: the issuer's thread shares the scheduler.
  if (lane == 0) wait_bar(cx, &cx.bars->raw_full[r], dq.raw.parity);
  __syncwarp();
  if ((dq.turn++ & 1) != (int)(threadIdx.x - 256) >> 7) {  // the other set's
    if (lane == 0) tc::bar_arrive(tc::smem_u32(&cx.bars->raw_empty[r]));
    dq.raw.next();
    dq.slot.next();
    return;
  }
  const uint8_t* raw = smem + C::kOffRaw + r * kRawBytes;
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint4 x[4];
    __half sc[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int tok = tok0 + 16 * e;
      x[e] = *reinterpret_cast<const uint4*>(raw + h * kBlockBytes + tok * 128 +
                                             ((c ^ (tok & 7)) << 4));
      const int at = is_v ? (h * 64 + tok) * 4 + (int)cx.rank * 2 + (c >> 2)
                          : tok * 4 + h * 2 + (c >> 2);
      sc[e] = reinterpret_cast<const __half*>(raw + 16384)[at];
    }
    if (h == 0 && dq.slot.wrapped) {
      if (lane == 0) wait_bar(cx, &cx.bars->empty[s], dq.slot.parity ^ 1);
      __syncwarp();
    }
    uint8_t* out = smem + C::kOffRing + s * C::kSlotBytes + h * kHalfBytes +
                   (c >> 2) * kBlockBytes;
    const int ch = (c & 3) * 2, flip = c >> 2;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int tok = tok0 + 16 * e;
      const __half2 s2 = __halves2half2(sc[e], sc[e]);
      const uint32_t w[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
      uint4 a, b;
      a.x = e4m3x2_to_f16x2(w[0] & 0xFFFF, s2);
      a.y = e4m3x2_to_f16x2(w[0] >> 16, s2);
      a.z = e4m3x2_to_f16x2(w[1] & 0xFFFF, s2);
      a.w = e4m3x2_to_f16x2(w[1] >> 16, s2);
      b.x = e4m3x2_to_f16x2(w[2] & 0xFFFF, s2);
      b.y = e4m3x2_to_f16x2(w[2] >> 16, s2);
      b.z = e4m3x2_to_f16x2(w[3] & 0xFFFF, s2);
      b.w = e4m3x2_to_f16x2(w[3] >> 16, s2);
      if (kCausal && h * 64 + tok >= tokens) a = b = make_uint4(0, 0, 0, 0);
      uint8_t* row = out + tok * 128;
      const int first = ch + flip, second = ch + 1 - flip;
      *reinterpret_cast<uint4*>(row + ((first ^ (tok & 7)) << 4)) = flip ? b : a;
      *reinterpret_cast<uint4*>(row + ((second ^ (tok & 7)) << 4)) = flip ? a : b;
    }
  }
  tc::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tc::bar_arrive(tc::smem_u32(&cx.bars->full[s]));
    tc::bar_arrive(tc::smem_u32(&cx.bars->raw_empty[r]));
  }
  dq.slot.next();
  dq.raw.next();
}

// ---- warp 1 of the leader: MMA issue -----------------------------------------
// A descriptor's low bits are the address in 16-byte steps, so the operands of
// a slot's MMAs are its base descriptor plus constants.  (With the descriptors
// built anew, issuing took 120 to 160 cycles an MMA, more than the 64 and 128
// that the MMAs themselves take.)
template <bool kFp8>
using Slots = Ring<Cfg<kFp8>::kSlots>;

template <bool kFp8>
__device__ __forceinline__ bool wait_slot(const Ctx& cx,
                                          const Slots<kFp8>& seq) {
  if (!wait_bar(cx, &cx.bars->full[seq.at], seq.parity)) return false;
  return !kFp8 ||
         wait_bar<true>(cx, &cx.bars->peer_full[seq.at], seq.parity);
}

template <bool kFp8>
__device__ __forceinline__ bool issue_qk(const Ctx& cx, bool me, Slots<kFp8>& seq,
                                         int gj, uint32_t tmem, uint32_t smem) {
  using C = Cfg<kFp8>;
  const uint32_t d = tmem + kColS + (gj & 1) * kT;
  const uint64_t a = tc::desc_sw128(smem, 16, 1024);
  const uint64_t b = tc::desc_sw128(
      smem + C::kOffRing + seq.at * C::kSlotBytes, 16, 1024);
  if (!wait_slot<kFp8>(cx, seq)) return false;
  tc::fence_after();
#pragma unroll
  for (int k = 0; k < 16; ++k)  // 16 channels each, 64 a column block
    tc::mma_pair(me, d, a + (((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4),
                 b + (((k >> 2) * kBlockBytes + (k & 3) * 32) >> 4),
                 C::kIdescQK, k ? 1u : 0u);
  tc::commit_pair(me, tc::smem_u32(&cx.bars->empty[seq.at]));
  seq.next();
  tc::commit_pair(me, tc::smem_u32(&cx.bars->s_full[gj & 1]));
  return true;
}

// tail: P comes with zeros in V, written by both CTAs.
template <bool kFp8>
__device__ __forceinline__ bool issue_pv(const Ctx& cx, bool me, Slots<kFp8>& seq,
                                         int gj, bool first, bool tail, uint32_t tmem,
                                         uint32_t smem) {
  using C = Cfg<kFp8>;
  uint64_t* p_full = &cx.bars->p_full[gj & 1];
  const uint32_t phase = (uint32_t)(gj >> 1) & 1;
  if (tail ? !wait_bar<true>(cx, p_full, phase) : !wait_bar(cx, p_full, phase))
    return false;
  const uint32_t pt = tmem + kColS + (gj & 1) * kT;
  const uint64_t b = tc::desc_sw128(
      smem + C::kOffRing + seq.at * C::kSlotBytes, kBlockBytes, 1024);
  if (!wait_slot<kFp8>(cx, seq)) return false;
  tc::fence_after();
#pragma unroll
  for (int k = 0; k < 8; ++k)  // 16 tokens each, 64 a half
    tc::mma_pair_ta(me, tmem, pt + k * 8,
                    b + (((k >> 2) * kHalfBytes + (k & 3) * 2048) >> 4),
                    C::kIdescPV, first && k == 0 ? 0u : 1u);
  tc::commit_pair(me, tc::smem_u32(&cx.bars->empty[seq.at]));
  seq.next();
  tc::commit_pair(me, tc::smem_u32(&cx.bars->pv_done[gj & 1]));
  return true;
}

// `then` is called behind the first QK.
template <bool kFp8, bool kCausal, typename F>
__device__ __forceinline__ void mma_piece(const Ctx& cx, const Piece& pc, int gj0,
                                          int n_piece, Slots<kFp8>& seq,
                                          uint32_t tmem, uint8_t* smem_ptr,
                                          F then) {
  const uint32_t smem = tc::smem_u32(smem_ptr);
  const bool me = (threadIdx.x & 31) == 0;
  if (!wait_bar<true>(cx, &cx.bars->q_full, (uint32_t)n_piece & 1)) {
    then();
    return;
  }
  tc::fence_after();
  const bool tails = kCausal && !kFp8 && pc.tail_tokens() < kT;
#pragma unroll (kFp8 ? 1 : 2)
  for (int j = -1; j < pc.n_tiles; ++j) {
    if (j + 1 < pc.n_tiles &&
        !issue_qk<kFp8>(cx, me, seq, gj0 + j + 1, tmem, smem)) {
      if (j < 0) then();
      return;
    }
    if (j < 0) then();
    if (j >= 0 && !issue_pv<kFp8>(cx, me, seq, gj0 + j, j == 0,
                                  tails && j + 1 == pc.n_tiles, tmem, smem))
      return;
  }
}

// FP8, one thread each of two warps of the other CTA: tells the issuer which
// slots its dequant warps have filled.  The dequant warps arrive locally; a
// release at cluster scope waits for more than 1,000 cycles, too long for
// their path and, twice a tile, for one thread.  So one thread releases K's
// slots and the other V's, and each also arrives, without the release, once it
// has seen the other's: the issuer, and with it the slot's next use, waits for
// both, so neither thread can miss a phase.
__device__ void relay_piece(const Ctx& cx, const Piece& pc, Slots<true>& seq,
                            bool v_side) {
  const uint32_t peer0 = tc::map_to(tc::smem_u32(&cx.bars->peer_full[0]), 0);
  const int units = 2 * pc.n_tiles;
#pragma unroll 1
  for (int k = 0; k < units; ++k, seq.next()) {
    if (!wait_bar(cx, &cx.bars->full[seq.at], seq.parity)) return;
    if (is_v_unit(k, units) == v_side)
      tc::arrive_cluster(peer0 + seq.at * 8);
    else
      tc::arrive_cluster_relaxed(peer0 + seq.at * 8);
  }
}

template <bool kCausal>
__device__ void dequant_piece(const Ctx& cx, const Piece& pc, uint8_t* smem,
                              Dequant& dq) {
  // units K0 K1 V0 K2 V1 .. V(n-2) V(n-1): unit 0 and the odd ones but the
  // last are K
  const int units = 2 * pc.n_tiles;
#pragma unroll 1
  for (int k = 0; k < units; ++k) {
    dequant_unit<kCausal>(cx, smem, dq, is_v_unit(k, units),
                          kCausal && k == units - 1 ? pc.tail_tokens() : kT);
  }
}

// ---- warps 4..7: Q, softmax, epilogue ---------------------------------------
// Place of this CTA's row r in q, or -1.
template <bool kCausal>
__device__ __forceinline__ long long q_row(const AttnParams& p, const Piece& pc,
                                           int r) {
  const int R = pc.row0 + r;
  if (R >= pc.rows_total) return -1;
  if (kCausal) {
    const int tok = R / p.group;
    return (((long long)pc.lead * p.q_len + pc.first + tok) * p.hq +
            pc.g * p.group + (R - tok * p.group)) * kHeadDim;
  }
  const int bq = R / p.rows, rb = R - bq * p.rows;
  const int b = pc.start + bq, i = rb / p.group;
  if (i >= block_rows(p, b)) return -1;
  return (((long long)b * p.q_len + i) * p.hq + pc.g * p.group +
          (rb - i * p.group)) * kHeadDim;
}

// Through the registers: a warp writes its 32 rows of Q, one row at a time: lane
// l moves chunk l (8 channels) of the row; bf16 all of them in flight (in the
// registers that the scores leave free), FP8 eight.
template <bool kFp8, bool kCausal>
__device__ __forceinline__ void write_q(const Ctx& cx, const Piece& pc,
                                        uint8_t* smem) {
  const AttnParams& p = *cx.a;
  const int lane = threadIdx.x & 31, w4 = (threadIdx.x >> 5) & 3;
  const long long src = q_row<kCausal>(p, pc, w4 * 32 + lane);
  const int cb = lane >> 3, c = lane & 7;
  constexpr int kRows = kFp8 ? 8 : 32;
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += kRows) {
    uint4 x[kRows];
#pragma unroll
    for (int e = 0; e < kRows; ++e) {
      const long long at = __shfl_sync(0xffffffffu, src, r0 + e);
      x[e] = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.q + at) + lane)
                     : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int e = 0; e < kRows; ++e) {
      const int row = w4 * 32 + r0 + e;
      if (kFp8) {
        uint32_t* v = reinterpret_cast<uint32_t*>(&x[e]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 b2 = *reinterpret_cast<const __nv_bfloat162*>(&v[k]);
          const __half2 h2 = __floats2half2_rn(__low2float(b2), __high2float(b2));
          v[k] = *reinterpret_cast<const uint32_t*>(&h2);
        }
      }
      *reinterpret_cast<uint4*>(smem + cb * (128 * 128) + row * 128 +
                                ((c ^ (row & 7)) << 4)) = x[e];
    }
  }
  tc::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0)
    tc::arrive_cluster(tc::map_to(tc::smem_u32(&cx.bars->q_full), 0));
}

// A chunk's whole tokens by tensor copies, one for each column block of 64
// channels: rows in the order of the tile, in the operand's layout.  (Through the
// registers, the loads in flight have to fit into the 28 KB of L1 that the rings
// leave: 7 us for the 64 KB, behind which every piece started.)  Thread 128 of
// each CTA starts them; bf16, they count on the leader's q_full.
template <bool kFp8>
__device__ __forceinline__ void copy_q(const Ctx& cx, const Piece& pc,
                                       uint8_t* smem) {
  // Without a give-up the last piece's queries have landed; with one they may be
  // under way still, and the barrier is not armed over them.
  if (*cx.abort) return;
  const AttnParams& p = *cx.a;
  const uint32_t bytes = 4 * cx.cta_rows * 128;
  uint32_t bar;
  if (kFp8) {
    bar = tc::smem_u32(&cx.bars->q_land);
    tc::bar_arrive_expect_tx(bar, bytes);
    bar = tc::map_to(bar, cx.rank);
  } else {
    bar = tc::smem_u32(&cx.bars->q_full);
    if (cx.rank == 0) tc::bar_arrive_expect_tx(bar, 2 * bytes);
    bar = tc::map_to(bar, 0);
  }
  const int tok = pc.lead * p.q_len + pc.first + pc.row0 / p.group;
#pragma unroll
  for (int cb = 0; cb < 4; ++cb)
    tc::tma_load_4d_pair(tc::smem_u32(smem) + cb * (128 * 128), cx.tm_q, bar,
                         cb * 64, 0, pc.g, tok);
}

// FP8: the landed bf16 queries to fp16, in place.
__device__ __forceinline__ void convert_q(const Ctx& cx, uint8_t* smem) {
  const int tid = threadIdx.x & 127;
#pragma unroll 4
  for (int i = tid; i < kQBytes / 16; i += 128) {
    uint4* at = reinterpret_cast<uint4*>(smem) + i;
    uint4 x = *at;
    uint32_t* v = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 b2 = *reinterpret_cast<const __nv_bfloat162*>(&v[k]);
      const __half2 h2 = __floats2half2_rn(__low2float(b2), __high2float(b2));
      v[k] = *reinterpret_cast<const uint32_t*>(&h2);
    }
    *at = x;
  }
  tc::fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0)
    tc::arrive_cluster(tc::map_to(tc::smem_u32(&cx.bars->q_full), 0));
}

__device__ __forceinline__ void store8(float* dst, const float* v, float k) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst),
               "f"(v[0] * k), "f"(v[1] * k), "f"(v[2] * k), "f"(v[3] * k),
               "f"(v[4] * k), "f"(v[5] * k), "f"(v[6] * k), "f"(v[7] * k)
               : "memory");
}

// This CTA's half of the last tile's V has landed: thread r makes the row of
// token r zeros if nothing is cached there.
__device__ __forceinline__ void zero_tail(const Ctx& cx, const Piece& pc,
                                          uint8_t* smem, int slot,
                                          uint32_t parity) {
  wait_bar(cx, &cx.bars->tail_full[slot], parity);
  const int r = threadIdx.x & 127;
  if (r >= pc.tail_tokens()) {
    uint8_t* row = smem + Cfg<false>::kOffRing + slot * Cfg<false>::kSlotBytes +
                   (r >> 6) * kHalfBytes + (r & 63) * 128;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      *reinterpret_cast<uint4*>(row + c * 16) = make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(row + kBlockBytes + c * 16) =
          make_uint4(0, 0, 0, 0);
    }
  }
  tc::fence_proxy_async_smem();
}

// Two fused steps, and two additions, in one instruction.
__device__ __forceinline__ float2 fma_pair(float x0, float x1, float a, float b) {
  float2 r;
  asm("{\n\t.reg .b64 x, m, n;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 m, {%4, %4};\n\tmov.b64 n, {%5, %5};\n\t"
      "fma.rn.ftz.f32x2 x, x, m, n;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x0), "f"(x1), "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void add_pair(float& s0, float& s1, float x0,
                                         float x1) {
  asm("{\n\t.reg .b64 s, x;\n\t"
      "mov.b64 s, {%0, %1};\n\tmov.b64 x, {%2, %3};\n\t"
      "add.rn.ftz.f32x2 s, s, x;\n\tmov.b64 {%0, %1}, s;\n\t}"
      : "+f"(s0), "+f"(s1)
      : "f"(x0), "f"(x1));
}

// Scores from column n on count for nothing.
template <int N>
__device__ __forceinline__ void hide(uint32_t* s, int n) {
#pragma unroll
  for (int k = 0; k < N; ++k)
    if (k >= n) s[k] = 0xff800000u;  // -inf
}

// `tails`: the parities of the slots' tail barriers.
template <bool kFp8, bool kCausal>
__device__ void softmax_tiles(const Ctx& cx, const Piece& pc, int gj0,
                              uint32_t tmem, uint8_t* smem, uint32_t& tails,
                              float& m, float& l) {
  using C = Cfg<kFp8>;
  const int lane = threadIdx.x & 31, w4 = (threadIdx.x >> 5) & 3;
  const uint32_t lane_base = tmem + ((uint32_t)(32 * w4) << 16);
  const float sl2 = cx.a->scale_log2;
  m = -INFINITY;
  l = 0.f;
  // tokens of the piece that this row sees, and that the warp's first row does
  int seen = 0, seen0 = 0;
  if (kCausal) {
    const int R = pc.row0 + w4 * 32;
    seen = pc.limit + (R + lane) / cx.a->group - pc.tok;
    seen0 = pc.limit + R / cx.a->group - pc.tok;
  }
  for (int jt = 0; jt < pc.n_tiles; ++jt) {
    const int gj = gj0 + jt;
    const bool masked = kCausal && seen0 < (jt + 1) * kT;
    const uint32_t sbuf = lane_base + kColS + (gj & 1) * kT;
    wait_bar(cx, &cx.bars->s_full[gj & 1], (uint32_t)(gj >> 1) & 1);
    tc::fence_after();
    // 32 columns at a time, read twice, in rolled loops, which fit the instruction
    // cache: ragged shared groups 82.3 us, 86.8 with the tile's scores in registers.
    // Causal bf16 holds them all: its short pieces, whose first tile nothing hides,
    // are faster so (4,096 tokens into an empty cache 144.7 us, 148.8 with 32).
    constexpr int kC = kFp8 || !kCausal ? 32 : kT;
    uint32_t raw[kC];
    const float* s = reinterpret_cast<const float*>(raw);
    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
    for (int c = 0; c < kT; c += kC) {
      tc::tmem_ld_cols<kC>(sbuf + c, raw);
      if (masked) hide<kC>(raw, seen - jt * kT - c);
#pragma unroll
      for (int k = 0; k < kC; ++k) mx4[k & 3] = fmaxf(mx4[k & 3], s[k]);
    }
    const float mx =
        fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
    bool need = false;
    float alpha = 1.f;
    if (jt == 0) {
      m = mx;
    } else if (mx > m + C::kRescaleLog2) {
      need = true;
      alpha = exp2f(m - mx);
      m = mx;
    }
    if (__any_sync(0xffffffffu, need)) {
      // O must be final for the tile before it is rescaled
      wait_bar(cx, &cx.bars->pv_done[(gj - 1) & 1],
               (uint32_t)((gj - 1) >> 1) & 1);
      tc::fence_after();
#pragma unroll 1
      for (int cb = 0; cb < 8; ++cb) {
        uint32_t o[32];
        tc::tmem_ld_cols<32>(lane_base + cb * 32, o);
#pragma unroll
        for (int k = 0; k < 32; ++k)
          o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
        tc::tmem_st_cols<32>(lane_base + cb * 32, o);
      }
      tc::tmem_wait_st();
      l *= alpha;
    }
    const float mu = (m == -INFINITY ? 0.f : m) - C::kShiftLog2;
    float sum4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int c = 0; c < kT; c += kC) {
      if (kC < kT) {
        tc::tmem_ld_cols<kC>(sbuf + c, raw);
        if (masked) hide<kC>(raw, seen - jt * kT - c);
      }
#pragma unroll
      for (int k = 0; k < kC; k += 2) {
        const float2 t = fma_pair(s[k], s[k + 1], sl2, -mu);
        const float x0 = exp2f(t.x), x1 = exp2f(t.y);
        add_pair(sum4[k & 3], sum4[(k & 3) + 1], x0, x1);
        if (kFp8) {
          const __half2 hh = __floats2half2_rn(x0, x1);
          raw[k >> 1] = *reinterpret_cast<const uint32_t*>(&hh);
        } else {
          const __nv_bfloat162 hh = __floats2bfloat162_rn(x0, x1);
          raw[k >> 1] = *reinterpret_cast<const uint32_t*>(&hh);
        }
      }
      // P over columns whose scores have been read
      tc::tmem_st_cols<kC / 2>(sbuf + c / 2, raw);
    }
    l += (sum4[0] + sum4[1]) + (sum4[2] + sum4[3]);
    tc::tmem_wait_st();
    tc::fence_before();
    const uint32_t p_full =
        tc::map_to(tc::smem_u32(&cx.bars->p_full[gj & 1]), 0);
    if (kCausal && !kFp8 && jt + 1 == pc.n_tiles && pc.tail_tokens() < kT) {
      // V of the piece's last tile is its last unit, two a tile
      const int slot = (2 * gj + 1) % C::kSlots;
      zero_tail(cx, pc, smem, slot, tails >> slot & 1);
      tails ^= 1u << slot;
      __syncwarp();
      if (lane == 0) tc::arrive_cluster(p_full);
      continue;
    }
    __syncwarp();
    if (lane == 0) tc::arrive_cluster_relaxed(p_full);
  }
}

__device__ __forceinline__ uint32_t bf16_pair(uint32_t lo, uint32_t hi, float k) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(lo) * k,
                                                 __uint_as_float(hi) * k);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A whole row tile of a chunk: rows to the output.
__device__ void write_out(const Ctx& cx, const Piece& pc, uint32_t tmem, float l) {
  const AttnParams& p = *cx.a;
  const int lane = threadIdx.x & 31, w4 = (threadIdx.x >> 5) & 3;
  const uint32_t lane_base = tmem + ((uint32_t)(32 * w4) << 16);
  const int R = pc.row0 + w4 * 32 + lane;
  const bool valid = w4 * 32 + lane < cx.cta_rows && R < pc.rows_total;
  const int tok = R / p.group;
  // out is 16-byte aligned; stores of 32 bytes, where they fit, take 5 us from 4,096
  // tokens into an empty cache (160 us with 16 bytes)
  const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
  __nv_bfloat16* dst =
      p.out + (((long long)pc.lead * p.q_len + pc.first + tok) * p.hq +
               pc.g * p.group + (R - tok * p.group)) * kHeadDim;
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
  for (int cb = 0; cb < 4; ++cb) {
    uint32_t o[64];
    tc::tmem_ld_cols<64>(lane_base + cb * 64, o);
    if (valid) {
#pragma unroll
      for (int k = 0; k < 64; k += 16) {
        uint32_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[e] = bf16_pair(o[k + 2 * e], o[k + 2 * e + 1], inv);
        __nv_bfloat16* to = dst + cb * 64 + k;
        if (wide) {
          asm volatile(
              "st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to),
              "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
              "r"(v[6]), "r"(v[7])
              : "memory");
        } else {
          reinterpret_cast<uint4*>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<uint4*>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
        }
      }
    }
  }
  tc::fence_before();  // the reads precede this warp's next P
}

// `shift`: the factor (log2) that O and l carry.
__device__ void epilogue(const Ctx& cx, const Piece& pc, uint32_t tmem, float m,
                         float l, float shift) {
  const int lane = threadIdx.x & 31, w4 = (threadIdx.x >> 5) & 3;
  const uint32_t lane_base = tmem + ((uint32_t)(32 * w4) << 16);
  const int r = w4 * 32 + lane;
  const bool valid = r < cx.cta_rows && pc.row0 + r < pc.rows_total;
  const long long row =
      (long long)pc.slot * kPrefixRows + cx.rank * 128 + r;
  float* dst = cx.pre_o + row * kHeadDim;
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll 1
  for (int cb = 0; cb < 4; ++cb) {
    uint32_t o[64];
    tc::tmem_ld_cols<64>(lane_base + cb * 64, o);
    if (valid) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        store8(dst + cb * 64 + 8 * k,
               reinterpret_cast<const float*>(o) + 8 * k, inv);
    }
  }
  if (valid)
    cx.pre_lse[row] =
        l > 0.f ? (m == -INFINITY ? 0.f : m) - shift + log2f(l) : -INFINITY;
  tc::fence_before();  // the reads precede this warp's next P
}

__device__ __forceinline__ Piece decode_piece(const SharedParams& p, int i,
                                              uint32_t rank) {
  int lo = 0, hi = p.groups - 1;  // the last group that starts at or before i
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.plan[mid].piece0 <= i) lo = mid; else hi = mid - 1;
  }
  const GroupPlan gp = p.plan[lo];
  const int in = i - gp.piece0, run = in / gp.tiles;
  const int c = run % gp.splits;
  const int j0 = run_start(gp, c), j1 = run_start(gp, c + 1);
  Piece pc;
  pc.lead = gp.lead;
  pc.start = gp.start;
  pc.rows_total = gp.count * p.a.rows;
  pc.g = run / gp.splits;
  pc.row0 = (in - run * gp.tiles) * kPrefixRows + (int)rank * 128;
  pc.tok = j0 * kT;
  pc.n_tiles = j1 - j0;
  pc.slot = i;
  return pc;
}

// The pieces of a CTA pair: groups' shared prefixes, numbered i, i + pairs, ..
struct PrefixWork {
  const SharedParams& p;
  uint32_t rank;
  int i, pieces;
  __device__ PrefixWork(const SharedParams& p, uint32_t rank)
      : p(p), rank(rank), i(blockIdx.x >> 1), pieces(p.plan[p.groups].piece0) {}
  __device__ __forceinline__ bool next(Piece& pc) {
    if (i >= pieces) return false;
    pc = decode_piece(p, i, rank);
    i += gridDim.x >> 1;
    return true;
  }
};

// A chunk's: whole row tiles in rounds, then the pair's run of the rest.
struct ChunkWork {
  const ChunkParams& p;
  uint32_t rank;
  ChunkHead h;
  ChunkRun run;
  int pair, round;
  __device__ ChunkWork(const ChunkParams& p, uint32_t rank)
      : p(p), rank(rank), h(*p.head), run(p.runs[blockIdx.x >> 1]),
        pair(blockIdx.x >> 1), round(0) {}
  __device__ __forceinline__ bool next(Piece& pc) {
    const int at = round & 1 ? p.pairs - 1 - pair : pair;
    const bool whole =
        round < h.rounds || (!h.split && round == h.rounds && at < h.rest);
    if (!whole && !(h.split && run.tiles)) return false;
    const ChunkPiece e =
        p.pieces[(long long)(whole ? round : h.rounds) * p.pairs +
                 (whole ? at : run.piece)];
    const int slot0 = whole ? 0 : p.rest[run.piece].x;
    int from = 0, to = e.tiles;
    pc.slot = -1;
    if (whole) {
      ++round;
    } else {
      from = run.from;
      to = min(to, from + run.tiles);
      // its first run's slot is the piece's first
      if (from) pc.slot = run.slot;
      else if (to < e.tiles) pc.slot = slot0;
      ++run.piece;
      run.tiles -= to - from;
      run.from = 0;
    }
    pc.lead = pc.start = e.b;
    pc.rows_total = e.rows;
    pc.g = e.g;
    pc.row0 = e.row0 + (int)rank * p.cta_rows;
    pc.tok = from * kT;
    pc.n_tiles = to - from;
    pc.last = e.last;
    pc.first = e.first;
    pc.limit = e.limit;
    return true;
  }
};

template <bool kFp8, bool kCausal>
__global__ void __cluster_dims__(2, 1, 1)
    __launch_bounds__(Cfg<kFp8>::kThreads, 1)
        prefix_attention_kernel(
            const __grid_constant__
                std::conditional_t<kCausal, ChunkParams, SharedParams> p,
            const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_v,
            const __grid_constant__ CUtensorMap tm_q) {
  using Work = std::conditional_t<kCausal, ChunkWork, PrefixWork>;
  using C = Cfg<kFp8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
      ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) Bars bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = tc::cluster_rank();

  int cta_rows = 128, q_tokens = 0;
  if constexpr (kCausal) {
    cta_rows = p.cta_rows;
    q_tokens = p.q_tokens;
  }
  if (tid == 0) {
    for (int s = 0; s < C::kSlots; ++s) {
      // bf16: the leader's expect_tx plus both CTAs' bytes; FP8: the four
      // dequant warps, and the other CTA's two relays
      tc::bar_init(tc::smem_u32(&bars.full[s]), kFp8 ? 4 : 1);
      tc::bar_init(tc::smem_u32(&bars.peer_full[s]), 2);
      tc::bar_init(tc::smem_u32(&bars.empty[s]), 1);
      tc::bar_init(tc::smem_u32(&bars.tail_full[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::bar_init(tc::smem_u32(&bars.s_full[s]), 1);
      tc::bar_init(tc::smem_u32(&bars.p_full[s]), 8);
      tc::bar_init(tc::smem_u32(&bars.pv_done[s]), 1);
    }
    // Q by tensor copies to both CTAs: the leader's expect_tx; otherwise the
    // warps that wrote or converted it
    tc::bar_init(tc::smem_u32(&bars.q_full), !kFp8 && q_tokens ? 1 : 8);
    tc::bar_init(tc::smem_u32(&bars.q_land), 1);
    for (int s = 0; s < kRaw; ++s) {
      tc::bar_init(tc::smem_u32(&bars.raw_full[s]), 1);
      tc::bar_init(tc::smem_u32(&bars.raw_empty[s]), 8);
    }
    tc::bar_init(tc::smem_u32(&bars.drain), 1);
    s_abort = 0;
    tc::bar_fence_init();
  }
  if (warp == 1) tc::tmem_alloc_pair(tc::smem_u32(&s_tmem), kTmemCols);
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();  // both CTAs' barriers and tensor memory are ready
  tc::fence_after();
  const uint32_t tmem = s_tmem;
  // The set-up ran beside the plan kernel, which writes what is read from
  // here on.  The tails' kernel is released only now: what follows it may then
  // take the plan as written.
  tc_grid_dependency_wait();
  tc_grid_launch_dependents();
  const Ctx cx{&bars, &s_abort,
               tc::map_to(tc::smem_u32(&s_abort), rank ^ 1u), rank, &p.a,
               p.pre_o, p.pre_lse, &tm_q, cta_rows, q_tokens};

  // Every role walks the pair's pieces by itself.
  Work work(p, rank);
  int gj0 = 0;
  if (warp < 4) {
    Producer<kFp8> pr;
    Slots<kFp8> seq;
    int n_piece = 0;
    Piece pc, nx;
    bool more = work.next(pc);
    for (; more; ++n_piece) {
      if (warp == 1 && rank == 0) {
        // the next piece's numbers are on their way before they are needed
        mma_piece<kFp8, kCausal>(cx, pc, gj0, n_piece, seq, tmem, smem,
                                 [&] { more = work.next(nx); });
      } else {
        if (lane == 0) {
          if (warp == 0 && pr.live)
            produce<kFp8, kCausal, false>(cx, pc, pr, smem, &tm_k);
          if (warp == 2 && pr.live)
            produce<kFp8, kCausal, true>(cx, pc, pr, smem, &tm_v);
          if constexpr (kFp8) {
            if (rank == 1 && (warp & 1)) relay_piece(cx, pc, seq, warp == 3);
          }
        }
        __syncwarp();
        more = work.next(nx);
      }
      gj0 += pc.n_tiles;
      pc = nx;
    }
  } else if (warp < 8) {
    float m = 0.f, l = 0.f;
    Piece prev{};
    uint32_t tails = 0;
    int n_piece = 0;
    while (true) {
      Piece pc{};
      const bool more = work.next(pc);
      // These warps have seen the last QK of the piece before: Q may be replaced,
      // under that piece's last PV.
      if (more) {
        if (!kCausal || !q_tokens)
          write_q<kFp8, kCausal>(cx, pc, smem);
        else if (tid == 128)
          copy_q<kFp8>(cx, pc, smem);
      }
      if (gj0) {
        // the last piece's MMAs are done: O may be read
        wait_bar(cx, &bars.pv_done[(gj0 - 1) & 1],
                 (uint32_t)((gj0 - 1) >> 1) & 1);
        tc::fence_after();
        if (kCausal && prev.slot < 0)
          write_out(cx, prev, tmem, l);
        else
          epilogue(cx, prev, tmem, m, l, C::kShiftLog2);
      }
      if (!more) break;
      if (kFp8 && kCausal && q_tokens) {
        wait_bar(cx, &bars.q_land, (uint32_t)n_piece++ & 1);
        convert_q(cx, smem);
      }
      softmax_tiles<kFp8, kCausal>(cx, pc, gj0, tmem, smem, tails, m, l);
      prev = pc;
      gj0 += pc.n_tiles;
    }
  } else if constexpr (kFp8) {
    Dequant dq;
    Piece pc;
    while (work.next(pc)) dequant_piece<kCausal>(cx, pc, smem, dq);
  }

  // teardown: no copy or MMA may still be in flight in either CTA.  Every
  // load was consumed by an MMA, and every MMA completes before drain.
  if (warp == 1 && rank == 0) {
    tc::commit_pair(lane == 0, tc::smem_u32(&bars.drain));
    wait_bar(cx, &bars.drain, 0, true);
    __syncwarp();
  }
  tc::fence_before();
  __syncthreads();
  if (s_abort) {
    // a wait ran out: loads that no MMA waited for land within microseconds
    const long long t0 = clock64();
    while (clock64() - t0 < 4000000LL) {
    }
  }
  tc::cluster_sync();
  tc::fence_after();
  if (warp == 1) tc::tmem_dealloc_pair(tmem, kTmemCols);
  tc::cluster_sync();  // neither CTA leaves while the other frees
}

template <bool kFp8, bool kCausal>
int pairs_resident() {
  using C = Cfg<kFp8>;
  if (cudaFuncSetAttribute(prefix_attention_kernel<kFp8, kCausal>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           C::kSmem) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, prefix_attention_kernel<kFp8, kCausal>, &cfg) !=
      cudaSuccess)
    return 0;
  return n;
}

template <bool kFp8, bool kCausal, typename P>
cudaError_t launch(const P& p, const CUtensorMap& tm_k,
                   const CUtensorMap& tm_v, const CUtensorMap& tm_q,
                   cudaStream_t s) {
  using C = Cfg<kFp8>;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(2 * p.pairs), dim3(C::kThreads), C::kSmem, s, attr);
  return cudaLaunchKernelEx(&cfg, prefix_attention_kernel<kFp8, kCausal>, p,
                            tm_k, tm_v, tm_q);
}

}  // namespace

cudaError_t launch_prefix_attention(const SharedParams& p,
                                    const CUtensorMap& tm_k,
                                    const CUtensorMap& tm_v, cudaStream_t s) {
  return p.a.k_scales ? launch<true, false>(p, tm_k, tm_v, tm_k, s)
                      : launch<false, false>(p, tm_k, tm_v, tm_k, s);
}

cudaError_t launch_chunk_attention(const ChunkParams& p,
                                   const CUtensorMap& tm_k,
                                   const CUtensorMap& tm_v,
                                   const CUtensorMap& tm_q, cudaStream_t s) {
  return p.a.k_scales ? launch<true, true>(p, tm_k, tm_v, tm_q, s)
                      : launch<false, true>(p, tm_k, tm_v, tm_q, s);
}

int prefix_attention_pairs(bool fp8) {
  return fp8 ? pairs_resident<true, false>() : pairs_resident<false, false>();
}

int chunk_attention_pairs(bool fp8) {
  return fp8 ? pairs_resident<true, true>() : pairs_resident<false, true>();
}

}  // namespace specv
