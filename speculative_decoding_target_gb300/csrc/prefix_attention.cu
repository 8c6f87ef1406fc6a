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
// shared tokens, 206 Gflop: 121-126 us, 1.64 to 1.70 Pflop/s, 0.86 to 0.89 of
// the measured bf16 rate; the tensor pipe is busy 77% of the time, DRAM reads
// 137.5 MB of the prefix's 134.2.  What is left is the first and last tile of
// each piece and the issuer's waits on the softmax.  FP8, 64 single tokens over
// 65,536, 103 Gflop: 121 us, 0.45 of that rate; the conversion of E4M3 to fp16
// through shared memory bounds it (issue slots 54% busy, the tensor pipe 52%).
//
// Every wait is bounded as in verify_attention_tc.cu.
#include <cuda_fp8.h>

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
  uint64_t raw_full[kRaw];     // FP8, own: staged bytes landed
  uint64_t raw_empty[kRaw];    // FP8, own: staged bytes converted
  uint64_t drain;              // both: every MMA issued is done
};

struct Ctx {
  Bars* bars;
  volatile int* abort;
  uint32_t peer_abort;         // cluster address of the other CTA's flag
  uint32_t rank;
  const SharedParams* p;
};

__device__ __forceinline__ void give_up(const Ctx& cx) {
  *cx.abort = 1;
  tc::store_cluster(cx.peer_abort, 1u);
  if (cx.p->a.status) atomicOr(cx.p->a.status, SPEC_STATUS_TIMEOUT);
}

// Barriers that carry generic writes of the other CTA (Q, dequantised tiles)
// are waited for at cluster scope; the others carry tensor-memory or TMA
// completions.
template <bool kCluster>
__device__ __noinline__ bool wait_slow(const Ctx& cx, uint32_t a,
                                       uint32_t parity, bool drain) {
  if (!drain && *cx.abort) return false;
  const long long bound = drain ? kDrainWaitCycles : cx.p->a.wait_cycles;
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
  int slot;                     // partial slot
};

__device__ __forceinline__ int page_id(const AttnParams& p, int lead, int t) {
  return __ldg(p.page_table + (long long)lead * p.max_pages + (t >> p.log2_ps));
}
// Looked at only when the page is used, so that the load of the id runs ahead.
__device__ __forceinline__ int checked_page(const AttnParams& p, int page) {
  if (page < 0 || page >= p.num_pages) {
    if (p.status) atomicOr(p.status, SPEC_STATUS_BAD_PAGE);
    page = 0;  // in bounds; the affected rows are unspecified
  }
  return page;
}

__device__ __forceinline__ long long pool_row(const AttnParams& p, int page,
                                              int g, int t) {
  return ((long long)(page * p.hkv + g) << p.log2_ps) + (t & (p.page_size - 1));
}

// ---- warp 0: loads ----------------------------------------------------------
// A half of 64 tokens is 64 / box_rows boxes of each column block.  With whole
// boxes (pages of 64 tokens and more, kOne) lane 0 works alone; otherwise lane
// b looks up the pages of box b, and lane 0 issues the copies, so that a copy's
// operands are uniform.  (Two lanes issuing a box each, with 64-bit ring
// arithmetic, took 900 cycles a slot and set the pace of the kernel.)
template <bool kFp8>
struct Producer {
  Ring<kFp8 ? kRaw : Cfg<kFp8>::kSlots> ring;
  bool live = true;
};

template <bool kOne>
__device__ __forceinline__ long long box_row(long long row, int b) {
  return kOne ? row : __shfl_sync(0xffffffffu, row, b);
}
template <bool kOne>
__device__ __forceinline__ bool all_lanes(bool ok) {
  return kOne ? ok : __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
}

// bf16: one slot, two halves of two column blocks of 64 channels x 64 tokens:
// K, the CTA's 64 tokens of all channels (row1 = row0); V, its 128 channels of
// all tokens.
template <bool kOne>
__device__ __forceinline__ void load_slot(const Ctx& cx, Producer<false>& pr,
                                          uint32_t smem, uint32_t full0,
                                          const CUtensorMap* map, bool is_v,
                                          long long row0, long long row1,
                                          int nb, int rpb) {
  using C = Cfg<false>;
  const int s = pr.ring.at;
  const bool leads = kOne || (threadIdx.x & 31) == 0;
  bool ok = true;
  if (leads && pr.ring.wrapped)
    ok = wait_bar(cx, &cx.bars->empty[s], pr.ring.parity ^ 1);
  ok = all_lanes<kOne>(ok && !*cx.abort);
  if (!ok) {
    pr.live = false;
    return;
  }
  if (leads && cx.rank == 0)
    tc::bar_arrive_expect_tx(tc::smem_u32(&cx.bars->full[s]),
                             2 * C::kSlotBytes);
  const uint32_t dst = smem + C::kOffRing + s * C::kSlotBytes;
  const uint32_t full = full0 + s * 8;
  const int x0 = is_v ? (int)cx.rank * 128 : 0;
  const int x1 = is_v ? x0 : 128;
  for (int b = 0; b < nb; ++b) {
    const int y0 = (int)box_row<kOne>(row0, b);
    const int y1 = (int)box_row<kOne>(row1, b);
    if (leads) {
      const uint32_t d = dst + b * rpb * 128;
      tc::tma_load_2d_pair(d, map, full, x0, y0);
      tc::tma_load_2d_pair(d + kBlockBytes, map, full, x0 + 64, y0);
      tc::tma_load_2d_pair(d + kHalfBytes, map, full, x1, y1);
      tc::tma_load_2d_pair(d + kHalfBytes + kBlockBytes, map, full, x1 + 64, y1);
    }
  }
  pr.ring.next();
}

__device__ __forceinline__ void copy_scales(uint32_t dst, const __half* scales,
                                            long long row, int rows,
                                            uint32_t full) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(reinterpret_cast<const uint8_t*>(scales) + row * 8), "r"(rows * 8),
      "r"(full)
      : "memory");
}

// FP8: one staging buffer of 16 KB and its scales.  K: two blocks of 128 bytes
// x 64 tokens; V: the CTA's 128 bytes of 128 tokens, the second 64 (row1) in
// the second block.
template <bool kOne>
__device__ __forceinline__ void load_raw(const Ctx& cx, Producer<true>& pr,
                                         uint32_t smem, const CUtensorMap* map,
                                         const __half* scales, bool is_v,
                                         long long row0, long long row1, int nb,
                                         int rpb) {
  using C = Cfg<true>;
  const int s = pr.ring.at;
  const bool leads = kOne || (threadIdx.x & 31) == 0;
  bool ok = true;
  if (leads && pr.ring.wrapped)
    ok = wait_bar(cx, &cx.bars->raw_empty[s], pr.ring.parity ^ 1);
  // Once a CTA gives up, its dequant warps release buffers that have not
  // landed; the flag is set before that, and arming a barrier whose bytes are
  // still under way is a fault.
  ok = all_lanes<kOne>(ok && !*cx.abort);
  if (!ok) {
    pr.live = false;
    return;
  }
  const uint32_t full = tc::smem_u32(&cx.bars->raw_full[s]);
  if (leads) tc::bar_arrive_expect_tx(full, 16384 + (is_v ? 1024 : 512));
  const uint32_t dst = smem + C::kOffRaw + s * kRawBytes;
  for (int b = 0; b < nb; ++b) {
    const long long y0 = box_row<kOne>(row0, b), y1 = box_row<kOne>(row1, b);
    if (leads) {
      const int x = is_v ? (int)cx.rank * 128 : 0;
      const uint32_t o = b * rpb;
      tc::tma_load_2d(dst + o * 128, map, full, x, (int)y0);
      tc::tma_load_2d(dst + kBlockBytes + o * 128, map, full,
                      is_v ? x : 128, (int)(is_v ? y1 : y0));
      copy_scales(dst + 16384 + o * 8, scales, y0, rpb, full);
      if (is_v) copy_scales(dst + 16384 + (64 + o) * 8, scales, y1, rpb, full);
    }
  }
  pr.ring.next();
}

// One warp loads the K units of the order K0 K1 V0 K2 V1 .., another the V
// units (with pages of 16 tokens a unit is 16 copies, more than one warp
// issues in a tile's time); both step through the whole ring.
template <bool kFp8, bool kOne>
__device__ __forceinline__ void produce_piece(const Ctx& cx, const Piece& pc,
                                              Producer<kFp8>& pr, uint32_t smem,
                                              const CUtensorMap* map,
                                              bool v_side) {
  const AttnParams& p = cx.p->a;
  const int lane = threadIdx.x & 31;
  const int rpb = p.box_rows, nb = kOne ? 1 : 64 / rpb;
  const uint32_t full0 = tc::map_to(tc::smem_u32(&cx.bars->full[0]), 0);
  const __half* scales = v_side ? p.v_scales : p.k_scales;
  // K: this CTA's 64 tokens of a tile; V: all 128, in two halves
  const int t0 = pc.tok + (kOne ? 0 : (lane & (nb - 1)) * rpb) +
                 (v_side ? 0 : (int)cx.rank * 64);
  int page0 = page_id(p, pc.lead, t0);
  int page1 = v_side ? page_id(p, pc.lead, t0 + 64) : 0;
  if (v_side) pr.ring.next();  // K0
  for (int j = 0; j < pc.n_tiles && pr.live; ++j) {
    // V: K of the next tile lies before V of this one; K: V of the tile
    // before the last
    if (v_side && j + 1 < pc.n_tiles) pr.ring.next();
    const int t = t0 + j * kT;
    const long long r0 = pool_row(p, checked_page(p, page0), pc.g, t);
    const long long r1 =
        v_side ? pool_row(p, checked_page(p, page1), pc.g, t + 64) : r0;
    if (j + 1 < pc.n_tiles) {
      page0 = page_id(p, pc.lead, t + kT);
      if (v_side) page1 = page_id(p, pc.lead, t + kT + 64);
    }
    if constexpr (kFp8)
      load_raw<kOne>(cx, pr, smem, map, scales, v_side, r0, r1, nb, rpb);
    else
      load_slot<kOne>(cx, pr, smem, full0, map, v_side, r0, r1, nb, rpb);
    if (!v_side && j > 0) pr.ring.next();  // V of tile j - 1
  }
  if (!v_side) pr.ring.next();  // V of the last tile
}

template <bool kFp8>
__device__ void produce(const Ctx& cx, const Piece& pc, Producer<kFp8>& pr,
                        uint8_t* smem, const CUtensorMap* map, bool v_side) {
  const uint32_t base = tc::smem_u32(smem);
  if (cx.p->a.box_rows == 64) {
    if ((threadIdx.x & 31) == 0)
      produce_piece<kFp8, true>(cx, pc, pr, base, map, v_side);
  } else {
    produce_piece<kFp8, false>(cx, pc, pr, base, map, v_side);
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

__device__ __forceinline__ void dequant_unit(const Ctx& cx, uint8_t* smem,
                                             Dequant& dq, bool is_v) {
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

__device__ void dequant_piece(const Ctx& cx, const Piece& pc, uint8_t* smem,
                              Dequant& dq) {
  // units K0 K1 V0 K2 V1 .. V(n-2) V(n-1): unit 0 and the odd ones but the
  // last are K
  const int units = 2 * pc.n_tiles;
#pragma unroll 1
  for (int k = 0; k < units; ++k)
    dequant_unit(cx, smem, dq, is_v_unit(k, units));
}

// ---- warp 1 of the leader, one thread: MMA issue ----------------------------
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
__device__ __forceinline__ bool issue_qk(const Ctx& cx, Slots<kFp8>& seq, int gj,
                                         uint32_t tmem, uint32_t smem) {
  using C = Cfg<kFp8>;
  const uint32_t d = tmem + kColS + (gj & 1) * kT;
  const uint64_t a = tc::desc_sw128(smem, 16, 1024);
  const uint64_t b = tc::desc_sw128(
      smem + C::kOffRing + seq.at * C::kSlotBytes, 16, 1024);
  if (!wait_slot<kFp8>(cx, seq)) return false;
  tc::fence_after();
#pragma unroll
  for (int k = 0; k < 16; ++k)  // 16 channels each, 64 a column block
    tc::mma_pair(d, a + (((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4),
                 b + (((k >> 2) * kBlockBytes + (k & 3) * 32) >> 4),
                 C::kIdescQK, k ? 1u : 0u);
  tc::commit_pair(tc::smem_u32(&cx.bars->empty[seq.at]));
  seq.next();
  tc::commit_pair(tc::smem_u32(&cx.bars->s_full[gj & 1]));
  return true;
}

template <bool kFp8>
__device__ __forceinline__ bool issue_pv(const Ctx& cx, Slots<kFp8>& seq, int gj,
                                         bool first, uint32_t tmem,
                                         uint32_t smem) {
  using C = Cfg<kFp8>;
  if (!wait_bar(cx, &cx.bars->p_full[gj & 1], (uint32_t)(gj >> 1) & 1))
    return false;
  const uint32_t pt = tmem + kColS + (gj & 1) * kT;
  const uint64_t b = tc::desc_sw128(
      smem + C::kOffRing + seq.at * C::kSlotBytes, kBlockBytes, 1024);
  if (!wait_slot<kFp8>(cx, seq)) return false;
  tc::fence_after();
#pragma unroll
  for (int k = 0; k < 8; ++k)  // 16 tokens each, 64 a half
    tc::mma_pair_ta(tmem, pt + k * 8,
                    b + (((k >> 2) * kHalfBytes + (k & 3) * 2048) >> 4),
                    C::kIdescPV, first && k == 0 ? 0u : 1u);
  tc::commit_pair(tc::smem_u32(&cx.bars->empty[seq.at]));
  seq.next();
  tc::commit_pair(tc::smem_u32(&cx.bars->pv_done[gj & 1]));
  return true;
}

template <bool kFp8>
__device__ void mma_piece(const Ctx& cx, const Piece& pc, int gj0, int n_piece,
                          Slots<kFp8>& seq, uint32_t tmem, uint8_t* smem_ptr) {
  const uint32_t smem = tc::smem_u32(smem_ptr);
  if (!wait_bar<true>(cx, &cx.bars->q_full, (uint32_t)n_piece & 1)) return;
  tc::fence_after();
#pragma unroll (kFp8 ? 1 : 2)
  for (int j = -1; j < pc.n_tiles; ++j) {
    if (j + 1 < pc.n_tiles &&
        !issue_qk<kFp8>(cx, seq, gj0 + j + 1, tmem, smem))
      return;
    if (j >= 0 && !issue_pv<kFp8>(cx, seq, gj0 + j, j == 0, tmem, smem)) return;
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

// ---- warps 4..7: Q, softmax, epilogue ---------------------------------------
// A warp writes its 32 rows of Q, one row at a time: lane l moves chunk l (8
// channels) of the row, eight rows in flight.
template <bool kFp8>
__device__ void write_q(const Ctx& cx, const Piece& pc, uint8_t* smem) {
  const AttnParams& p = cx.p->a;
  const int lane = threadIdx.x & 31, w4 = (threadIdx.x >> 5) & 3;
  // this lane's row: its place in q, or -1
  const int R = pc.row0 + w4 * 32 + lane;
  long long src = -1;
  if (R < pc.rows_total) {
    const int bq = R / p.rows, r = R - bq * p.rows;
    const int b = pc.start + bq, i = r / p.group;
    if (i < block_rows(p, b))
      src = (((long long)b * p.q_len + i) * p.hq + pc.g * p.group +
             (r - i * p.group)) * kHeadDim;
  }
  const int cb = lane >> 3, c = lane & 7;
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += 8) {
    uint4 x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const long long at = __shfl_sync(0xffffffffu, src, r0 + e);
      x[e] = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.q + at) + lane)
                     : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
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

__device__ __forceinline__ void store8(float* dst, const float* v, float k) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst),
               "f"(v[0] * k), "f"(v[1] * k), "f"(v[2] * k), "f"(v[3] * k),
               "f"(v[4] * k), "f"(v[5] * k), "f"(v[6] * k), "f"(v[7] * k)
               : "memory");
}

template <bool kFp8>
__device__ void softmax_tiles(const Ctx& cx, const Piece& pc, int gj0,
                              uint32_t tmem, float& m, float& l) {
  using C = Cfg<kFp8>;
  const int lane = threadIdx.x & 31, w4 = (threadIdx.x >> 5) & 3;
  const uint32_t lane_base = tmem + ((uint32_t)(32 * w4) << 16);
  const float sl2 = cx.p->a.scale_log2;
  m = -INFINITY;
  l = 0.f;
  for (int jt = 0; jt < pc.n_tiles; ++jt) {
    const int gj = gj0 + jt;
    const uint32_t sbuf = lane_base + kColS + (gj & 1) * kT;
    wait_bar(cx, &cx.bars->s_full[gj & 1], (uint32_t)(gj >> 1) & 1);
    tc::fence_after();
    // bf16: the tile's scores in registers; FP8: 32 columns at a time, read
    // twice, in rolled loops
    constexpr int kC = kFp8 ? 32 : kT;
    uint32_t raw[kC];
    const float* s = reinterpret_cast<const float*>(raw);
    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
    for (int c = 0; c < kT; c += kC) {
      tc::tmem_ld_cols<kC>(sbuf + c, raw);
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
      if (kFp8) tc::tmem_ld_cols<kC>(sbuf + c, raw);
#pragma unroll
      for (int k = 0; k < kC; k += 2) {
        const float x0 = exp2f(fmaf(s[k], sl2, -mu));
        const float x1 = exp2f(fmaf(s[k + 1], sl2, -mu));
        sum4[k & 3] += x0;
        sum4[(k & 3) + 1] += x1;
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
    __syncwarp();
    if (lane == 0)
      tc::arrive_cluster_relaxed(
          tc::map_to(tc::smem_u32(&cx.bars->p_full[gj & 1]), 0));
  }
}

// `shift`: the factor (log2) that O and l carry.
__device__ void epilogue(const Ctx& cx, const Piece& pc, uint32_t tmem, float m,
                         float l, float shift) {
  const int lane = threadIdx.x & 31, w4 = (threadIdx.x >> 5) & 3;
  const uint32_t lane_base = tmem + ((uint32_t)(32 * w4) << 16);
  const int r = w4 * 32 + lane;
  const bool valid = pc.row0 + r < pc.rows_total;
  const long long row =
      (long long)pc.slot * kPrefixRows + cx.rank * 128 + r;
  float* dst = cx.p->pre_o + row * kHeadDim;
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
    cx.p->pre_lse[row] =
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

template <bool kFp8>
__global__ void __cluster_dims__(2, 1, 1)
    __launch_bounds__(Cfg<kFp8>::kThreads, 1)
        prefix_attention_kernel(const __grid_constant__ SharedParams p,
                                const __grid_constant__ CUtensorMap tm_k,
                                const __grid_constant__ CUtensorMap tm_v) {
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

  if (tid == 0) {
    for (int s = 0; s < C::kSlots; ++s) {
      // bf16: the leader's expect_tx plus both CTAs' bytes; FP8: the four
      // dequant warps, and the other CTA's two relays
      tc::bar_init(tc::smem_u32(&bars.full[s]), kFp8 ? 4 : 1);
      tc::bar_init(tc::smem_u32(&bars.peer_full[s]), 2);
      tc::bar_init(tc::smem_u32(&bars.empty[s]), 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::bar_init(tc::smem_u32(&bars.s_full[s]), 1);
      tc::bar_init(tc::smem_u32(&bars.p_full[s]), 8);
      tc::bar_init(tc::smem_u32(&bars.pv_done[s]), 1);
    }
    tc::bar_init(tc::smem_u32(&bars.q_full), 8);
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
  const int pieces = p.plan[p.groups].piece0;
  const Ctx cx{&bars, &s_abort,
               tc::map_to(tc::smem_u32(&s_abort), rank ^ 1u), rank, &p};

  // Every role walks the pair's pieces by itself.
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;
  if (warp < 4) {
    Producer<kFp8> pr;
    Slots<kFp8> seq;
    int gj0 = 0, n_piece = 0;
    for (int i = first; i < pieces; i += step, ++n_piece) {
      const Piece pc = decode_piece(p, i, rank);
      if (warp == 0 || warp == 2) {
        const bool v_side = warp != 0;
        if (pr.live)
          produce<kFp8>(cx, pc, pr, smem, v_side ? &tm_v : &tm_k, v_side);
      } else if (lane == 0) {
        if (rank == 0 && warp == 1)
          mma_piece<kFp8>(cx, pc, gj0, n_piece, seq, tmem, smem);
        if constexpr (kFp8) {
          if (rank == 1) relay_piece(cx, pc, seq, warp == 3);
        }
      }
      __syncwarp();
      gj0 += pc.n_tiles;
    }
  } else if (warp < 8) {
    float m = 0.f, l = 0.f;
    Piece prev{};
    int gj0 = 0;
    for (int i = first;; i += step) {
      const bool more = i < pieces;
      Piece pc{};
      if (more) pc = decode_piece(p, i, rank);
      if (gj0) {
        // the last piece's MMAs are done: Q may be replaced and O read, the
        // new Q first, so that its QK runs under the epilogue
        wait_bar(cx, &bars.pv_done[(gj0 - 1) & 1],
                 (uint32_t)((gj0 - 1) >> 1) & 1);
        tc::fence_after();
      }
      if (more) write_q<kFp8>(cx, pc, smem);
      if (gj0) epilogue(cx, prev, tmem, m, l, C::kShiftLog2);
      if (!more) break;
      softmax_tiles<kFp8>(cx, pc, gj0, tmem, m, l);
      prev = pc;
      gj0 += pc.n_tiles;
    }
  } else if constexpr (kFp8) {
    Dequant dq;
    for (int i = first; i < pieces; i += step)
      dequant_piece(cx, decode_piece(p, i, rank), smem, dq);
  }

  // teardown: no copy or MMA may still be in flight in either CTA.  Every
  // load was consumed by an MMA, and every MMA completes before drain.
  if (warp == 1 && rank == 0 && lane == 0) {
    tc::commit_pair(tc::smem_u32(&bars.drain));
    wait_bar(cx, &bars.drain, 0, true);
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

template <bool kFp8>
int pairs_resident() {
  using C = Cfg<kFp8>;
  if (cudaFuncSetAttribute(prefix_attention_kernel<kFp8>,
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
  if (cudaOccupancyMaxActiveClusters(&n, prefix_attention_kernel<kFp8>, &cfg) !=
      cudaSuccess)
    return 0;
  return n;
}

template <bool kFp8>
cudaError_t launch(const SharedParams& p, const CUtensorMap& tm_k,
                   const CUtensorMap& tm_v, cudaStream_t s) {
  using C = Cfg<kFp8>;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(2 * p.pairs), dim3(C::kThreads), C::kSmem, s, attr);
  return cudaLaunchKernelEx(&cfg, prefix_attention_kernel<kFp8>, p, tm_k, tm_v);
}

}  // namespace

cudaError_t launch_prefix_attention(const SharedParams& p,
                                    const CUtensorMap& tm_k,
                                    const CUtensorMap& tm_v, cudaStream_t s) {
  return p.a.k_scales ? launch<true>(p, tm_k, tm_v, s)
                      : launch<false>(p, tm_k, tm_v, s);
}

int prefix_attention_pairs(bool fp8) {
  return fp8 ? pairs_resident<true>() : pairs_resident<false>();
}

}  // namespace specv
