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
// Warp roles (both CTAs, the issuer in the leader only):
//   warp 0      producer: TMA boxes of the CTA's halves into a ring of 16 KB
//               slots [64 tokens x 128 channels], 128-byte swizzle, in the
//               order in which the issuer consumes them: K0 K1 V0 K2 V1 ...
//   warp 1      issuer: QK_0, then per tile QK_{j+1}, PV_j, so that the
//               softmax of tile j has a QK and a PV's time to run in
//   warps 2..5  softmax: one thread per row; running maximum and sum in base
//               2 and fp32; O is rescaled only when the maximum grows by 2^8;
//               epilogue (normalised fp32 partial, log-sum-exp)
//   warps 6..9  FP8 only: E4M3 bytes times scale to fp16 slots
//
// P is rounded once to the type of V (bf16; fp16 for FP8 KV): the relative
// error of a weight, at most 2^-8, is independent from token to token and no larger
// than that of the bf16 output itself.  (The verify kernel splits P into two
// bf16 terms, free where HBM is the bound; here it would add half again to
// the MMAs.)
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
constexpr int kSlotBytes = 64 * 128 * 2;      // 64 tokens x 128 channels
constexpr int kBlockBytes = 64 * 128;         // its column block of 64
constexpr int kQBytes = 128 * kHeadDim * 2;   // 4 column blocks of 128 rows
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 256;
constexpr float kRescaleLog2 = 8.0f;
constexpr int kMaxSlots = 9;
constexpr int kRaw = 3;                       // FP8 staging buffers
constexpr int kRawBytes = 16384 + 1024;       // bytes and scales

template <bool kFp8>
struct Cfg {
  static constexpr int kSlots = kFp8 ? 6 : kMaxSlots;
  static constexpr int kThreads = kFp8 ? 320 : 192;
  static constexpr int kOffRing = kQBytes;
  static constexpr int kOffRaw = kOffRing + kSlots * kSlotBytes;
  static constexpr int kSmem = kOffRaw + (kFp8 ? kRaw * kRawBytes : 0) + 1024;
  static constexpr uint32_t kAB = kFp8 ? 0u : 1u;  // fp16 or bf16 inputs
  static constexpr uint32_t kIdescQK = (1u << 4) | (kAB << 7) | (kAB << 10) |
                                       ((uint32_t)(kT >> 3) << 17) |
                                       ((uint32_t)(256 >> 4) << 24);
  static constexpr uint32_t kIdescPV = (1u << 4) | (kAB << 7) | (kAB << 10) |
                                       (1u << 16) | ((uint32_t)(256 >> 3) << 17) |
                                       ((uint32_t)(256 >> 4) << 24);
};

struct Bars {
  uint64_t full[kMaxSlots];    // leader: the slot holds both CTAs' halves
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

// A CTA pair's share of one segment.
struct Piece {
  int lead, start, rows_total;  // page-table row, first request, group rows
  int g, row0;                  // KV head, first row of this CTA's 128
  int tok, n_tiles;
  int slot;                     // partial slot
};

__device__ __forceinline__ int checked_page(const AttnParams& p, int lead,
                                            int t) {
  int page = __ldg(p.page_table + (long long)lead * p.max_pages +
                   (t >> p.log2_ps));
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
// Box b of a 64-token half: tokens b * box_rows ..; a lane owns one box of a
// column block in each 64 tokens that its CTA loads per tile.
struct Producer {
  long long seq = 0;     // slots (bf16) or staging buffers (FP8) used so far
  bool live = true;
};

// bf16: one slot, two column blocks of 64 channels x 64 tokens
__device__ __forceinline__ bool load_slot(const Ctx& cx, Producer& pr,
                                          uint8_t* smem, const CUtensorMap* map,
                                          int x0, long long row, int lane,
                                          int nb, int box_rows) {
  using C = Cfg<false>;
  const int s = (int)(pr.seq % C::kSlots);
  const long long use = pr.seq / C::kSlots;
  const bool ok = use == 0 ||
                  wait_bar(cx, &cx.bars->empty[s], (uint32_t)(use - 1) & 1);
  if (!__all_sync(0xffffffffu, ok && !*cx.abort)) return false;
  const uint32_t full = tc::smem_u32(&cx.bars->full[s]);
  if (cx.rank == 0 && lane == 0)
    tc::bar_arrive_expect_tx(full, 2 * kSlotBytes);
  __syncwarp();
  if (lane < 2 * nb) {
    const int blk = lane / nb, bi = lane - blk * nb;
    tc::tma_load_2d_pair(
        tc::smem_u32(smem + C::kOffRing + s * kSlotBytes + blk * kBlockBytes +
                     bi * box_rows * 128),
        map, tc::map_to(full, 0), x0 + blk * 64, (int)row);
  }
  ++pr.seq;
  return true;
}

// FP8: one staging buffer of 16 KB and its scales
__device__ __forceinline__ bool load_raw(const Ctx& cx, Producer& pr,
                                         uint8_t* smem, const CUtensorMap* map,
                                         const __half* scales, bool is_v,
                                         long long row, int lane, int nb,
                                         int box_rows) {
  using C = Cfg<true>;
  const int s = (int)(pr.seq % kRaw);
  const long long use = pr.seq / kRaw;
  const bool ok = use == 0 ||
                  wait_bar(cx, &cx.bars->raw_empty[s], (uint32_t)(use - 1) & 1);
  if (!__all_sync(0xffffffffu, ok && !*cx.abort)) return false;
  const uint32_t full = tc::smem_u32(&cx.bars->raw_full[s]);
  if (lane == 0)
    tc::bar_arrive_expect_tx(full, 16384 + (is_v ? 1024 : 512));
  __syncwarp();
  const uint32_t base = tc::smem_u32(smem + C::kOffRaw + s * kRawBytes);
  if (lane < 2 * nb) {
    // K: two blocks of 128 bytes x 64 tokens; V: the CTA's 128 bytes of 128
    // tokens, the second 64 in the second block
    const int blk = lane / nb, bi = lane - blk * nb;
    tc::tma_load_2d(base + blk * kBlockBytes + bi * box_rows * 128, map, full,
                    is_v ? (int)cx.rank * 128 : blk * 128, (int)row);
    if (is_v || blk == 0) {
      const uint32_t dst = base + 16384 + (blk * 64 + bi * box_rows) * 8;
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
          "[%0], [%1], %2, [%3];" ::"r"(dst),
          "l"(reinterpret_cast<const uint8_t*>(scales) + row * 8),
          "r"(box_rows * 8), "r"(full)
          : "memory");
    }
  }
  ++pr.seq;
  return true;
}

template <bool kFp8>
__device__ void produce(const Ctx& cx, const Piece& pc, Producer& pr,
                        uint8_t* smem, const CUtensorMap* tm_k,
                        const CUtensorMap* tm_v) {
  const AttnParams& p = cx.p->a;
  const int lane = threadIdx.x & 31;
  const int rpb = p.box_rows, nb = 64 / rpb;
  const int bi = lane % nb, blk = (lane / nb) & 1;
  // K: this CTA's 64 tokens; V: all 128, as two halves (bf16: both by every
  // lane, one after the other; FP8: half blk by this lane)
  const int tk = pc.tok + (int)cx.rank * 64 + bi * rpb;
  const int tv = pc.tok + bi * rpb;
  int pk = 0, pv0 = 0, pv1 = 0;
  if (lane < 2 * nb) {
    pk = checked_page(p, pc.lead, tk);
    pv0 = checked_page(p, pc.lead, tv);
    pv1 = checked_page(p, pc.lead, tv + 64);
  }
  for (int j = -1; j < pc.n_tiles; ++j) {
    // step j loads K of tile j + 1, then V of tile j
    if (j + 1 < pc.n_tiles) {
      const int t = tk + (j + 1) * kT;
      const long long row = pool_row(p, pk, pc.g, t);
      if (lane < 2 * nb && j + 2 < pc.n_tiles)
        pk = checked_page(p, pc.lead, t + kT);
      if (kFp8) {
        if (!load_raw(cx, pr, smem, tm_k, p.k_scales, false, row, lane, nb, rpb))
          pr.live = false;
      } else {
        for (int h = 0; h < 2 && pr.live; ++h)
          pr.live = load_slot(cx, pr, smem, tm_k, h * 128, row, lane, nb, rpb);
      }
      if (!pr.live) return;
    }
    if (j >= 0) {
      const int t = tv + j * kT;
      const long long r0 = pool_row(p, pv0, pc.g, t);
      const long long r1 = pool_row(p, pv1, pc.g, t + 64);
      if (lane < 2 * nb && j + 1 < pc.n_tiles) {
        pv0 = checked_page(p, pc.lead, t + kT);
        pv1 = checked_page(p, pc.lead, t + kT + 64);
      }
      if (kFp8) {
        if (!load_raw(cx, pr, smem, tm_v, p.v_scales, true, blk ? r1 : r0, lane,
                      nb, rpb))
          pr.live = false;
      } else {
        for (int h = 0; h < 2 && pr.live; ++h)
          pr.live = load_slot(cx, pr, smem, tm_v, (int)cx.rank * 128,
                              h ? r1 : r0, lane, nb, rpb);
      }
      if (!pr.live) return;
    }
  }
}

// ---- warps 6..9 (FP8): staged bytes to fp16 slots ---------------------------
// A staging buffer makes two slots of 64 tokens x 128 channels.  Thread t
// converts 16-byte chunk c = t & 7 (16 channels) of tokens (t >> 3) + 16 e;
// the two 16-byte stores of lanes c and c + 4 fall into the same banks of two
// column blocks, so the upper half stores its pair in the other order.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t pair16, __half2 sc) {
  const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
      static_cast<__nv_fp8x2_storage_t>(pair16), __NV_E4M3);
  const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&hr), sc);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void dequant_unit(const Ctx& cx, uint8_t* smem,
                                             long long& rseq, long long& sseq,
                                             bool is_v) {
  using C = Cfg<true>;
  const int tid = threadIdx.x - 192, lane = threadIdx.x & 31;
  const int c = tid & 7, tok0 = tid >> 3;
  const int r = (int)(rseq % kRaw);
  wait_bar(cx, &cx.bars->raw_full[r], (uint32_t)(rseq / kRaw) & 1);
  const uint8_t* raw = smem + C::kOffRaw + r * kRawBytes;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int s = (int)(sseq % C::kSlots);
    const long long use = sseq / C::kSlots;
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
    if (use > 0) wait_bar(cx, &cx.bars->empty[s], (uint32_t)(use - 1) & 1);
    uint8_t* out = smem + C::kOffRing + s * kSlotBytes + (c >> 2) * kBlockBytes;
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
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0)
      tc::arrive_cluster(tc::map_to(tc::smem_u32(&cx.bars->full[s]), 0));
    ++sseq;
  }
  __syncwarp();
  if (lane == 0) tc::bar_arrive(tc::smem_u32(&cx.bars->raw_empty[r]));
  ++rseq;
}

__device__ void dequant_piece(const Ctx& cx, const Piece& pc, uint8_t* smem,
                              long long& rseq, long long& sseq) {
  for (int j = -1; j < pc.n_tiles; ++j) {
    if (j + 1 < pc.n_tiles) dequant_unit(cx, smem, rseq, sseq, false);
    if (j >= 0) dequant_unit(cx, smem, rseq, sseq, true);
  }
}

// ---- warp 1 of the leader, one thread: MMA issue ----------------------------
template <bool kFp8>
__device__ __forceinline__ bool issue_qk(const Ctx& cx, long long& seq, int gj,
                                         uint32_t tmem, uint8_t* smem) {
  using C = Cfg<kFp8>;
  const uint32_t d = tmem + kColS + (gj & 1) * kT;
  const uint32_t q = tc::smem_u32(smem);
#pragma unroll
  for (int h = 0; h < 2; ++h, ++seq) {
    const int s = (int)(seq % C::kSlots);
    if (!wait_bar<kFp8>(cx, &cx.bars->full[s],
                        (uint32_t)(seq / C::kSlots) & 1))
      return false;
    tc::fence_after();
    const uint32_t kb = tc::smem_u32(smem + C::kOffRing + s * kSlotBytes);
#pragma unroll
    for (int k = 0; k < 8; ++k) {  // 16 channels each
      const uint64_t a = tc::desc_sw128(
          q + (2 * h + (k >> 2)) * (128 * 128) + (k & 3) * 32, 16, 1024);
      const uint64_t b =
          tc::desc_sw128(kb + (k >> 2) * kBlockBytes + (k & 3) * 32, 16, 1024);
      tc::mma_pair(d, a, b, C::kIdescQK, (h | k) ? 1u : 0u);
    }
    tc::commit_pair(tc::smem_u32(&cx.bars->empty[s]));
  }
  tc::commit_pair(tc::smem_u32(&cx.bars->s_full[gj & 1]));
  return true;
}

template <bool kFp8>
__device__ __forceinline__ bool issue_pv(const Ctx& cx, long long& seq, int gj,
                                         bool first, uint32_t tmem,
                                         uint8_t* smem) {
  using C = Cfg<kFp8>;
  if (!wait_bar(cx, &cx.bars->p_full[gj & 1], (uint32_t)(gj >> 1) & 1))
    return false;
  const uint32_t pt = tmem + kColS + (gj & 1) * kT;
#pragma unroll
  for (int h = 0; h < 2; ++h, ++seq) {
    const int s = (int)(seq % C::kSlots);
    if (!wait_bar<kFp8>(cx, &cx.bars->full[s],
                        (uint32_t)(seq / C::kSlots) & 1))
      return false;
    tc::fence_after();
    const uint32_t vb = tc::smem_u32(smem + C::kOffRing + s * kSlotBytes);
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // 16 tokens each
      const uint64_t b = tc::desc_sw128(vb + k * 2048, kBlockBytes, 1024);
      tc::mma_pair_ta(tmem, pt + (h * 4 + k) * 8, b, C::kIdescPV,
                      (first && (h | k) == 0) ? 0u : 1u);
    }
    tc::commit_pair(tc::smem_u32(&cx.bars->empty[s]));
  }
  tc::commit_pair(tc::smem_u32(&cx.bars->pv_done[gj & 1]));
  return true;
}

template <bool kFp8>
__device__ void mma_piece(const Ctx& cx, const Piece& pc, int gj0, int n_piece,
                          long long& seq, uint32_t tmem, uint8_t* smem) {
  if (!wait_bar<true>(cx, &cx.bars->q_full, (uint32_t)n_piece & 1)) return;
  tc::fence_after();
  if (!issue_qk<kFp8>(cx, seq, gj0, tmem, smem)) return;
  for (int j = 0; j < pc.n_tiles; ++j) {
    if (j + 1 < pc.n_tiles &&
        !issue_qk<kFp8>(cx, seq, gj0 + j + 1, tmem, smem))
      return;
    if (!issue_pv<kFp8>(cx, seq, gj0 + j, j == 0, tmem, smem)) return;
  }
}

// ---- warps 2..5: Q, softmax, epilogue ---------------------------------------
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
    uint32_t raw[kT];
    tc::tmem_ld_cols<kT>(sbuf, raw);
    const float* s = reinterpret_cast<const float*>(raw);
    float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int k = 4; k < kT; ++k) mx4[k & 3] = fmaxf(mx4[k & 3], s[k]);
    const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
    bool need = false;
    float alpha = 1.f;
    if (jt == 0) {
      m = mx;
    } else if (mx > m + kRescaleLog2) {
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
    const float mu = m == -INFINITY ? 0.f : m;
    float sum4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kT; k += 2) {
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
    l += (sum4[0] + sum4[1]) + (sum4[2] + sum4[3]);
    tc::tmem_st_cols<kT / 2>(sbuf, raw);
    tc::tmem_wait_st();
    tc::fence_before();
    __syncwarp();
    if (lane == 0)
      tc::arrive_cluster_relaxed(
          tc::map_to(tc::smem_u32(&cx.bars->p_full[gj & 1]), 0));
  }
}

__device__ void epilogue(const Ctx& cx, const Piece& pc, int gl, uint32_t tmem,
                         float m, float l) {
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
        l > 0.f ? (m == -INFINITY ? 0.f : m) + log2f(l) : -INFINITY;
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
  // the tails' kernel may be scheduled now; it waits for this grid
  tc_grid_launch_dependents();
  tc_grid_dependency_wait();  // the plan is written by the kernel before
  const int pieces = p.plan[p.groups].piece0;
  if ((int)(blockIdx.x >> 1) >= pieces) return;  // both CTAs of the pair
  const uint32_t rank = tc::cluster_rank();

  if (tid == 0) {
    for (int s = 0; s < C::kSlots; ++s) {
      // bf16: the leader's expect_tx plus both CTAs' bytes; FP8: the four
      // dequant warps of both CTAs
      tc::bar_init(tc::smem_u32(&bars.full[s]), kFp8 ? 8 : 1);
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
      tc::bar_init(tc::smem_u32(&bars.raw_empty[s]), 4);
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
  const Ctx cx{&bars, &s_abort,
               tc::map_to(tc::smem_u32(&s_abort), rank ^ 1u), rank, &p};

  int gj0 = 0, n_piece = 0;
  Producer pr;
  long long mseq = 0, rseq = 0, sseq = 0;
  float m = 0.f, l = 0.f;
  Piece prev{};
  for (int i = blockIdx.x >> 1; i < pieces; i += gridDim.x >> 1) {
    const Piece pc = decode_piece(p, i, rank);
    if (warp == 0) {
      if (pr.live) produce<kFp8>(cx, pc, pr, smem, &tm_k, &tm_v);
      __syncwarp();
    } else if (warp == 1) {
      if (rank == 0 && lane == 0)
        mma_piece<kFp8>(cx, pc, gj0, n_piece, mseq, tmem, smem);
      __syncwarp();
    } else if (warp < 6) {
      if (n_piece) {
        // the last piece's MMAs are done: Q may be replaced and O read, the
        // new Q first, so that its QK runs under the epilogue
        wait_bar(cx, &bars.pv_done[(gj0 - 1) & 1],
                 (uint32_t)((gj0 - 1) >> 1) & 1);
        tc::fence_after();
      }
      write_q<kFp8>(cx, pc, smem);
      if (n_piece) epilogue(cx, prev, gj0 - 1, tmem, m, l);
      softmax_tiles<kFp8>(cx, pc, gj0, tmem, m, l);
    } else if (kFp8) {
      dequant_piece(cx, pc, smem, rseq, sseq);
    }
    prev = pc;
    gj0 += pc.n_tiles;
    ++n_piece;
  }
  if (warp >= 2 && warp < 6 && n_piece) {
    wait_bar(cx, &bars.pv_done[(gj0 - 1) & 1],
             (uint32_t)((gj0 - 1) >> 1) & 1);
    tc::fence_after();
    epilogue(cx, prev, gj0 - 1, tmem, m, l);
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
