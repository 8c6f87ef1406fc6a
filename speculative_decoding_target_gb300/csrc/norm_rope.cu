// RMS norms of query and key heads, their rotary positions, and the append of
// keys and values to the paged cache, in one pass.
//
//   y_c = x_c w_c / sqrt(mean x^2 + eps),  w_c = offset + weight_c,
// then the rotation of rope_append.cu (whose angles these are: exact fixed-point
// fractions of a turn), with the factor 1 / sqrt taken out of both members of a
// pair and applied last.  Each value is rounded once, where it is stored.
//
// A token's rows are read once and written once, 32 KB at 24 + 4 heads; HBM bounds
// it if the instructions stay few.  So half a warp takes a row, 16 channels a lane
// in two 16-byte pieces, whose pairs lie in the two pieces (or inside them, when
// interleaved): four shuffles for the sum of squares, one set of sines for all
// rows of a token, and packed fp32 arithmetic.  (A warp a row with 8 channels a
// lane took 64.8 us for 8,192 tokens where this takes 51.8, the copy rate 39.7.
// What is left is the chain of a token, at one barrier each: issue 55% busy.  Rows
// copied a token or two ahead through shared memory: 54.6 to 57; two tokens at a
// time with 128 registers: 56; one barrier for the angles of two tokens 52.2, of
// four 53.3.)
//
// Half layouts whose rotary / 2 is no multiple of 8 channels do not split that
// way; they take the kernel in rope_append.cu.
#include "append.cuh"
#include "common.cuh"
#include "packed.cuh"
#include "spec_verify.h"

namespace specv {
namespace {

constexpr int kPairs = 2;       // pairs of rows of a warp whose loads are in flight
// Warps of a CTA and CTAs of an SM.  bf16: three of eight (8,192 tokens 51.8 us;
// four, with 64 registers, 54.2).  FP8: two of ten, four of which have keys or
// values alone, which are quantised (five ragged prompts 52.9 us, a batch of
// blocks 4.4; three of eight 56.6 and 5.0, four of six 67.6 and 5.6).
template <bool kFp8>
struct Shape {
  static constexpr int kWarps = kFp8 ? 10 : 8;
  static constexpr int kCtasPerSm = kFp8 ? 2 : 3;
  static constexpr int kThreads = kWarps * 32;
};

// Eight bf16 channels as four packed pairs of neighbours.
__device__ __forceinline__ void widen(uint4 v, u64 (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    x[k] = pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
}
__device__ __forceinline__ uint32_t narrow(u64 v) {
  const float2 f = unpack2(v);
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 narrow(const u64 (&x)[4]) {
  return make_uint4(narrow(x[0]), narrow(x[1]), narrow(x[2]), narrow(x[3]));
}
// Eight floats (16-byte aligned) as packed neighbours.
__device__ __forceinline__ void load8(const float* p, u64 (&x)[4]) {
  const ulonglong2 lo = *reinterpret_cast<const ulonglong2*>(p);
  const ulonglong2 hi = *reinterpret_cast<const ulonglong2*>(p + 4);
  x[0] = lo.x;
  x[1] = lo.y;
  x[2] = hi.x;
  x[3] = hi.y;
}

// Correctly rounded quotients by a finite scale s, with r the correctly rounded
// reciprocal (Markstein 1990: q within one step of x / s, the remainder x - q s
// exact in one fused step, q + r (x - q s) is the rounded quotient).  Quotients so
// small that the remainder is not exact are zeros in E4M3 whatever their last
// digit; the sign is x's, of zeros too.  (Ragged prompts 54.3 us with divisions,
// 52.9 so.)
__device__ __forceinline__ float2 quotients(u64 x, u64 r, u64 minus_s) {
  const u64 q = mul2(x, r);
  const u64 v = fma2(fma2(q, minus_s, x), r, q);
  return unpack2(v | (x & 0x8000000080000000ull));
}

// Quantise-on-write of a row by half a warp: lane l holds channels 16l .. 16l+15
// and four lanes share a 64-channel block; the rule of quantise_row.
__device__ __forceinline__ void quantise_half(const float (&x)[16], int l,
                                              uint8_t* dst, __half* sdst,
                                              bool store) {
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  __half scale = __float2half_rn(__fdiv_rn(amax, 448.f));
  if (__half2float(scale) == 0.f) scale = __float2half_rn(1.f);
  const float sf = __half2float(scale);
  // by an infinite scale, of values too large for any: zeros, or NaN of infinities
  const bool finite = sf <= 65504.f;
  const float rf = finite ? __frcp_rn(sf) : 0.f, ms = finite ? -sf : 0.f;
  const u64 r = pack2(rf, rf), minus_s = pack2(ms, ms);
  uint32_t packed[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 qv = quotients(pack2(x[2 * e], x[2 * e + 1]), r, minus_s);
    const uint32_t pair =
        __nv_cvt_float2_to_fp8x2(qv, __NV_SATFINITE, __NV_E4M3) & 0xFFFFu;
    packed[e >> 1] |= pair << (16 * (e & 1));
  }
  if (!store) return;
  *reinterpret_cast<uint4*>(dst + l * 16) =
      make_uint4(packed[0], packed[1], packed[2], packed[3]);
  if ((l & 3) == 0) sdst[l >> 2] = scale;
}

template <bool kInterleaved, bool kFp8>
__global__ void __launch_bounds__(Shape<kFp8>::kThreads,
                                  Shape<kFp8>::kCtasPerSm)
    norm_rope_kernel(const RopeParams p) {
  constexpr int kWarps = Shape<kFp8>::kWarps;
  // two buffers: a token's table is written while slow warps still read the
  // one before it
  __shared__ __align__(16) float s_cos[2][kHeadDim / 2], s_sin[2][kHeadDim / 2];
  __shared__ __align__(16) float s_w[2][kHeadDim];
  __shared__ __align__(16) float s_row[kFp8 ? 2 * kWarps : 1][kFp8 ? kHeadDim : 4];
  // the attention call that follows may be scheduled now (it waits for this
  // grid before touching memory)
  tc_grid_launch_dependents();
  const AppendParams& a = p.a;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int sub = lane >> 4, l = lane & 15;  // row of a pair, lane of the row
  const int half = p.rotary >> 1;
  const uint64_t turn = tid < half ? turn_of(p.freq[tid]) : 0ull;
  for (int c = tid; c < kHeadDim; c += kWarps * 32) {
    s_w[0][c] = norm_weight(p, p.q_weight, c);
    s_w[1][c] = norm_weight(p, p.k_weight, c);
  }
  // The lane's two pieces of 8 channels, from ca and from cb on, and the pairs of
  // each (interleaved: pa and pb on; otherwise pa on, in both).  Lanes that do
  // not rotate take the remaining channels.
  int ca = 8 * l, cb = 128 + 8 * l, pa = 4 * l, pb = 64 + 4 * l;
  bool rot_a = ca < p.rotary, rot_b = cb < p.rotary;
  if (!kInterleaved) {
    const int n = p.rotary >> 4;
    rot_a = rot_b = l < n;
    pa = 8 * l;
    if (rot_a) {
      cb = half + 8 * l;
    } else {
      ca = p.rotary + 8 * (l - n);
      cb = ca + ((kHeadDim - p.rotary) >> 1);
    }
  }
  const int q_pairs = (p.hq + 1) >> 1, kv_pairs = (a.hkv + 1) >> 1;
  const int n_kv = 2 * kv_pairs, n_pairs = q_pairs + n_kv;
  // up to 2^31 - 1 tokens: the step past the last one needs the 32nd bit
  const uint32_t q_len = a.q_len, tokens = a.batch * q_len;
  const int step_b = gridDim.x / q_len;
  const uint32_t step_i = gridDim.x - step_b * q_len;
  int buf = 0;
  // With more pairs than the warps hold, the tokens are walked once for each
  // round of them: what a pair is, is worked out once a round.
  for (int round = 0; round < n_pairs; round += kWarps * kPairs) {
    int kind[kPairs], r[kPairs];
    bool there[kPairs];
    uint32_t src_at[kPairs];
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      int pr = round + w + e * kWarps;
      // FP8: keys and values go to the last warps of the first round, which have no
      // second pair when the warps hold all in two
      if (kFp8 && n_kv <= kWarps && n_pairs >= kWarps && pr < n_pairs)
        pr = pr < kWarps - n_kv ? pr
             : pr < kWarps      ? pr - kWarps + n_kv + q_pairs
                                : pr - n_kv;
      // 0 queries, 1 keys, 2 values, 3 none
      kind[e] = pr < q_pairs ? 0 : pr < q_pairs + kv_pairs ? 1 : pr < n_pairs ? 2 : 3;
      r[e] = 2 * (pr - (kind[e] == 0   ? 0
                        : kind[e] == 1 ? q_pairs
                                       : q_pairs + kv_pairs)) + sub;
      there[e] = kind[e] < 3 && r[e] < (kind[e] == 0 ? p.hq : a.hkv);
      src_at[e] = r[e] * kHeadDim + (kind[e] == 2 ? 16 * l : ca);
    }
    int b = blockIdx.x / q_len;
    uint32_t i = blockIdx.x - b * q_len;
    for (uint32_t tok = blockIdx.x; tok < tokens; tok += gridDim.x, buf ^= 1) {
      const int width = a.q_lens ? min(max(a.q_lens[b], 0), a.q_len) : a.q_len;
      const long long t = (long long)a.seq_lens[b] - width + i;
      const bool live = (int)i < width && t >= 0;
      long long slot = -1;  // row of KV head 0 in the pool
      if (live && t < a.max_tokens) {
        const int page =
            a.page_table[(long long)b * a.max_pages + (t >> a.log2_ps)];
        const int at = (int)(t & (a.page_size - 1));
        if (page >= 0 && page < a.num_pages) {
          slot = (long long)page * a.hkv * a.page_size + at;
          if (tid == 0 && round == 0 && a.cache_loc)
            a.cache_loc[tok] = (long long)page * a.page_size + at;
        } else if (a.status && tid == 0) {
          atomicOr(a.status, SPEC_STATUS_BAD_PAGE);
        }
      }
      if (tid == 0 && round == 0) {
        if (a.positions) a.positions[tok] = live ? (int32_t)t : -1;
        if (a.cache_loc && slot < 0) a.cache_loc[tok] = -1;
      }
      const __nv_bfloat16* q_src = p.q + b * p.q_req + i * p.q_tok;
      const __nv_bfloat16* k_src = a.k_new + b * p.k_req + i * p.k_tok;
      const __nv_bfloat16* v_src = a.v_new + b * p.v_req + i * p.v_tok;
      __nv_bfloat16* q_dst = p.q_out + (long long)tok * p.hq * kHeadDim;
      if (live && tid < half) {
        const uint64_t frac = (uint64_t)t * turn;
        float sn, cs;
        sincospif((float)(int32_t)(frac >> 32) * 4.656612873077393e-10f, &sn, &cs);
        s_cos[buf][tid] = cs * p.factor;
        s_sin[buf][tid] = sn * p.factor;
      }
      u64 c_a[4], s_a[4], c_b[4], s_b[4];
      uint4 xa[kPairs], xb[kPairs];
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        xa[e] = xb[e] = make_uint4(0u, 0u, 0u, 0u);
        if (!there[e] || !live) continue;
        const __nv_bfloat16* src =
            (kind[e] == 0 ? q_src : kind[e] == 1 ? k_src : v_src) + src_at[e];
        xa[e] = __ldcs(reinterpret_cast<const uint4*>(src));
        xb[e] = __ldcs(
            reinterpret_cast<const uint4*>(src + (kind[e] == 2 ? 8 : cb - ca)));
      }
      __syncthreads();  // (the loads are on their way)
      load8(&s_cos[buf][kInterleaved ? 0 : (rot_a ? pa : 0)], c_a);
      load8(&s_sin[buf][kInterleaved ? 0 : (rot_a ? pa : 0)], s_a);
      if (kInterleaved) {
        // a pair of channels is one packed pair: cosine twice, sine with signs
        const float4 ka = *reinterpret_cast<const float4*>(&s_cos[buf][pa]);
        const float4 za = *reinterpret_cast<const float4*>(&s_sin[buf][pa]);
        const float4 kb = *reinterpret_cast<const float4*>(&s_cos[buf][pb]);
        const float4 zb = *reinterpret_cast<const float4*>(&s_sin[buf][pb]);
        const float ca4[4] = {ka.x, ka.y, ka.z, ka.w};
        const float sa4[4] = {za.x, za.y, za.z, za.w};
        const float cb4[4] = {kb.x, kb.y, kb.z, kb.w};
        const float sb4[4] = {zb.x, zb.y, zb.z, zb.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          c_a[k] = rot_a ? pack2(ca4[k], ca4[k]) : pack2(1.f, 1.f);
          s_a[k] = rot_a ? pack2(-sa4[k], sa4[k]) : 0ull;
          c_b[k] = rot_b ? pack2(cb4[k], cb4[k]) : pack2(1.f, 1.f);
          s_b[k] = rot_b ? pack2(-sb4[k], sb4[k]) : 0ull;
        }
      } else if (!rot_a) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          c_a[k] = pack2(1.f, 1.f);
          s_a[k] = 0ull;
        }
      }
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        const bool is_q = kind[e] == 0, is_v = kind[e] == 2;
        if (kind[e] == 3 || (!is_q && slot < 0)) continue;
        const long long row = slot + (long long)r[e] * a.page_size;  // in the pool
        if (!is_v && live) {
          u64 ya[4], yb[4];
          widen(xa[e], ya);
          widen(xb[e], yb);
          u64 ss2 = mul2(ya[0], ya[0]);
#pragma unroll
          for (int k = 1; k < 4; ++k) ss2 = fma2(ya[k], ya[k], ss2);
#pragma unroll
          for (int k = 0; k < 4; ++k) ss2 = fma2(yb[k], yb[k], ss2);
          const float2 sf = unpack2(ss2);
          float ss = sf.x + sf.y;
#pragma unroll
          for (int o = 8; o; o >>= 1)
            ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float n = rsqrtf(fmaf(ss, 1.f / kHeadDim, p.eps));
          u64 wa[4], wb[4];
          load8(&s_w[!is_q][ca], wa);
          load8(&s_w[!is_q][cb], wb);
          const u64 n2 = pack2(n, n);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            ya[k] = mul2(ya[k], wa[k]);
            yb[k] = mul2(yb[k], wb[k]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (kInterleaved) {
              const float2 fa = unpack2(ya[k]), fb = unpack2(yb[k]);
              ya[k] = mul2(fma2(ya[k], c_a[k], mul2(pack2(fa.y, fa.x), s_a[k])), n2);
              yb[k] = mul2(fma2(yb[k], c_b[k], mul2(pack2(fb.y, fb.x), s_b[k])), n2);
            } else {
              const u64 minus = s_a[k] ^ 0x8000000080000000ull;
              const u64 u = fma2(ya[k], c_a[k], mul2(yb[k], minus));
              yb[k] = mul2(fma2(yb[k], c_a[k], mul2(ya[k], s_a[k])), n2);
              ya[k] = mul2(u, n2);
            }
          }
          if (kFp8 && !is_q) {
            float* mine = s_row[2 * w + sub];
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              *reinterpret_cast<u64*>(mine + ca + 2 * k) = ya[k];
              *reinterpret_cast<u64*>(mine + cb + 2 * k) = yb[k];
            }
            __syncwarp();
            float x[16];
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              *reinterpret_cast<float4*>(x + k) =
                  *reinterpret_cast<const float4*>(mine + 16 * l + k);
            quantise_half(x, l, static_cast<uint8_t*>(a.k_pages) + row * kHeadDim,
                          a.k_scales + row * (kHeadDim / 64), there[e]);
            continue;
          }
          xa[e] = narrow(ya);
          xb[e] = narrow(yb);
        }
        if (kFp8 && is_v) {
          u64 y[4];
          float x[16];
          widen(xa[e], y);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = unpack2(y[k]);
            x[2 * k] = f.x;
            x[2 * k + 1] = f.y;
          }
          widen(xb[e], y);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = unpack2(y[k]);
            x[8 + 2 * k] = f.x;
            x[9 + 2 * k] = f.y;
          }
          quantise_half(x, l, static_cast<uint8_t*>(a.v_pages) + row * kHeadDim,
                        a.v_scales + row * (kHeadDim / 64), there[e]);
          continue;
        }
        if (!there[e]) continue;
        __nv_bfloat16* dst =
            is_q ? q_dst + r[e] * kHeadDim
                 : static_cast<__nv_bfloat16*>(is_v ? a.v_pages : a.k_pages) +
                       row * kHeadDim;
        *reinterpret_cast<uint4*>(dst + (is_v ? 16 * l : ca)) = xa[e];
        *reinterpret_cast<uint4*>(dst + (is_v ? 16 * l + 8 : cb)) = xb[e];
      }
      b += step_b;
      i += step_i;
      if (i >= q_len) {
        i -= q_len;
        ++b;
      }
    }
  }
}

template <bool kInterleaved, bool kFp8>
cudaError_t launch(const RopeParams& p, int tokens, int sms, cudaStream_t s) {
  using S = Shape<kFp8>;
  norm_rope_kernel<kInterleaved, kFp8>
      <<<min(tokens, sms * S::kCtasPerSm), S::kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

bool norm_rope_fits(const RopeParams& p, bool interleaved) {
  return interleaved || p.rotary % 16 == 0;
}

cudaError_t launch_norm_rope(const RopeParams& p, bool interleaved, int sms,
                             cudaStream_t s) {
  const int tokens = p.a.batch * p.a.q_len;
  if (tokens == 0) return cudaSuccess;
  if (p.a.fp8)
    return interleaved ? launch<true, true>(p, tokens, sms, s)
                       : launch<false, true>(p, tokens, sms, s);
  return interleaved ? launch<true, false>(p, tokens, sms, s)
                     : launch<false, false>(p, tokens, sms, s);
}

}  // namespace specv
