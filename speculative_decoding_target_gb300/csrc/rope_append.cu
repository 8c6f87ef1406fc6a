// Rotary positions on a block's queries and keys, with the append of the
// rotated keys and the values to the paged cache in the same pass.
//
// A pair of channels (x, y) of a token at position t becomes
//   (m (x cos a - y sin a), m (y cos a + x sin a)),   a = t f_j,
// for the rotary / 2 frequencies f_j; pair j is channels (j, j + rotary/2) or,
// interleaved, (2j, 2j+1), and the channels from rotary on are copied.  Each
// value is rounded once, where it is stored.
//
// The angle.  t f_j reaches 10^5 and more turns, where an fp32 product has no
// digits left below a turn.  The frequency is turned once per CTA into a
// 64-bit fixed-point fraction of a turn, F = 2^64 frac(f / 2 pi); t F modulo
// 2^64 is then the exact fraction of a turn that t steps of F make, its top 32
// bits go to sincospi, and the only error is F's rounding (t 2^-64 turns) and
// that of f / 2 pi in 64 bits.
//
// A token's rows are read once and written once: 32 KB a token at 24 + 4 heads.
// One CTA of eight warps takes a token at a time; thread j makes the sine and
// cosine of pair j, and every warp takes every eighth row (query heads, then
// keys, then values), four rows in flight.  A lane's four pairs are the same
// for every row, so their sines stay in registers.
//
// Measured: 8,192 tokens (268 MB) 48 us in a graph, 0.83 of the copy rate, 49.5
// a call; what is left is instructions (issue 66% busy, the ALU 56%), not
// trigonometry (without it: the same time).  On an earlier form of the loop, a
// call took 51.6 us with four CTAs an SM, 56.0 with three and 57.9 with five
// (spills), and 58.8 where lengths and page ids were read ahead, which cost more
// instructions than it hid.
#include "append.cuh"
#include "common.cuh"
#include "spec_verify.h"

namespace specv {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 4;        // rows of a warp whose loads are in flight
constexpr int kCtasPerSm = 4;

__device__ __forceinline__ void unpack4(uint2 r, float* x) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
  x[0] = __low2float(h[0]);
  x[1] = __high2float(h[0]);
  x[2] = __low2float(h[1]);
  x[3] = __high2float(h[1]);
}

__device__ __forceinline__ uint2 pack4(const float* x) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(x[2], x[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                    *reinterpret_cast<const uint32_t*>(&hi));
}

template <bool kInterleaved, bool kNorm>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm)
    rope_append_kernel(const RopeParams p) {
  // two buffers: a token's table is written while slow warps still read the
  // one before it
  __shared__ __align__(16) float2 s_cs[2][kHeadDim / 2];
  __shared__ __align__(16) float s_row[kWarps][kHeadDim];
  __shared__ __align__(16) float s_w[kNorm ? 2 : 1][kNorm ? kHeadDim : 1];
  // the attention call that follows may be scheduled now (it waits for this
  // grid before touching memory)
  tc_grid_launch_dependents();
  const AppendParams& a = p.a;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int half = p.rotary >> 1;
  const uint64_t turn = tid < half ? turn_of(p.freq[tid]) : 0ull;
  // The lane's two quads of channels.  Its pairs are 4 lane .. 4 lane + 3:
  // both members inside the quads, whatever the layout; lanes past the
  // rotated part take the remaining channels in order.
  const bool rot = lane < (p.rotary >> 3);
  int qa = 2 * lane, qb = 2 * lane + 1;
  if (!kInterleaved) {
    const int n8 = p.rotary >> 3;
    qa = rot ? lane : 2 * lane;
    qb = rot ? lane + n8 : qa + 1;
  }
  if constexpr (kNorm) {
    s_w[0][tid] = norm_weight(p, p.q_weight, tid);
    s_w[1][tid] = norm_weight(p, p.k_weight, tid);
    __syncthreads();
  }
  const int n_rows = p.hq + 2 * a.hkv;
  // up to 2^31 - 1 tokens: the step past the last one needs the 32nd bit
  const uint32_t q_len = a.q_len, tokens = a.batch * q_len;
  int buf = 0;
  int b = blockIdx.x / q_len;
  uint32_t i = blockIdx.x - b * q_len;
  const int step_b = gridDim.x / q_len;
  const uint32_t step_i = gridDim.x - step_b * q_len;
  for (uint32_t tok = blockIdx.x; tok < tokens; tok += gridDim.x, buf ^= 1) {
    // the token's rows, at this lane's channels (8 lane on for values)
    const __nv_bfloat16* q_src = p.q + b * p.q_req + i * p.q_tok;
    const __nv_bfloat16* k_src = a.k_new + b * p.k_req + i * p.k_tok;
    const __nv_bfloat16* v_src = a.v_new + b * p.v_req + i * p.v_tok + 8 * lane;
    __nv_bfloat16* q_dst = p.q_out + (long long)tok * p.hq * kHeadDim;
    const int width =
        a.q_lens ? min(max(a.q_lens[b], 0), a.q_len) : a.q_len;
    const long long t = (long long)a.seq_lens[b] - width + i;
    const bool live = (int)i < width && t >= 0;
    long long slot = -1;  // row of KV head 0 in the pool
    if (live && t < a.max_tokens) {
      const int page =
          a.page_table[(long long)b * a.max_pages + (t >> a.log2_ps)];
      const int at = (int)(t & (a.page_size - 1));
      if (page >= 0 && page < a.num_pages) {
        slot = (long long)page * a.hkv * a.page_size + at;
        if (tid == 0 && a.cache_loc)
          a.cache_loc[tok] = (long long)page * a.page_size + at;
      } else if (a.status && tid == 0) {
        atomicOr(a.status, SPEC_STATUS_BAD_PAGE);
      }
    }
    if (tid == 0) {
      if (a.positions) a.positions[tok] = live ? (int32_t)t : -1;
      if (a.cache_loc && slot < 0) a.cache_loc[tok] = -1;
    }
    if (live && tid < half) {
      const uint64_t frac = (uint64_t)t * turn;
      float sn, cs;
      sincospif((float)(int32_t)(frac >> 32) * 4.656612873077393e-10f, &sn,
                &cs);
      s_cs[buf][tid] = make_float2(cs * p.factor, sn * p.factor);
    }
    bool ready = false;
    float cs[4], sn[4];
    for (int base = w; base < n_rows; base += kWarps * kRows) {
      uint2 xa[kRows], xb[kRows];
#pragma unroll
      for (int e = 0; e < kRows; ++e) {
        const int r = base + e * kWarps;
        xa[e] = xb[e] = make_uint2(0u, 0u);
        if (r >= n_rows || !live) continue;
        if (r < p.hq + a.hkv) {
          const __nv_bfloat16* src = r < p.hq
                                         ? q_src + r * kHeadDim
                                         : k_src + (r - p.hq) * kHeadDim;
          if (kInterleaved) {
            const uint4 v =
                __ldcs(reinterpret_cast<const uint4*>(src + 8 * lane));
            xa[e] = make_uint2(v.x, v.y);
            xb[e] = make_uint2(v.z, v.w);
          } else {
            xa[e] = __ldcs(reinterpret_cast<const uint2*>(src + 4 * qa));
            xb[e] = __ldcs(reinterpret_cast<const uint2*>(src + 4 * qb));
          }
        } else {
          const uint4 v = __ldcs(reinterpret_cast<const uint4*>(
              v_src + (r - p.hq - a.hkv) * kHeadDim));
          xa[e] = make_uint2(v.x, v.y);
          xb[e] = make_uint2(v.z, v.w);
        }
      }
      if (!ready) {  // once per token, after the first loads are on their way
        __syncthreads();
        ready = true;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 c =
              rot ? s_cs[buf][4 * lane + e] : make_float2(1.f, 0.f);
          cs[e] = c.x;
          sn[e] = c.y;
        }
      }
#pragma unroll
      for (int e = 0; e < kRows; ++e) {
        const int r = base + e * kWarps;
        if (r >= n_rows) continue;
        if (r < p.hq + a.hkv) {
          const bool key = r >= p.hq;
          if (key && slot < 0) continue;
          if (live && (kNorm || rot)) {
            float x[8];
            unpack4(xa[e], x);
            unpack4(xb[e], x + 4);
            if constexpr (kNorm) {
              float ss = 0.f;
#pragma unroll
              for (int k = 0; k < 8; ++k) ss = fmaf(x[k], x[k], ss);
#pragma unroll
              for (int o = 16; o; o >>= 1)
                ss += __shfl_xor_sync(0xffffffffu, ss, o);
              const float n = rsqrtf(fmaf(ss, 1.f / kHeadDim, p.eps));
              const float4 wa =
                  *reinterpret_cast<const float4*>(&s_w[key][4 * qa]);
              const float4 wb =
                  *reinterpret_cast<const float4*>(&s_w[key][4 * qb]);
              x[0] *= n * wa.x; x[1] *= n * wa.y;
              x[2] *= n * wa.z; x[3] *= n * wa.w;
              x[4] *= n * wb.x; x[5] *= n * wb.y;
              x[6] *= n * wb.z; x[7] *= n * wb.w;
            }
            float y[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int i0 = kInterleaved ? 2 * k : k;
              const int i1 = kInterleaved ? 2 * k + 1 : k + 4;
              y[i0] = x[i0] * cs[k] - x[i1] * sn[k];
              y[i1] = x[i1] * cs[k] + x[i0] * sn[k];
            }
            if (key && a.fp8) {
              *reinterpret_cast<float4*>(&s_row[w][4 * qa]) =
                  make_float4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<float4*>(&s_row[w][4 * qb]) =
                  make_float4(y[4], y[5], y[6], y[7]);
            } else {
              xa[e] = pack4(y);
              xb[e] = pack4(y + 4);
            }
          } else if (key && a.fp8) {
            unpack4(xa[e], &s_row[w][4 * qa]);
            unpack4(xb[e], &s_row[w][4 * qb]);
          }
          if (key && a.fp8) {
            const long long row = slot + (long long)(r - p.hq) * a.page_size;
            __syncwarp();
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = s_row[w][8 * lane + k];
            quantise_row(x, lane,
                         static_cast<uint8_t*>(a.k_pages) + row * kHeadDim,
                         a.k_scales + row * (kHeadDim / 64));
            __syncwarp();
          } else {
            __nv_bfloat16* dst =
                key ? static_cast<__nv_bfloat16*>(a.k_pages) +
                          (slot + (long long)(r - p.hq) * a.page_size) *
                              kHeadDim
                    : q_dst + r * kHeadDim;
            if (kInterleaved) {
              *reinterpret_cast<uint4*>(dst + 8 * lane) =
                  make_uint4(xa[e].x, xa[e].y, xb[e].x, xb[e].y);
            } else {
              *reinterpret_cast<uint2*>(dst + 4 * qa) = xa[e];
              *reinterpret_cast<uint2*>(dst + 4 * qb) = xb[e];
            }
          }
        } else if (slot >= 0) {
          const long long row =
              slot + (long long)(r - p.hq - a.hkv) * a.page_size;
          if (a.fp8) {
            float x[8];
            unpack4(xa[e], x);
            unpack4(xb[e], x + 4);
            quantise_row(x, lane,
                         static_cast<uint8_t*>(a.v_pages) + row * kHeadDim,
                         a.v_scales + row * (kHeadDim / 64));
          } else {
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.v_pages) +
                                      row * kHeadDim + 8 * lane) =
                make_uint4(xa[e].x, xa[e].y, xb[e].x, xb[e].y);
          }
        }
      }
    }
    if (!ready) __syncthreads();  // a warp without rows
    b += step_b;
    i += step_i;
    if (i >= q_len) {
      i -= q_len;
      ++b;
    }
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, bool interleaved, int sms,
                               cudaStream_t s) {
  if (p.k_weight && norm_rope_fits(p, interleaved))
    return launch_norm_rope(p, interleaved, sms, s);
  const int tokens = p.a.batch * p.a.q_len;
  if (tokens == 0) return cudaSuccess;
  const int grid = min(tokens, sms * kCtasPerSm);
  if (p.k_weight)
    rope_append_kernel<false, true><<<grid, kWarps * 32, 0, s>>>(p);
  else if (interleaved)
    rope_append_kernel<true, false><<<grid, kWarps * 32, 0, s>>>(p);
  else
    rope_append_kernel<false, false><<<grid, kWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace specv
