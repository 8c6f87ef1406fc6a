// Launch parameters of the block KV append kernels (kv_append.cu,
// rope_append.cu) and the quantise-on-write step they share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace specv {

struct AppendParams {
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  void* k_pages;
  void* v_pages;
  __half* k_scales;
  __half* v_scales;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* q_lens;  // optional [B]: rows of each block (<= q_len)
  int32_t* positions;   // optional
  int64_t* cache_loc;   // optional
  uint32_t* status;     // checked mode only
  int batch, q_len, hkv, page_size, log2_ps, num_pages, max_pages;
  long long max_tokens;
  int fp8;
};

// Rotary positions on a block's queries and keys, and the append of its keys
// and values (rope_append.cu).  Strides are in elements.
struct RopeParams {
  AppendParams a;
  const __nv_bfloat16* q;   // optional, with q_out
  __nv_bfloat16* q_out;     // [B, q_len, Hq, 256]
  const double* freq;       // [rotary / 2] radians per position
  int hq, rotary;
  float factor;             // on the rotated channels
  long long q_req, q_tok, k_req, k_tok, v_req, v_tok;
  // head norms before the rotation (q_weight also NULL without queries)
  const void* q_weight;     // [256], bf16 or fp32; k_weight NULL: no norms
  const void* k_weight;
  int w_bf16;
  float eps, w_offset;
};

// A channel's factor behind its head's norm.
__device__ __forceinline__ float norm_weight(const RopeParams& p, const void* w,
                                             int c) {
  if (!w) return 0.f;  // no queries
  return p.w_offset + (p.w_bf16
                           ? __bfloat162float(
                                 static_cast<const __nv_bfloat16*>(w)[c])
                           : static_cast<const float*>(w)[c]);
}

// A frequency as a 64-bit fraction of a turn (rope_append.cu).
__device__ __forceinline__ uint64_t turn_of(double f) {
  const double turns = f * 0.15915494309189533577;  // 1 / 2 pi
  const double frac = turns - floor(turns);
  // 2^64 frac; a fraction that rounds up to a whole turn is none
  return frac < 1.0 ? __double2ull_rz(frac * 18446744073709551616.0) : 0ull;
}

// Quantise-on-write of one cached row by a whole warp: lane l holds channels
// 8l .. 8l+7 in x and the eight lanes of a 64-channel block share its scale.
// The scale and the codes are computed in fp32 with correctly rounded
// division, so the stored bytes follow the rule stated in spec_verify.h:
//   scale = fp16_rn(amax / 448) (1 if it rounds to zero),
//   byte  = E4M3_rn_satfinite(x / scale)
__device__ __forceinline__ void quantise_row(const float (&x)[8], int lane,
                                             uint8_t* dst, __half* sdst) {
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1)  // the 8 lanes of this 64-channel block
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  __half scale = __float2half_rn(__fdiv_rn(amax, 448.f));
  if (__half2float(scale) == 0.f) scale = __float2half_rn(1.f);
  const float sf = __half2float(scale);
  uint32_t packed[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 qv = make_float2(__fdiv_rn(x[2 * e], sf),
                                  __fdiv_rn(x[2 * e + 1], sf));
    const uint32_t pair =
        __nv_cvt_float2_to_fp8x2(qv, __NV_SATFINITE, __NV_E4M3) & 0xFFFFu;
    packed[e >> 1] |= pair << (16 * (e & 1));
  }
  *reinterpret_cast<uint2*>(dst + lane * 8) = make_uint2(packed[0], packed[1]);
  if ((lane & 7) == 0) sdst[lane >> 3] = scale;
}

cudaError_t launch_rope_append(const RopeParams& p, bool interleaved, int sms,
                               cudaStream_t s);
// Norms as well (norm_rope.cu), for the layouts that fit its lanes.
bool norm_rope_fits(const RopeParams& p, bool interleaved);
cudaError_t launch_norm_rope(const RopeParams& p, bool interleaved, int sms,
                             cudaStream_t s);
cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t s);

}  // namespace specv
