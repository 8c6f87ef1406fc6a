// Launch parameters of log probabilities with entropy and alternatives
// (logprobs.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace specv {

constexpr int kLogprobMaxVocab = 524288;
constexpr int kLogprobMaxTop = 32;

struct LogprobParams {
  const void* logits;         // [rows, vocab], fp32 or bf16
  long long row_stride;       // elements
  const int32_t* token;       // optional [rows]
  const float* temperature;   // optional [rows]
  float* logprob;             // optional [rows], with token
  float* entropy;             // optional [rows]
  int32_t* top_ids;           // [rows, top], with top > 0
  float* top_logprobs;        // [rows, top]
  int rows, vocab, top;
};

cudaError_t launch_logprobs(const LogprobParams& p, bool bf16, int sms,
                            cudaStream_t s);

}  // namespace specv
