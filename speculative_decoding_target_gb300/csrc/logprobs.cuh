// Launch parameters of log probabilities with entropy and alternatives
// (logprobs.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace specv {

constexpr int kLogprobMaxVocab = 524288;
constexpr int kLogprobMaxTop = 32;

// A CTA's part of a row that others have parts of.
struct LogprobPart {
  int row;           // -1: none
  float m, s, h;     // largest logit, sums against it
  unsigned long long top[kLogprobMaxTop];
};

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
  LogprobPart* parts;         // [2 logprob_runs(sms)]
  int slices;                 // of a row; 0: CTAs take whole rows
};

// CTAs of a call, at most.
int logprob_runs(int sms);
// Whether a call of so many rows cuts them into runs, and needs `parts`.
bool logprob_in_runs(int rows, int sms);
cudaError_t launch_logprobs(LogprobParams p, bool bf16, int sms, cudaStream_t s);

}  // namespace specv
