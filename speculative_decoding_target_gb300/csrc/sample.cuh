// Launch parameters of sampling with temperature, top-k, top-p and min-p
// (sample.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace specv {

struct SampleParams {
  const void* logits;         // [rows, vocab], fp32 or bf16
  long long row_stride;       // elements
  const float* temperature;   // optional [rows]
  const int32_t* top_k;       // optional [rows]
  const float* top_p;         // optional [rows]
  const float* min_p;         // optional [rows]
  const float* u;             // [rows]
  int32_t* token;             // [rows]
  float* probs;               // optional [rows, vocab]
  float* filtered;            // optional [rows, vocab]
  int rows, vocab;
  int chunk;                  // tokens per CTA of a row's cluster
  int padded;                 // the same, rounded up
};

constexpr int kSampleMaxVocab = 524288;

cudaError_t launch_sample(SampleParams p, bool bf16, int sms, cudaStream_t s);

}  // namespace specv
