// Log probabilities of given tokens under softmax(logits / T), with the
// distribution's entropy and its likeliest tokens, and their gradient
// (logprobs.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace dflash {

constexpr int kMaxTopK = 32;   // alternatives a row may ask for: one per lane of a warp

// The factor of a logit in the exponent of 2.
inline float logprob_scale2(float temperature) { return 1.4426950408889634f / temperature; }

struct LogprobArgs {
  const void* logits;       // [rows] rows of vocab logits, row_stride elements apart
  int64_t row_stride;
  const int32_t* tokens;    // [rows] or nullptr
  int rows, vocab, top_k;
  float temperature;
  float* logprob;           // [rows] or nullptr
  float* entropy;           // [rows] or nullptr
  float* lse;               // [rows] or nullptr
  int32_t* top_ids;         // [rows][top_k] (top_k > 0)
  float* top_logprobs;
};

struct LogprobGradArgs {
  const void* logits;
  int64_t row_stride;
  const int32_t* tokens;    // [rows]; nullptr without d_logprob
  int rows, vocab;
  float temperature;
  const float* lse;         // [rows]
  const float* entropy;     // [rows]; nullptr without d_entropy
  const float* d_logprob;   // [rows] or nullptr
  const float* d_entropy;   // [rows] or nullptr
  void* d_logits;           // rows d_row_stride elements apart; may be the logits
  int64_t d_row_stride;
};

// One launch each; bf16: the logits (and their gradient) are bf16, else fp32.
cudaError_t token_logprobs_launch(const LogprobArgs& a, bool bf16, int sms, cudaStream_t s);
cudaError_t token_logprobs_backward_launch(const LogprobGradArgs& a, bool bf16, cudaStream_t s);

}  // namespace dflash
