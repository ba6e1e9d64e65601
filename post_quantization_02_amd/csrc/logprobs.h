// Launchers of the tokens' log probabilities (logprobs.hip).
#pragma once

#include "kronq_internal.h"

namespace kronq {

constexpr int kTopMost = 64;              // alternatives of a row

struct LogprobsArgs {
  const void* logits;
  int64_t ld;
  const int32_t* targets;                 // NULL: none
  int64_t rows;
  int vocab, top;
  float *logp, *lse, *entropy;            // NULL: not wanted (logp: no targets)
  float* top_logp;
  int32_t* top_ids;
};

struct LogprobsGradArgs {
  const void* logits;
  int64_t ld;
  const int32_t* targets;
  int64_t rows;
  int vocab, top;
  const float *lse, *entropy;
  const float *d_logp, *d_entropy, *d_top;   // NULL: none
  const int32_t* top_ids;
  void* out;
  int64_t ld_out;
};

size_t logprobs_ws_bytes(int64_t rows, int64_t vocab, int top);
kronq_status logprobs_launch(const LogprobsArgs& a, int32_t dtype, void* ws, hipStream_t s);
// workgroups of a call's launch, for the check of their number
int64_t logprobs_grad_grid(int64_t rows, int64_t vocab);
kronq_status logprobs_grad_launch(const LogprobsGradArgs& a, int32_t dtype, hipStream_t s);

}  // namespace kronq
