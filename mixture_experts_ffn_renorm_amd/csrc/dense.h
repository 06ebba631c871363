// Host-side launchers of the dense operators around the routed experts
// (gated block, adapters, token log probabilities), and what their argument
// checks share.
#pragma once

#include "moe_common.h"

namespace moe_host {

// Log probabilities of given tokens, entropy and alternatives of logit rows.
struct LogprobArgs {
  const void* logits;        // [M, V] bf16 or fp32
  int bf16;
  const int32_t* tokens;     // [M]
  int M, V, top;
  float* logprobs;           // [M]
  float* entropy;            // [M]
  float* lse;                // [M]
  int32_t* top_ids;          // [M, top]
  float* top_logprobs;       // [M, top]
  void* partial;             // logprob_partial_bytes
};
size_t logprob_partial_bytes(int M, int V, int top, int bf16);
hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t s);

struct LogprobGradArgs {
  const void* logits;        // [M, V] bf16 or fp32
  int bf16;
  const int32_t* tokens;     // [M]
  const float* lse;          // [M]
  const float* entropy;      // [M] (grad_entropy not null)
  const float* grad_logprobs;  // [M]
  const float* grad_entropy;   // [M] or null
  int M, V;
  void* grad_logits;         // [M, V], may be logits
};
hipError_t launch_token_logprobs_backward(const LogprobGradArgs& a, hipStream_t s);

}  // namespace moe_host
