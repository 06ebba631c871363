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
size_t logprob_partial_bytes(int top);
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

// Gated block: act = SiLU(x Wg^T) * (x Wu^T), w13 = [Wg; Wu].
struct GatedArgs {
  const uint16_t* x;         // [M, H]
  const uint16_t* w13;       // [2I, H]
  int M, H, I;
  uint16_t* out;             // [M, I]
};
hipError_t launch_gated(const GatedArgs& a, hipStream_t s);

// Its gradient, with gate and up formed again.
struct GatedGradArgs {
  const uint16_t* x;         // [M, H]
  const uint16_t* w13;       // [2I, H]
  const uint16_t* grad_out;  // [M, I]
  int M, H, I;
  uint16_t* grad_x;          // [M, H] or null
  uint16_t* grad_w13;        // [2I, H] or null
  void* workspace;           // gated_backward_bytes
};
size_t gated_backward_bytes(int M, int H, int I);
hipError_t launch_gated_backward(const GatedGradArgs& a, hipStream_t s);

// Low-rank adapters: out = f(addend + scale[s] (x A_s^T) B_s^T), s = slots[m].
struct AdapterArgs {
  const uint16_t* x;         // [M, K]
  const uint16_t* a;         // [S, R, K]
  const uint16_t* b;         // [S, N, R]
  const float* scales;       // [S] or null
  const int32_t* slots;      // [M]
  int M, K, N, R, S, gated;
  const uint16_t* addend;    // [M, N] or null; may be out (not gated)
  uint16_t* out;             // [M, N], gated [M, N / 2]
  void* workspace;           // adapters_bytes
};
size_t adapters_bytes(int M, int R);
hipError_t launch_adapters(const AdapterArgs& a, hipStream_t s);

// bytes (a multiple of 16) of zeros
hipError_t launch_zero(void* p, size_t bytes, hipStream_t s);

}  // namespace moe_host
