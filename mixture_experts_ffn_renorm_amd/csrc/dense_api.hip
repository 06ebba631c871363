// C ABI of the dense operators around the routed experts: argument checks and
// launches.  Declarations and the contract of every call are in
// include/moe_mi355x.h.
#include <initializer_list>

#include "dense.h"
#include "moe_mi355x.h"

using namespace moe_host;

namespace {

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// An operand's memory (null: the operand is absent).
struct Span {
  const void* p;
  size_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}
// Whether an output shares memory with another output or an input.
bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span* q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) return true;
    for (const Span& i : ins)
      if (overlap(*o, i)) return true;
  }
  return false;
}

#define MOE_TRY_LAUNCH(expr) \
  do {                       \
    if ((expr) != hipSuccess) return MOE_ERR_HIP; \
  } while (0)

constexpr int kMaxVocabulary = 1 << 19;
constexpr int kMaxLogitRows = 1 << 21;
constexpr long long kMaxLogits = 1LL << 35;
constexpr int kMaxAlternatives = 32;
constexpr int kMaxRows = 1 << 21;
constexpr int kMaxRank = 128;
constexpr int kMaxAdapters = 4096;
constexpr int kMaxFeatures = 1 << 17;

int check_logits(int logits_fp32, int M, int V) {
  if (M < 0 || V <= 0 || (logits_fp32 != 0 && logits_fp32 != 1)) return MOE_ERR_INVALID_ARG;
  if (M >= kMaxLogitRows || V > kMaxVocabulary || (long long)M * V > kMaxLogits)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Sizes of the gated block: as for the layer's experts, one expert.
int check_gated(int M, int H, int I) {
  if (M < 0 || H <= 0 || I <= 0) return MOE_ERR_INVALID_ARG;
  if (H % 8 != 0 || I % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if (M >= kMaxRows || H > kMaxFeatures || I > kMaxFeatures) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Sizes of the adapters' products.
int check_adapters(int M, int K, int R) {
  if (M < 0 || K <= 0 || R <= 0) return MOE_ERR_INVALID_ARG;
  if (K % 8 != 0 || R % 8 != 0 || R > kMaxRank || K > kMaxFeatures || M >= kMaxRows)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_linear_adapters_workspace_size(int M, int K, int R) {
  if (check_adapters(M, K, R) != MOE_OK) return 0;
  return adapters_bytes(M > 0 ? M : 1, R);
}

int moe_linear_adapters(const uint16_t* x, const moe_adapters* adapters, const int32_t* slots,
                        int M, int K, int N, int gated, const uint16_t* addend, uint16_t* out,
                        void* workspace, size_t ws_bytes, void* stream) {
  if (adapters == nullptr || N <= 0 || (gated != 0 && gated != 1)) return MOE_ERR_INVALID_ARG;
  const moe_adapters& w = *adapters;
  const int st = check_adapters(M, K, w.rank);
  if (st != MOE_OK) return st;
  if (w.count <= 0) return MOE_ERR_INVALID_ARG;
  if (N % (gated ? 16 : 8) != 0 || N > kMaxFeatures || w.count > kMaxAdapters)
    return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!x || !w.a || !w.b || !slots || !out) return MOE_ERR_INVALID_ARG;
  if (!a16(x) || !a16(w.a) || !a16(w.b) || !a16(out) || !a16(addend) || !a16(workspace))
    return MOE_ERR_INVALID_ARG;
  const size_t need = adapters_bytes(M, w.rank);
  if (workspace == nullptr || ws_bytes < need) return MOE_ERR_WORKSPACE;
  // addend may be out itself: each output is read where it is written
  const bool in_place = addend == out && !gated;
  const size_t S = w.count, R = w.rank;
  if (clash({{out, (size_t)M * (gated ? N / 2 : N) * 2}, {workspace, need}},
            {{x, (size_t)M * K * 2}, {w.a, S * R * K * 2}, {w.b, S * R * N * 2},
             {w.scales, S * 4}, {slots, (size_t)M * 4},
             {in_place ? nullptr : addend, (size_t)M * N * 2}}))
    return MOE_ERR_INVALID_ARG;
  const AdapterArgs a{x, w.a, w.b, w.scales, slots, M, K, N, w.rank, w.count, gated, addend, out,
                      workspace};
  MOE_TRY_LAUNCH(launch_adapters(a, static_cast<hipStream_t>(stream)));
  return MOE_OK;
}

int moe_linear_gated(const uint16_t* x, const uint16_t* w13, int M, int H, int I, uint16_t* out,
                     void* stream) {
  const int st = check_gated(M, H, I);
  if (st != MOE_OK) return st;
  if (M == 0) return MOE_OK;
  if (!x || !w13 || !out || !a16(x) || !a16(w13) || !a16(out)) return MOE_ERR_INVALID_ARG;
  if (clash({{out, (size_t)M * I * 2}}, {{x, (size_t)M * H * 2}, {w13, (size_t)I * H * 4}}))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY_LAUNCH(launch_gated(GatedArgs{x, w13, M, H, I, out}, static_cast<hipStream_t>(stream)));
  return MOE_OK;
}

size_t moe_linear_gated_backward_workspace_size(int M, int H, int I) {
  if (check_gated(M, H, I) != MOE_OK) return 0;
  const size_t n = M == 0 ? 0 : gated_backward_bytes(M, H, I);
  return n > 16 ? n : 16;
}

int moe_linear_gated_backward(const uint16_t* x, const uint16_t* w13, const uint16_t* grad_out,
                              int M, int H, int I, uint16_t* grad_x, uint16_t* grad_w13,
                              void* workspace, size_t ws_bytes, void* stream) {
  const int st = check_gated(M, H, I);
  if (st != MOE_OK) return st;
  if (!grad_x && !grad_w13 && M > 0) return MOE_ERR_INVALID_ARG;
  if (!a16(x) || !a16(w13) || !a16(grad_out) || !a16(grad_x) || !a16(grad_w13) || !a16(workspace))
    return MOE_ERR_INVALID_ARG;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const size_t rows = (size_t)M * H * 2, weights = (size_t)I * H * 4;
  if (M == 0) {   // no rows: the weights' gradient is 0
    if (overlap({grad_w13, weights}, {w13, weights})) return MOE_ERR_INVALID_ARG;
    if (grad_w13) MOE_TRY_LAUNCH(launch_zero(grad_w13, weights, s));
    return MOE_OK;
  }
  if (!x || !w13 || !grad_out) return MOE_ERR_INVALID_ARG;
  const size_t need = gated_backward_bytes(M, H, I);
  if (workspace == nullptr || ws_bytes < need) return MOE_ERR_WORKSPACE;
  if (clash({{grad_x, rows}, {grad_w13, weights}, {workspace, need}},
            {{x, rows}, {w13, weights}, {grad_out, (size_t)M * I * 2}}))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY_LAUNCH(launch_gated_backward(
      GatedGradArgs{x, w13, grad_out, M, H, I, grad_x, grad_w13, workspace}, s));
  return MOE_OK;
}

size_t moe_token_logprobs_workspace_size(int logits_fp32, int M, int V, int top) {
  if (check_logits(logits_fp32, M, V) != MOE_OK || top < 0 || top > kMaxAlternatives || top > V)
    return 0;
  return logprob_partial_bytes(top);
}

int moe_token_logprobs(const void* logits, int logits_fp32, const int32_t* tokens, int M, int V,
                       int top, float* logprobs, float* entropy, float* lse, int32_t* top_ids,
                       float* top_logprobs, void* workspace, size_t ws_bytes, void* stream) {
  const int st = check_logits(logits_fp32, M, V);
  if (st != MOE_OK) return st;
  if (top < 0 || top > V) return MOE_ERR_INVALID_ARG;
  if (top > kMaxAlternatives) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!logits || !tokens || !logprobs || !entropy || !lse || (top > 0 && (!top_ids || !top_logprobs)))
    return MOE_ERR_INVALID_ARG;
  if (!a16(logits) || !a16(workspace)) return MOE_ERR_INVALID_ARG;
  const size_t need = logprob_partial_bytes(top);
  if (workspace == nullptr || ws_bytes < need) return MOE_ERR_WORKSPACE;
  const size_t row = (size_t)M * 4, alt = row * top;
  if (clash({{logprobs, row}, {entropy, row}, {lse, row}, {top > 0 ? top_ids : nullptr, alt},
             {top > 0 ? top_logprobs : nullptr, alt}, {workspace, need}},
            {{logits, (size_t)M * V * (logits_fp32 ? 4 : 2)}, {tokens, row}}))
    return MOE_ERR_INVALID_ARG;
  const LogprobArgs a{logits, !logits_fp32, tokens, M, V, top, logprobs, entropy, lse, top_ids,
                      top_logprobs, workspace};
  MOE_TRY_LAUNCH(launch_token_logprobs(a, static_cast<hipStream_t>(stream)));
  return MOE_OK;
}

int moe_token_logprobs_backward(const void* logits, int logits_fp32, const int32_t* tokens,
                                const float* lse, const float* entropy,
                                const float* grad_logprobs, const float* grad_entropy, int M,
                                int V, void* grad_logits, void* stream) {
  const int st = check_logits(logits_fp32, M, V);
  if (st != MOE_OK) return st;
  if (M == 0) return MOE_OK;
  if (!logits || !tokens || !lse || !grad_logprobs || !grad_logits || (grad_entropy && !entropy))
    return MOE_ERR_INVALID_ARG;
  if (!a16(logits) || !a16(grad_logits)) return MOE_ERR_INVALID_ARG;
  const size_t all = (size_t)M * V * (logits_fp32 ? 4 : 2), row = (size_t)M * 4;
  // grad_logits may be logits itself: each logit is read where its gradient is written
  if (clash({{grad_logits, all}},
            {{grad_logits == logits ? nullptr : logits, all}, {tokens, row}, {lse, row},
             {grad_entropy ? entropy : nullptr, row}, {grad_logprobs, row}, {grad_entropy, row}}))
    return MOE_ERR_INVALID_ARG;
  const LogprobGradArgs a{logits, !logits_fp32, tokens, lse, entropy, grad_logprobs, grad_entropy,
                          M, V, grad_logits};
  MOE_TRY_LAUNCH(launch_token_logprobs_backward(a, static_cast<hipStream_t>(stream)));
  return MOE_OK;
}

}  // extern "C"
