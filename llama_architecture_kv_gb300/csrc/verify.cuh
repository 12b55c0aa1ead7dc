// Verification of drafted tokens (declarations).
#pragma once
#include "common.cuh"

namespace llm {

struct VerifyArgs {
  const float* p;         // [B][S + 1][V] target probabilities
  const float* q;         // [B][S][V] draft probabilities, or null
  const int32_t* drafts;  // [B][S]
  const int32_t* count;   // [B] drafts of each row, or null (S)
  const float* u;         // [B][S + 1]
  int32_t B, S, V;
  int32_t* ids;           // [B][S + 1]: the kept drafts, the drawn token, then -1
  int32_t* accepted;      // [B]
};
// rows of V logits to softmax(logits / temp), in place; temp == 0: a 1 at the first largest logit
cudaError_t launch_probs(float* x, int rows, int V, float temp, cudaStream_t s);
cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s);

}  // namespace llm
