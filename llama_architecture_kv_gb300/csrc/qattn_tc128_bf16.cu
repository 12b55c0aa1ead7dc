// The tensor-core attention over an 8-bit cache: head size 128, bf16 queries, 16 to 64 accumulator
// columns (qattn_tc.cuh).
#include "qattn_tc.cuh"

namespace llm {

LLM_QATTN_TC(qattn_tc128_bf16) {
  if (nc == 1) return launch_qattn_tc<128, 2, 1, 1>(kmap, vmap, a, grid, s, pdl);
  if (nc == 2) return launch_qattn_tc<128, 2, 2, 1>(kmap, vmap, a, grid, s, pdl);
  if (nc == 4) return launch_qattn_tc<128, 2, 4, 1>(kmap, vmap, a, grid, s, pdl);
  return cudaErrorInvalidValue;
}

}  // namespace llm
