// The tensor-core attention over an 8-bit cache: head size 64, f32 queries, 96 and 128 accumulator
// columns (qattn_tc.cuh).
#include "qattn_tc.cuh"

namespace llm {

LLM_QATTN_TC(qattn_tc64_f32_wide) {
  if (nc == 6) return launch_qattn_tc<64, 4, 6, 0>(kmap, vmap, a, grid, s, pdl);
  if (nc == 8) return launch_qattn_tc<64, 4, 8, 0>(kmap, vmap, a, grid, s, pdl);
  return cudaErrorInvalidValue;
}

}  // namespace llm
