// The tensor-core attention over an 8-bit cache: head size 64, f32 queries, 16 to 64 accumulator
// columns (qattn_tc.cuh).
#include "qattn_tc.cuh"

namespace llm {

LLM_QATTN_TC(qattn_tc64_f32) {
  if (nc == 1) return launch_qattn_tc<64, 4, 1, 0>(kmap, vmap, a, grid, s, pdl);
  if (nc == 2) return launch_qattn_tc<64, 4, 2, 0>(kmap, vmap, a, grid, s, pdl);
  if (nc == 4) return launch_qattn_tc<64, 4, 4, 0>(kmap, vmap, a, grid, s, pdl);
  return cudaErrorInvalidValue;
}

}  // namespace llm
