// Attention of rows that share positions, where few columns do (qshare.cuh): head size 64, f32 queries.
#include "qattn_tc.cuh"

namespace llm {

LLM_QATTN_TC(qattn_sh64_f32) {
  if (nc == 1) return launch_qattn_tc<64, 4, 1, 0, 1>(kmap, vmap, a, grid, s, pdl);
  if (nc == 2) return launch_qattn_tc<64, 4, 2, 0, 1>(kmap, vmap, a, grid, s, pdl);
  if (nc == 4) return launch_qattn_tc<64, 4, 4, 0, 1>(kmap, vmap, a, grid, s, pdl);
  if (nc == 8) return launch_qattn_tc<64, 4, 8, 0, 1>(kmap, vmap, a, grid, s, pdl);
  return cudaErrorInvalidValue;
}

}  // namespace llm
