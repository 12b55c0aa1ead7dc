// Attention of rows that share positions, each row by itself (qshare.cu): head size 64, bf16 queries.
#include "qattn_tc.cuh"

namespace llm {

LLM_QATTN_TC(qattn_by64_bf16) {
  if (nc == 1) return launch_qattn_tc<64, 2, 1, 1, 2>(kmap, vmap, a, grid, s, pdl);
  if (nc == 2) return launch_qattn_tc<64, 2, 2, 1, 2>(kmap, vmap, a, grid, s, pdl);
  if (nc == 4) return launch_qattn_tc<64, 2, 4, 1, 2>(kmap, vmap, a, grid, s, pdl);
  return cudaErrorInvalidValue;
}

}  // namespace llm
