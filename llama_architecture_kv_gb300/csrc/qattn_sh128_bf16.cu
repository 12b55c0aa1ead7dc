// Attention of rows that share positions, where few columns do (qshare.cuh): head size 128, bf16 queries.
#include "qattn_tc.cuh"

namespace llm {

LLM_QATTN_TC(qattn_sh128_bf16) {
  if (nc == 1) return launch_qattn_tc<128, 2, 1, 1, 1>(kmap, vmap, a, grid, s, pdl);
  if (nc == 2) return launch_qattn_tc<128, 2, 2, 1, 1>(kmap, vmap, a, grid, s, pdl);
  if (nc == 4) return launch_qattn_tc<128, 2, 4, 1, 1>(kmap, vmap, a, grid, s, pdl);
  return cudaErrorInvalidValue;
}

}  // namespace llm
