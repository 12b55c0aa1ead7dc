// Attention of rows that share positions (qshare.cuh): head size 64, f32 queries.
#include "qshare.cuh"

namespace llm {

LLM_QSHARE(qshare64_f32) { return launch_qshare<64, 0>(kmap, vmap, qmap, a, grid, s, pdl); }

}  // namespace llm
