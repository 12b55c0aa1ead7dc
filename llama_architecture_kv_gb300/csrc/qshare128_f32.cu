// Attention of rows that share positions (qshare.cuh): head size 128, f32 queries.
#include "qshare.cuh"

namespace llm {

LLM_QSHARE(qshare128_f32) { return launch_qshare<128, 0>(kmap, vmap, qmap, a, grid, s, pdl); }

}  // namespace llm
