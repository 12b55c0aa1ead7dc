// Attention of rows that share positions (qshare.cuh): head size 64, bf16 queries.
#include "qshare.cuh"

namespace llm {

LLM_QSHARE(qshare64_bf16) { return launch_qshare<64, 1>(kmap, vmap, qmap, a, grid, s, pdl); }

}  // namespace llm
