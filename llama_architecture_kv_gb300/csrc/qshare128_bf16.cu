// Attention of rows that share positions (qshare.cuh): head size 128, bf16 queries.
#include "qshare.cuh"

namespace llm {

LLM_QSHARE(qshare128_bf16) { return launch_qshare<128, 1>(kmap, vmap, qmap, a, grid, s, pdl); }

}  // namespace llm
