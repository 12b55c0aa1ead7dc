// The tensor-core attention over an 8-bit cache, head size 128 (qattn_tc.cuh).
#include "qattn_tc.cuh"

namespace llm {

cudaError_t launch_qattn_tc128(const CUtensorMap& kmap, const CUtensorMap& vmap, const QAttnArgs& a, int qt, int nc,
                              int grid, cudaStream_t s, bool pdl) {
  return launch_qattn_tc_hd<128>(kmap, vmap, a, qt, nc, grid, s, pdl);
}

}  // namespace llm
