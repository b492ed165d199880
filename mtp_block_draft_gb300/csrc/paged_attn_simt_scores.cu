// Attention over a paged cache on the CUDA cores: capped or biased scores.
#include "paged_attn_simt.cuh"

namespace dmtp {

cudaError_t paged_attn_simt_scores(const PagedAttn& p, int grid, int dtype, Rows f, cudaStream_t st) {
  return launch_rows<true>(p, grid, dtype, f, st);
}

}  // namespace dmtp
