// Attention over a paged cache on the tensor cores: E2M1 rows, capped or biased scores.
#include "paged_attn_tc.cuh"

namespace dmtp {

cudaError_t paged_attn_tc_e2m1_scores(const PagedAttn& p, int grid, cudaStream_t st) {
  return launch_rows<kE2M1, true>(p, grid, st);
}

}  // namespace dmtp
