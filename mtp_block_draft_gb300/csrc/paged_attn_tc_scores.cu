// Attention over a paged cache on the tensor cores: bf16 and E4M3 rows, capped or biased scores.
#include "paged_attn_tc.cuh"

namespace dmtp {

cudaError_t paged_attn_tc_scores(const PagedAttn& p, int grid, Rows f, cudaStream_t st) {
  return f == kE4M3 ? launch_rows<kE4M3, true>(p, grid, st) : launch_rows<kRaw, true>(p, grid, st);
}

}  // namespace dmtp
