// Attention over a paged cache on the tensor cores: E2M1 rows.
#include "paged_attn_tc.cuh"

namespace dmtp {

cudaError_t paged_attn_tc_e2m1(const PagedAttn& p, int grid, cudaStream_t st) {
  return launch_rows<kE2M1, false>(p, grid, st);
}

}  // namespace dmtp
