// Attention over a paged cache on the CUDA cores: scores as they are.
#include "paged_attn_simt.cuh"

namespace dmtp {

int paged_simt_grid(int head_dim) { return 152 * (head_dim <= 128 ? 3 : 2); }

cudaError_t paged_attn_simt(const PagedAttn& p, const PagedPlan& pl, int dtype, Rows f, bool mod, cudaStream_t st) {
  return mod ? paged_attn_simt_scores(p, pl.grid, dtype, f, st) : launch_rows<false>(p, pl.grid, dtype, f, st);
}

}  // namespace dmtp
