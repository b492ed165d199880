// Attention over a paged cache on the tensor cores: bf16 and E4M3 rows, scores as they are.
#include "paged_attn_tc.cuh"

namespace dmtp {

int paged_tc_grid(int head_dim, Rows f, int qn) {
  return f == kRaw ? grid_rows<kRaw>(head_dim, qn) : f == kE4M3 ? grid_rows<kE4M3>(head_dim, qn) : grid_rows<kE2M1>(head_dim, qn);
}
cudaError_t paged_attn_tc(const PagedAttn& p, const PagedPlan& pl, Rows f, bool mod, cudaStream_t st) {
  if (mod) return f == kE2M1 ? paged_attn_tc_e2m1_scores(p, pl.grid, st) : paged_attn_tc_scores(p, pl.grid, f, st);
  return f == kE2M1   ? paged_attn_tc_e2m1(p, pl.grid, st)
         : f == kE4M3 ? launch_rows<kE4M3, false>(p, pl.grid, st)
                      : launch_rows<kRaw, false>(p, pl.grid, st);
}

}  // namespace dmtp
