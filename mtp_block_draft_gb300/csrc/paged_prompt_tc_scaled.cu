// Attention of many rows over a paged cache on the tensor cores: E4M3 and E2M1 rows.
#include "paged_prompt_tc.cuh"

namespace dmtp {

cudaError_t paged_prompt_tc_scaled(const PagedPrompt& p, const PromptPlan& pl, Rows f, bool mod, cudaStream_t st) {
  return f == kE4M3 ? launch_rows<kE4M3>(p, pl, mod, st) : launch_rows<kE2M1>(p, pl, mod, st);
}

}  // namespace dmtp
