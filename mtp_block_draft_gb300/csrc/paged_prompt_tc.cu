// Attention of many rows over a paged cache on the tensor cores: bf16 rows.
#include "paged_prompt_tc.cuh"

namespace dmtp {

cudaError_t paged_prompt_tc(const PagedPrompt& p, const PromptPlan& pl, Rows f, bool mod, cudaStream_t st) {
  return f == kRaw ? launch_rows<kRaw>(p, pl, mod, st) : paged_prompt_tc_scaled(p, pl, f, mod, st);
}

}  // namespace dmtp
