// fq_attention.cu -- paged attention over whole sequences (fq_attention_window.cu has that over a window of them: the
// instances are many and compile side by side), and its workspace.
#include "fq_attention.cuh"

namespace fq {

size_t attention_workspace_bytes(int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t max_len) {
  const Plan plan = plan_of(B, Hq, Hk, D, max_len, max_len, 0);
  if (!plan.join) return 0;
  return static_cast<size_t>(plan.grid) * (sizeof(Meta) + 2 * kHeads * plan.hg * (4 + padded(D)) * sizeof(float));
}

bool launch_attention_split(const PagedArgs& p, int dtype, cudaStream_t s) {
  return p.window < p.max_len ? launch_attention_window(p, dtype, s) : launch_split<false>(p, dtype, s);
}

}  // namespace fq
