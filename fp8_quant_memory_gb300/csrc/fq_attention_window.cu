// fq_attention_window.cu -- paged attention over the last `window` tokens of each sequence and its first `sinks`.
#include "fq_attention.cuh"

namespace fq {

bool launch_attention_window(const PagedArgs& p, int dtype, cudaStream_t s) { return launch_split<true>(p, dtype, s); }

}  // namespace fq
