// fq_matmul_fused.cu -- the matrix product's kernels with bias, activation and residual in their epilogue.
#include "fq_matmul.cuh"

namespace fq {
namespace {

// The wide kernel is compiled for each activation and type: its epilogue works on registers, and a choice among the
// activations at each of them took 5 us a tile (4096 x 8192 x 4096, seven rounds of tiles: 202 us with bias, gelu_tanh and
// residual, against 115 without an epilogue).
template <int kAct>
bool launch_wide_act(const MatmulArgs& a, const MmArgs& p, const MatmulPlan& plan, cudaStream_t s) {
  return p.dtype == DT_BF16 ? launch_wide<kAct, __nv_bfloat16>(a, p, plan, s) : launch_wide<kAct, __half>(a, p, plan, s);
}

bool launch_wide_any(const MatmulArgs& a, const MmArgs& p, const MatmulPlan& plan, cudaStream_t s) {
  switch (p.activation) {
    case FQ_ACT_RELU: return launch_wide_act<FQ_ACT_RELU>(a, p, plan, s);
    case FQ_ACT_GELU: return launch_wide_act<FQ_ACT_GELU>(a, p, plan, s);
    case FQ_ACT_GELU_TANH: return launch_wide_act<FQ_ACT_GELU_TANH>(a, p, plan, s);
    case FQ_ACT_SILU: return launch_wide_act<FQ_ACT_SILU>(a, p, plan, s);
    default: return launch_wide_act<FQ_ACT_NONE>(a, p, plan, s);
  }
}

}  // namespace

bool launch_matmul_fused(const MatmulArgs& given, const MatmulPlan& plan, int dtype, cudaStream_t s) {
  const MatmulArgs a = valid_strides(given);
  const MmArgs p = device_args(a, dtype);
  switch (plan.rows) {
    case 16: return launch_narrow<16, true>(a, p, plan, s);
    case 32: return launch_narrow<32, true>(a, p, plan, s);
    case 64: return launch_narrow<64, true>(a, p, plan, s);
    case 128: return launch_narrow<128, true>(a, p, plan, s);
    default: return launch_wide_any(a, p, plan, s);
  }
}

}  // namespace fq
