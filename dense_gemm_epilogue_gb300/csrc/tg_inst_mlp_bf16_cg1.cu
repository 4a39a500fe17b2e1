// Feed-forward tile kernels on BF16 operands, single CTAs (their own translation unit).
#include "tg_inst_mlp.cuh"

namespace tg {
cudaError_t launch_mlp_bf16_cg1(const MlpLaunch &a) { return launch_mlp_kind<Kind::BF16, 1>(a); }
}  // namespace tg
