// Feed-forward tile kernels on BF16 operands, CTA pairs (their own translation unit).
#include "tg_inst_mlp.cuh"

namespace tg {
cudaError_t launch_mlp_bf16_cg2(const MlpLaunch &a) { return launch_mlp_kind<Kind::BF16, 2>(a); }
}  // namespace tg
