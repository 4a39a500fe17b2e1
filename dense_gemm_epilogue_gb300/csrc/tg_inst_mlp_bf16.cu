// Feed-forward kernels on BF16 operands (their own translation unit).
#include "tg_inst_mlp.cuh"

namespace tg {
cudaError_t launch_mlp_bf16(const MlpLaunch &a) { return launch_mlp_kind<Kind::BF16>(a); }
}  // namespace tg
