// Feed-forward kernels on FP16 operands (their own translation unit).
#include "tg_inst_mlp.cuh"

namespace tg {
cudaError_t launch_mlp_fp16(const MlpLaunch &a) { return launch_mlp_kind<Kind::FP16>(a); }
}  // namespace tg
