// Feed-forward tile kernels on FP16 operands, CTA pairs (their own translation unit).
#include "tg_inst_mlp.cuh"

namespace tg {
cudaError_t launch_mlp_fp16_cg2(const MlpLaunch &a) { return launch_mlp_kind<Kind::FP16, 2>(a); }
}  // namespace tg
