// Weight-streaming kernels on BF16 operands (their own translation unit).
#include "tg_inst_mlp.cuh"

namespace tg {
cudaError_t launch_stream_bf16(const StreamLaunch &a) { return launch_stream_kind<Kind::BF16>(a); }
}  // namespace tg
