// Weight-streaming kernels on FP16 operands (their own translation unit).
#include "tg_inst_mlp.cuh"

namespace tg {
cudaError_t launch_stream_fp16(const StreamLaunch &a) { return launch_stream_kind<Kind::FP16>(a); }
}  // namespace tg
