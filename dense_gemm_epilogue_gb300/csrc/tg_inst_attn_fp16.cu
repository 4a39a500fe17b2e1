// Attention kernels with FP16 operands.
#include "tg_inst_attn.cuh"

namespace tg {
cudaError_t launch_attn_forward_fp16(const AttnForward &a, int tiles_per_cta, int device, cudaStream_t stream) {
    return launch_attn_forward_kind<Kind::FP16>(a, tiles_per_cta, device, stream);
}
cudaError_t launch_attn_backward_fp16(const AttnBackward &a, const AttnDelta &d, int device, cudaStream_t stream) {
    return launch_attn_backward_kind<Kind::FP16>(a, d, device, stream);
}
}  // namespace tg
