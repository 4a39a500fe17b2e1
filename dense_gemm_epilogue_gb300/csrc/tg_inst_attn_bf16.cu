// Attention kernels with BF16 operands.
#include "tg_inst_attn.cuh"

namespace tg {
cudaError_t launch_attn_forward_bf16(const AttnForward &a, int tiles_per_cta, int device, cudaStream_t stream) {
    return launch_attn_forward_kind<Kind::BF16>(a, tiles_per_cta, device, stream);
}
cudaError_t launch_attn_backward_bf16(const AttnBackward &a, const AttnDelta &d, int device, cudaStream_t stream) {
    return launch_attn_backward_kind<Kind::BF16>(a, d, device, stream);
}
}  // namespace tg
