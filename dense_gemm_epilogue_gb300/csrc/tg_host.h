// Host services shared by the operators' entry points: the device's state,
// the per-stream workspace, tensor-map encoding (defined in tg_gemm.cu) and the
// column sums' last step (in tg_mlp.cu).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include "../../include/tg_gemm.h"

namespace tg {
namespace host {

struct Device {
    int id = 0;
    int sms = 0;
    uint32_t *status = nullptr;
    uint64_t wait_limit_ns = 0;
};

// The current device (set up on first use); TG_ERR_UNSUPPORTED when it is not
// a compute capability 10.3 GPU.
tg_status device(Device *out);

// The workspace of (device, stream): room for `tiles` partial 256 x 256 FP32
// tiles; flags and the ticket counter, all zero between launches.
struct Scratch {
    float *ws = nullptr;
    int64_t tiles = 0;
    uint32_t *flags = nullptr;         // of the CTA-pair kernels (four per tile)
    uint32_t *ticket = nullptr;
    uint32_t *gate = nullptr;          // MlpParams::gate
    uint32_t *stream_flags = nullptr;  // of the weight-streaming kernel (kStreamFlags words)
};
constexpr int64_t kStreamFlags = 8 * 512;
tg_status scratch(const Device &dev, cudaStream_t stream, int64_t tiles, Scratch *out);
// Whether scratch() would have to allocate while the stream is being captured,
// which spoils the capture.
bool scratch_blocked(const Device &dev, cudaStream_t stream, int64_t tiles);

// 2-D tensor map of a row-major matrix of 2- or 4-byte elements: box of
// row_bytes (128 or 64, with the swizzle of that width) x box_rows, zero fill.
bool encode_rows(CUtensorMap *map, tg_out_dtype t, const void *base, int64_t rows, int64_t cols,
                 int64_t ld, int box_rows, int row_bytes = 128);

// out0[c] (and out1[c] when given) = sum over `parts` rows of the partials.
cudaError_t colsum_finish(const float *partial0, const float *partial1, int32_t parts, int64_t n,
                          float *out0, float *out1, cudaStream_t stream);

}  // namespace host
}  // namespace tg
