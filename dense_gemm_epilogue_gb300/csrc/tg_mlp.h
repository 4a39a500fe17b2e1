// Internal interface between the feed-forward front end (tg_mlp.cu) and the
// kernel instantiations (one translation unit per operand type).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include "tg_kernel_mlp.cuh"
#include "tg_kernel_stream.cuh"

namespace tg {

// The products the tile kernel runs (operand majorness and epilogue).
enum class MlpOp : int {
    LINEAR = 0,  // K-major x K-major; bias, activation, residual, saved Z
    GATED = 1,   // K-major x two K-major; act(g) * u, saved G and U
    DGRAD = 2,   // K-major x MN-major (one or two operand pairs)
    WGRAD = 3,   // MN-major x MN-major (one or two entries)
};

struct MlpLaunch {
    MlpMaps maps;
    MlpParams p;
    MlpOp op;
    int cg;        // CTAs per team (1 or 2)
    int block_n;
    int grid;      // CTAs (a multiple of cg)
    int device;
    cudaStream_t stream;
};

struct StreamLaunch {
    StreamMaps maps;
    StreamParams p;
    int nt;
    StreamOp op;
    int grid;
    int device;
    cudaStream_t stream;
};

cudaError_t launch_mlp_bf16_cg1(const MlpLaunch &a);
cudaError_t launch_mlp_bf16_cg2(const MlpLaunch &a);
cudaError_t launch_mlp_fp16_cg1(const MlpLaunch &a);
cudaError_t launch_mlp_fp16_cg2(const MlpLaunch &a);
cudaError_t launch_stream_bf16(const StreamLaunch &a);
cudaError_t launch_stream_fp16(const StreamLaunch &a);

}  // namespace tg
