// Instantiation and launch of the feed-forward kernels for one operand type.
#pragma once

#include <atomic>
#include "tg_mlp.h"

namespace tg {

// Dynamic shared memory opt-in, once per device; `max_clusters` (when given)
// receives how many clusters the device holds at once.
template <class K>
static cudaError_t mlp_configure(K kernel, int smem, int device, std::atomic<uint64_t> &done,
                                 cudaLaunchConfig_t *cfg, int *max_clusters) {
    const uint64_t bit = (device >= 0 && device < 64) ? (1ull << device) : 0;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (max_clusters) {
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, kernel, cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        if (bit) max_clusters[device] = n;
    }
    if (bit) done.fetch_or(bit, std::memory_order_acq_rel);
    return cudaSuccess;
}

template <Kind KD, int CG, int BN, int AM, int BM, MlpEpi EP>
static cudaError_t launch_mlp_one(const MlpLaunch &a) {
    using C = MlpConfig<KD, CG, BN, AM, BM, EP>;
    auto kernel = tg_mlp_kernel<KD, CG, BN, AM, BM, EP>;
    static std::atomic<uint64_t> done{0};
    static int max_clusters[64] = {0};
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(CG, 1, 1);
    cfg.blockDim = dim3(C::NUM_THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = a.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = mlp_configure(kernel, C::SMEM_BYTES, a.device, done, &cfg, max_clusters);
    if (e != cudaSuccess) return e;
    int grid = a.grid;
    if (a.device >= 0 && a.device < 64 && grid > CG * max_clusters[a.device])
        grid = CG * max_clusters[a.device];
    cfg.gridDim = dim3(grid < CG ? CG : grid, 1, 1);
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a.maps, a.p);
}

template <Kind KD, int CG, int BN>
static cudaError_t launch_mlp_bn(const MlpLaunch &a) {
    if constexpr (CG == 1 || BN == 256) {  // (256 x 128 pair tiles: gradients only)
        if (a.op == MlpOp::LINEAR) return launch_mlp_one<KD, CG, BN, 0, 0, MlpEpi::LINEAR>(a);
        if (a.op == MlpOp::GATED) return launch_mlp_one<KD, CG, BN, 0, 0, MlpEpi::GATED>(a);
    }
    switch (a.op) {
    case MlpOp::DGRAD: return launch_mlp_one<KD, CG, BN, 0, 1, MlpEpi::PLAIN>(a);
    case MlpOp::WGRAD: return launch_mlp_one<KD, CG, BN, 1, 1, MlpEpi::PLAIN>(a);
    default: break;
    }
    return cudaErrorInvalidValue;
}

template <Kind KD, int CG>
static cudaError_t launch_mlp_kind(const MlpLaunch &a) {
    return a.block_n == 256 ? launch_mlp_bn<KD, CG, 256>(a) : launch_mlp_bn<KD, CG, 128>(a);
}

template <Kind KD, int NT, StreamOp OP>
static cudaError_t launch_stream_one(const StreamLaunch &a) {
    using C = StreamConfig<KD, NT, OP>;
    auto kernel = tg_stream_kernel<KD, NT, OP>;
    static std::atomic<uint64_t> done{0};
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(a.grid, 1, 1);
    cfg.blockDim = dim3(C::NUM_THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = a.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = mlp_configure(kernel, C::SMEM_BYTES, a.device, done, &cfg, (int *)nullptr);
    if (e != cudaSuccess) return e;
    return cudaLaunchKernelEx(&cfg, kernel, a.maps, a.p);
}

template <Kind KD, StreamOp OP>
static cudaError_t launch_stream_nt(const StreamLaunch &a) {
    switch (a.nt) {
    case 16: return launch_stream_one<KD, 16, OP>(a);
    case 32: return launch_stream_one<KD, 32, OP>(a);
    default: break;
    }
    if constexpr (OP != StreamOp::GATED) return launch_stream_one<KD, 64, OP>(a);
    return cudaErrorInvalidValue;  // (gated: up to 32 tokens)
}

template <Kind KD>
static cudaError_t launch_stream_kind(const StreamLaunch &a) {
    switch (a.op) {
    case StreamOp::GATED: return launch_stream_nt<KD, StreamOp::GATED>(a);
    case StreamOp::DGRAD: return launch_stream_nt<KD, StreamOp::DGRAD>(a);
    default: return launch_stream_nt<KD, StreamOp::LINEAR>(a);
    }
}

}  // namespace tg
