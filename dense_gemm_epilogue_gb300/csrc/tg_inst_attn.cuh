// Instantiation and launch of the attention kernels for one operand type.
#pragma once

#include <atomic>
#include "tg_attn.h"
#include "tg_kernel_attn_bwd.cuh"

namespace tg {

template <class K>
static cudaError_t attn_smem(K kernel, int smem, int device, std::atomic<uint64_t> &done) {
    const uint64_t bit = (device >= 0 && device < 64) ? (1ull << device) : 0;
    if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

template <class P>
static cudaError_t attn_launch(void (*kernel)(const P), dim3 grid, int threads, int smem,
                               cudaStream_t stream, const P &p) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <Kind KD, int DT, int NQ>
static cudaError_t launch_attn_one(const AttnForward &a, int device, cudaStream_t stream) {
    using C = AttnConfig<KD, DT, NQ>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = attn_smem(tg_attn_kernel<KD, DT, NQ>, C::SMEM_BYTES, device, done);
    if (e != cudaSuccess) return e;
    return attn_launch<AttnForward>(tg_attn_kernel<KD, DT, NQ>,
                                    dim3((unsigned)(a.tiles * a.h.kv_heads * a.splits)), C::NUM_THREADS,
                                    C::SMEM_BYTES, stream, a);
}

template <Kind KD>
static cudaError_t launch_attn_forward_kind(const AttnForward &a, int nq, int device, cudaStream_t stream) {
    cudaError_t e;
    if (a.h.dim <= 64)
        e = nq == 2 ? launch_attn_one<KD, 64, 2>(a, device, stream) : launch_attn_one<KD, 64, 1>(a, device, stream);
    else
        e = nq == 2 ? launch_attn_one<KD, 128, 2>(a, device, stream) : launch_attn_one<KD, 128, 1>(a, device, stream);
    if (e != cudaSuccess || a.splits == 1) return e;
    // A block a row where that is a few blocks an SM at most.
    const int64_t tiles = (int64_t)a.tiles * a.h.kv_heads;
    const bool wide = tiles * a.join_rows <= 1024;
    const dim3 grid((unsigned)tiles, wide ? a.join_rows : (a.join_rows + JOIN_WARPS - 1) / JOIN_WARPS);
    return wide ? attn_launch<AttnForward>(tg_attn_join_kernel<KD, true>, grid, 32 * JOIN_WARPS, 0, stream, a)
                : attn_launch<AttnForward>(tg_attn_join_kernel<KD, false>, grid, 32 * JOIN_WARPS, 0, stream, a);
}

template <Kind KD, int DT>
static cudaError_t launch_attn_backward_dim(AttnBackward a, int device, cudaStream_t stream) {
    using CK = AttnKeysConfig<KD, DT>;
    using CR = AttnRowsConfig<KD, DT>;
    constexpr int SMEM = CK::SMEM_BYTES > CR::SMEM_BYTES ? CK::SMEM_BYTES : CR::SMEM_BYTES;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = attn_smem(tg_attn_backward_kernel<KD, DT>, SMEM, device, done);
    if (e != cudaSuccess) return e;
    const int64_t keys = a.dk.ptr || a.dv.ptr ? (int64_t)a.blocks * a.h.kv_heads * a.key_parts : 0;
    const int64_t rows = a.dq.ptr ? (int64_t)a.tiles * a.h.kv_heads * a.row_parts : 0;
    if (keys + rows == 0) return cudaSuccess;
    a.key_ctas = (int32_t)keys;
    return attn_launch<AttnBackward>(tg_attn_backward_kernel<KD, DT>, dim3((unsigned)(keys + rows)), CK::NUM_THREADS,
                                     SMEM, stream, a);
}

template <Kind KD>
static cudaError_t launch_attn_backward_kind(const AttnBackward &a, const AttnDelta &d, int device,
                                             cudaStream_t stream) {
    if (d.rows > 0) {
        const int64_t grid = ((int64_t)d.rows * d.heads + DELTA_THREADS / 16 - 1) / (DELTA_THREADS / 16);
        const cudaError_t e = attn_launch<AttnDelta>(tg_attn_delta_kernel<KD>, dim3((unsigned)grid), DELTA_THREADS, 0, stream, d);
        if (e != cudaSuccess) return e;
    }
    const cudaError_t e = a.h.dim <= 64 ? launch_attn_backward_dim<KD, 64>(a, device, stream)
                                        : launch_attn_backward_dim<KD, 128>(a, device, stream);
    const int64_t keys = a.key_parts > 1 ? (int64_t)a.blocks * a.h.kv_heads : 0;
    const int64_t rows = a.row_parts > 1 ? (int64_t)a.tiles * a.h.kv_heads : 0;
    if (e != cudaSuccess || keys + rows == 0) return e;
    // (four blocks to a tile: 16 to 64 rows a warp would be a long chain of loads)
    return attn_launch<AttnBackward>(tg_attn_parts_kernel<KD>, dim3((unsigned)(keys + rows), 4), PARTS_THREADS, 0,
                                     stream, a);
}

}  // namespace tg
