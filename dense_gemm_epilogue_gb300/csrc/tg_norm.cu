// Layer norm over rows, forward and backward.
//
//   y = (x - mean) rstd gamma + beta,  mean = sum x / n,
//   rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//   a = dy gamma,  xh = (x - mean) rstd
//   dx = rstd (a - sum a / n - xh sum (a xh) / n)
//   dgamma = sum over rows of dy xh,  dbeta = sum over rows of dy
//
// Bound: memory; forward reads and writes each row once, backward reads x and
// dy and writes dx once.  A row stays in registers (16 elements a thread)
// between its statistics and its output, so nothing is read twice; the
// variance is the second moment about the mean just found, not a difference
// of large sums.  A group of 32, 128, 256 or 512 threads takes a row of up to
// 512, 2048, 4096 or 8192 columns; a cluster of 2, 4 or 8 blocks of 512
// shares longer rows (to 65536) and adds its partial sums through distributed
// shared memory.  All sums are FP32.
//
// Backward keeps each thread's columns fixed over all rows of its group, so
// the column sums dgamma and dbeta accumulate in registers and leave the block
// once; tg_colsum_finish_kernel adds the blocks' partials in a fixed order.
// No atomics: repeated calls agree bit for bit.  Two or three rows
// are in flight behind the one in work (NormRows), so that their loads overlap
// its reductions.
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/tg_gemm.h"
#include "tg_host.h"
#include "tg_rows.cuh"

namespace tg {

constexpr int NORM_PER = 16;  // elements of a row per thread

struct NormParams {
    int64_t m, n;
    const void *x, *dy;
    int64_t ldx, lddy;
    const float *gamma, *beta;
    float eps;
    void *y;  // forward: y; backward: dx
    int64_t ldy;
    float *mean, *rstd;              // forward outputs (may be NULL)
    const float *mean_in, *rstd_in;  // backward inputs
    float *pgamma, *pbeta;           // backward: partial column sums (NULL: not wanted)
    float inv_n;
};

// A thread's 16 elements of a row.  VEC: 16-byte vectors, vector v at column
// (v * THREADS + t) * VW.  Else single elements, element i at i * THREADS + t.
template <class Ty, int THREADS, bool VEC>
struct NormCols {
    static constexpr int VW = Ty::VW;
    __device__ __forceinline__ static int at(int i, int t) {
        return VEC ? ((i / VW) * THREADS + t) * VW + i % VW : i * THREADS + t;
    }
    __device__ __forceinline__ static void store(typename Ty::T *row, int t, int n,
                                                 const float (&y)[NORM_PER]) {
        if constexpr (VEC) {
#pragma unroll
            for (int v = 0; v < NORM_PER / VW; ++v) {
                const int c = (v * THREADS + t) * VW;
                if (c < n) row_store<Ty>(row, c, n, y + v * VW);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NORM_PER; ++i) {
                const int c = i * THREADS + t;
                if (c < n) row[c] = Ty::down(y[i]);
            }
        }
    }
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows on their way: MATS matrices' rows r, r + groups, ... of this group.
// VEC: each thread copies its own vectors into its own slots of a DEPTH-row
// ring in shared memory (cp.async, zero fill past the row's end) and reads
// them back itself, so no barrier is needed and DEPTH - 1 rows are in flight
// without a register.  Else: one row ahead, in registers.
template <class Ty, int THREADS, bool VEC, int MATS, int DEPTH>
struct NormRows {
    using T = typename Ty::T;
    static constexpr int VW = Ty::VW, VECS = NORM_PER / VW;
    const T *base[MATS];
    int64_t ld[MATS];
    int64_t m, groups;
    int n, t, slot;
    uint4 *ring;
    T ahead[MATS][VEC ? 1 : NORM_PER];

    __device__ __forceinline__ void ask(int64_t r, int at) {
        if constexpr (VEC) {
            if (r < m) {
#pragma unroll
                for (int a = 0; a < MATS; ++a) {
                    const T *row = base[a] + r * ld[a];
#pragma unroll
                    for (int v = 0; v < VECS; ++v) {
                        const int c = (v * THREADS + t) * VW;
                        const int left = n - c;
                        const uint32_t bytes =
                            left >= VW ? 16u : (left > 0 ? (uint32_t)(left * (int)sizeof(T)) : 0u);
                        cp_async_16(smem_u32(ring + ((at * MATS + a) * VECS + v) * blockDim.x + threadIdx.x),
                                    left > 0 ? row + c : row, bytes);
                    }
                }
            }
            cp_async_commit();
        } else {
            if (r < m) {
#pragma unroll
                for (int a = 0; a < MATS; ++a) {
                    const T *row = base[a] + r * ld[a];
#pragma unroll
                    for (int i = 0; i < NORM_PER; ++i) {
                        const int c = i * THREADS + t;
                        ahead[a][i] = c < n ? __ldcs(row + c) : (T)0;
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void start(int64_t first) {
        slot = 0;
#pragma unroll
        for (int d = 0; d < (VEC ? DEPTH - 1 : 1); ++d) ask(first + d * groups, d);
    }
    // This row's values, with the row after the last one asked for set off.
    __device__ __forceinline__ void take(int64_t r, float (&y)[MATS][NORM_PER]) {
        if constexpr (VEC) {
            cp_async_wait<DEPTH - 2>();
#pragma unroll
            for (int a = 0; a < MATS; ++a)
#pragma unroll
                for (int v = 0; v < VECS; ++v)
                    row_unpack<Ty>(ring[((slot * MATS + a) * VECS + v) * blockDim.x + threadIdx.x],
                                   y[a] + v * VW);
            ask(r + (DEPTH - 1) * groups, slot == 0 ? DEPTH - 1 : slot - 1);
            slot = slot + 1 == DEPTH ? 0 : slot + 1;
        } else {
#pragma unroll
            for (int a = 0; a < MATS; ++a)
#pragma unroll
                for (int i = 0; i < NORM_PER; ++i) y[a][i] = Ty::up(ahead[a][i]);
            ask(r + groups, 0);
        }
    }
};

constexpr int NORM_DEPTH = 4, NORM_BACK_DEPTH = 3;

__device__ __forceinline__ float2 warp_sum2(float2 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    return v;
}

// Sum of two values over the group of TR threads, times the cluster's CS
// blocks.  `turn` alternates between two buffers, so one barrier per call
// suffices: a buffer is written again two calls later, after every reader
// has passed the barrier in between.
template <int TR, int CS>
struct GroupSum {
    float2 *warps;   // [2][16]
    float2 *blocks;  // [2][8]
    int turn;
    __device__ __forceinline__ float2 operator()(float2 v) {
        v = warp_sum2(v);
        if constexpr (TR > 32) {
            const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
            if (lane == 0) warps[turn * 16 + w] = v;
            __syncthreads();
            v = lane < TR / 32 ? warps[turn * 16 + lane] : make_float2(0.0f, 0.0f);
            v = warp_sum2(v);
            if constexpr (CS > 1) {
                if (threadIdx.x < CS) {
                    const uint32_t dst = map_shared_rank(
                        smem_u32(blocks + turn * 8 + cluster_ctarank()), threadIdx.x);
                    st_cluster_u32(dst, __float_as_uint(v.x));
                    st_cluster_u32(dst + 4, __float_as_uint(v.y));
                }
                cluster_sync_all();
                v = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int b = 0; b < CS; ++b) {
                    v.x += blocks[turn * 8 + b].x;
                    v.y += blocks[turn * 8 + b].y;
                }
            }
            turn ^= 1;
        }
        return v;
    }
};

template <int TR>
constexpr int norm_block() {
    return TR < 128 ? 128 : TR;
}

template <class Ty, int TR, int CS, bool VEC>
__global__ void __launch_bounds__(norm_block<TR>()) tg_norm_kernel(const NormParams p) {
    using T = typename Ty::T;
    extern __shared__ uint4 ring[];
    __shared__ float2 warps[2 * 16];
    __shared__ float2 blocks[2 * 8];
    constexpr int GROUPS = norm_block<TR>() / TR;
    constexpr int THREADS = TR * CS;  // threads that share a row
    using Cols = NormCols<Ty, THREADS, VEC>;
    const int t = (int)(threadIdx.x % TR) + (CS > 1 ? (int)cluster_ctarank() * TR : 0);
    const int64_t group = ((int64_t)blockIdx.x / CS) * GROUPS + threadIdx.x / TR;
    const int64_t groups = ((int64_t)gridDim.x / CS) * GROUPS;
    const int n = (int)p.n;
    GroupSum<TR, CS> sum{warps, blocks, 0};
    griddep_launch();
    if constexpr (CS > 1) cluster_sync_all();  // every block runs before its memory is written
    griddep_wait();
    NormRows<Ty, THREADS, VEC, 1, NORM_DEPTH> rows;
    rows.base[0] = static_cast<const T *>(p.x);
    rows.ld[0] = p.ldx;
    rows.m = p.m;
    rows.groups = groups;
    rows.n = n;
    rows.t = t;
    rows.ring = ring;
    rows.start(group);
    // The group's columns never change: gamma and beta stay in registers.
    float gam[NORM_PER], bet[NORM_PER];
#pragma unroll
    for (int i = 0; i < NORM_PER; ++i) {
        const int c = Cols::at(i, t);
        gam[i] = (p.gamma && c < n) ? __ldg(p.gamma + c) : 1.0f;
        bet[i] = (p.beta && c < n) ? __ldg(p.beta + c) : 0.0f;
    }
    T *y = static_cast<T *>(p.y);
    const bool whole = n == THREADS * NORM_PER;
    for (int64_t r = group; r < p.m; r += groups) {
        float w[1][NORM_PER];
        rows.take(r, w);
        float(&v)[NORM_PER] = w[0];
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NORM_PER; ++i) s += v[i];
        const float mean = sum(make_float2(s, 0.0f)).x * p.inv_n;
#pragma unroll
        for (int i = 0; i < NORM_PER; ++i) v[i] -= mean;
        if (!whole) {
#pragma unroll
            for (int i = 0; i < NORM_PER; ++i)
                if (Cols::at(i, t) >= n) v[i] = 0.0f;
        }
        float q = 0.0f;
#pragma unroll
        for (int i = 0; i < NORM_PER; ++i) q = fmaf(v[i], v[i], q);
        const float var = sum(make_float2(q, 0.0f)).x * p.inv_n;
        const float rstd = 1.0f / sqrtf(var + p.eps);
        if (t == 0) {
            if (p.mean) p.mean[r] = mean;
            if (p.rstd) p.rstd[r] = rstd;
        }
#pragma unroll
        for (int i = 0; i < NORM_PER; ++i) v[i] = fmaf(v[i] * rstd, gam[i], bet[i]);
        Cols::store(y + r * p.ldy, t, n, v);
    }
}

template <class Ty, int TR, int CS, bool VEC>
__global__ void __launch_bounds__(norm_block<TR>()) tg_norm_backward_kernel(const NormParams p) {
    using T = typename Ty::T;
    extern __shared__ uint4 ring[];
    __shared__ float2 warps[2 * 16];
    __shared__ float2 blocks[2 * 8];
    constexpr int GROUPS = norm_block<TR>() / TR;
    constexpr int THREADS = TR * CS;
    using Cols = NormCols<Ty, THREADS, VEC>;
    const int t = (int)(threadIdx.x % TR) + (CS > 1 ? (int)cluster_ctarank() * TR : 0);
    const int64_t group = ((int64_t)blockIdx.x / CS) * GROUPS + threadIdx.x / TR;
    const int64_t groups = ((int64_t)gridDim.x / CS) * GROUPS;
    const int n = (int)p.n;
    GroupSum<TR, CS> sum{warps, blocks, 0};
    griddep_launch();
    if constexpr (CS > 1) cluster_sync_all();
    griddep_wait();
    NormRows<Ty, THREADS, VEC, 2, NORM_BACK_DEPTH> rows;
    rows.base[0] = static_cast<const T *>(p.x);
    rows.base[1] = static_cast<const T *>(p.dy);
    rows.ld[0] = p.ldx;
    rows.ld[1] = p.lddy;
    rows.m = p.m;
    rows.groups = groups;
    rows.n = n;
    rows.t = t;
    rows.ring = ring;
    rows.start(group);
    T *dx = static_cast<T *>(p.y);
    float gam[NORM_PER], sg[NORM_PER], sb[NORM_PER];
#pragma unroll
    for (int i = 0; i < NORM_PER; ++i) {
        const int c = Cols::at(i, t);
        gam[i] = (p.gamma && c < n) ? __ldg(p.gamma + c) : 1.0f;
        sg[i] = sb[i] = 0.0f;
    }
    float nmean = group < p.m ? __ldg(p.mean_in + group) : 0.0f;
    float nrstd = group < p.m ? __ldg(p.rstd_in + group) : 0.0f;
    for (int64_t r = group; r < p.m; r += groups) {
        float w[2][NORM_PER];
        rows.take(r, w);
        float(&xh)[NORM_PER] = w[0];
        float(&d)[NORM_PER] = w[1];
        const float mean = nmean, rstd = nrstd;
        if (r + groups < p.m) {
            nmean = __ldg(p.mean_in + r + groups);
            nrstd = __ldg(p.rstd_in + r + groups);
        }
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NORM_PER; ++i) {
            // Columns past the row's end hold dy = 0 and add nothing.
            const float h = (xh[i] - mean) * rstd;
            xh[i] = h;
            sg[i] = fmaf(d[i], h, sg[i]);
            sb[i] += d[i];
            d[i] *= gam[i];
            s1 += d[i];
            s2 = fmaf(d[i], h, s2);
        }
        const float2 s = sum(make_float2(s1, s2));
        if (dx) {
            const float c1 = s.x * p.inv_n, c2 = s.y * p.inv_n;
#pragma unroll
            for (int i = 0; i < NORM_PER; ++i) d[i] = rstd * (d[i] - fmaf(xh[i], c2, c1));
            Cols::store(dx + r * p.ldy, t, n, d);
        }
    }
#pragma unroll
    for (int i = 0; i < NORM_PER; ++i) {
        const int c = Cols::at(i, t);
        if (c < n) {
            if (p.pgamma) p.pgamma[group * p.n + c] = sg[i];
            if (p.pbeta) p.pbeta[group * p.n + c] = sb[i];
        }
    }
}

}  // namespace tg

namespace {

using namespace tg;

constexpr int64_t kNormMaxCols = 65536;

// Threads of a row's group and blocks of its cluster.
struct NormShape {
    int tr, cs;
};
NormShape norm_shape(int64_t n) {
    if (n <= 32 * NORM_PER) return {32, 1};
    if (n <= 128 * NORM_PER) return {128, 1};
    if (n <= 256 * NORM_PER) return {256, 1};
    if (n <= 512 * NORM_PER) return {512, 1};
    if (n <= 2 * 512 * NORM_PER) return {512, 2};
    if (n <= 4 * 512 * NORM_PER) return {512, 4};
    return {512, 8};
}

// Row groups of a launch: at most `waves` blocks per SM (rounded to clusters),
// no more groups than rows.
int64_t norm_grid(const NormShape &s, int64_t m, int sms, int per_sm) {
    const int64_t groups = s.tr < 128 ? 128 / s.tr : 1;  // per block
    int64_t blocks = (m + groups - 1) / groups;
    int64_t cap = (int64_t)sms * per_sm / s.cs;
    if (cap < 1) cap = 1;
    if (blocks > cap) blocks = cap;
    return blocks * s.cs;
}

// Blocks per SM: what registers and rings leave room for; in backward also few
// enough that the partial column sums (8 n bytes per group, written and read
// once) stay small beside the rows.
int forward_per_sm(const NormShape &s) { return s.tr >= 512 ? 1 : s.tr == 256 ? 3 : 6; }
int backward_per_sm(const NormShape &s) { return s.tr >= 512 ? 1 : s.tr == 256 ? 2 : 4; }
int64_t backward_groups(int64_t m, int64_t n, int sms) {
    const NormShape s = norm_shape(n);
    const int64_t per_block = s.tr < 128 ? 128 / s.tr : 1;
    return norm_grid(s, m, sms, backward_per_sm(s)) / s.cs * per_block;
}

template <class Ty, int TR, int CS, bool VEC>
cudaError_t launch_shape(const NormParams &p, bool backward, int64_t grid, int device,
                         cudaStream_t stream) {
    constexpr int ROW = norm_block<TR>() * NORM_PER * (int)sizeof(typename Ty::T);
    constexpr int SMEM = VEC ? NORM_DEPTH * ROW : 0, SMEM_BACK = VEC ? NORM_BACK_DEPTH * 2 * ROW : 0;
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << device;
    if (VEC && !(done.load(std::memory_order_acquire) & bit)) {
        cudaError_t e = cudaFuncSetAttribute(tg_norm_kernel<Ty, TR, CS, VEC>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(tg_norm_backward_kernel<Ty, TR, CS, VEC>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BACK);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_acq_rel);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CS;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(norm_block<TR>(), 1, 1);
    cfg.dynamicSmemBytes = backward ? SMEM_BACK : SMEM;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = CS > 1 ? 2 : 1;
    return backward ? cudaLaunchKernelEx(&cfg, tg_norm_backward_kernel<Ty, TR, CS, VEC>, p)
                    : cudaLaunchKernelEx(&cfg, tg_norm_kernel<Ty, TR, CS, VEC>, p);
}

template <class Ty, bool VEC>
cudaError_t launch_type(const NormParams &p, bool backward, int64_t grid, int device,
                        cudaStream_t stream) {
    const NormShape s = norm_shape(p.n);
    if (s.tr == 32) return launch_shape<Ty, 32, 1, VEC>(p, backward, grid, device, stream);
    if (s.tr == 128) return launch_shape<Ty, 128, 1, VEC>(p, backward, grid, device, stream);
    if (s.tr == 256) return launch_shape<Ty, 256, 1, VEC>(p, backward, grid, device, stream);
    if (s.cs == 1) return launch_shape<Ty, 512, 1, VEC>(p, backward, grid, device, stream);
    if (s.cs == 2) return launch_shape<Ty, 512, 2, VEC>(p, backward, grid, device, stream);
    if (s.cs == 4) return launch_shape<Ty, 512, 4, VEC>(p, backward, grid, device, stream);
    return launch_shape<Ty, 512, 8, VEC>(p, backward, grid, device, stream);
}

cudaError_t launch_norm(const NormParams &p, tg_out_dtype t, bool backward, bool vec, int64_t grid,
                        int device, cudaStream_t stream) {
    if (t == TG_OUT_F32)
        return vec ? launch_type<TypeF32, true>(p, backward, grid, device, stream)
                   : launch_type<TypeF32, false>(p, backward, grid, device, stream);
    if (t == TG_OUT_BF16)
        return vec ? launch_type<TypeBF16, true>(p, backward, grid, device, stream)
                   : launch_type<TypeBF16, false>(p, backward, grid, device, stream);
    return vec ? launch_type<TypeF16, true>(p, backward, grid, device, stream)
               : launch_type<TypeF16, false>(p, backward, grid, device, stream);
}

bool norm_type_ok(tg_out_dtype t) { return t == TG_OUT_F32 || t == TG_OUT_BF16 || t == TG_OUT_F16; }
int type_bytes(tg_out_dtype t) { return t == TG_OUT_F32 ? 4 : 2; }

// A rows x n matrix of the type: present, element-aligned, ld >= n.
bool matrix_ok(const void *p, int64_t ld, int64_t n, int e) {
    return p && (uintptr_t)p % e == 0 && ld >= n && ld < ((int64_t)1 << 40);
}
bool vec_ok(const void *p, int64_t ld, int e) {
    return (uintptr_t)p % 16 == 0 && (ld * e) % 16 == 0;
}
bool f32_ok(const void *p) { return (uintptr_t)p % 4 == 0; }

}  // namespace

extern "C" tg_status tg_layer_norm(int64_t M, int64_t N, const void *X, int64_t ldx,
                                   const float *gamma, const float *beta, float eps, void *Y,
                                   int64_t ldy, float *mean, float *rstd, tg_out_dtype dtype,
                                   void *stream) {
    if (M < 0 || N < 0 || M > INT32_MAX || !norm_type_ok(dtype) || !(eps >= 0.0f))
        return TG_ERR_INVALID_VALUE;
    if (N > kNormMaxCols) return TG_ERR_UNSUPPORTED;
    if (M == 0) return TG_OK;
    if (N == 0) return TG_ERR_INVALID_VALUE;  // the mean of no elements
    const int e = type_bytes(dtype);
    if (!matrix_ok(X, ldx, N, e) || !matrix_ok(Y, ldy, N, e)) return TG_ERR_INVALID_VALUE;
    if (!f32_ok(gamma) || !f32_ok(beta) || !f32_ok(mean) || !f32_ok(rstd)) return TG_ERR_INVALID_VALUE;
    tg::host::Device dev;
    tg_status st = tg::host::device(&dev);
    if (st != TG_OK) return st;
    NormParams p = {};
    p.m = M;
    p.n = N;
    p.x = X;
    p.ldx = ldx;
    p.gamma = gamma;
    p.beta = beta;
    p.eps = eps;
    p.y = Y;
    p.ldy = ldy;
    p.mean = mean;
    p.rstd = rstd;
    p.inv_n = 1.0f / (float)N;
    const NormShape s = norm_shape(N);
    const int64_t grid = norm_grid(s, M, dev.sms, forward_per_sm(s));
    const bool vec = vec_ok(X, ldx, e) && vec_ok(Y, ldy, e);
    return launch_norm(p, dtype, false, vec, grid, dev.id, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? TG_OK
               : TG_ERR_CUDA;
}

extern "C" int64_t tg_layer_norm_backward_workspace_bytes(int64_t M, int64_t N) {
    if (M < 0 || N < 0 || M > INT32_MAX || N > kNormMaxCols) return -1;
    tg::host::Device dev;
    if (tg::host::device(&dev) != TG_OK) return -1;
    return M == 0 || N == 0 ? 0 : 2 * 4 * N * backward_groups(M, N, dev.sms);
}

extern "C" tg_status tg_layer_norm_backward(int64_t M, int64_t N, const void *dY, int64_t lddy,
                                            const void *X, int64_t ldx, const float *gamma,
                                            const float *mean, const float *rstd, void *dX,
                                            int64_t lddx, float *dgamma, float *dbeta,
                                            tg_out_dtype dtype, void *workspace,
                                            int64_t workspace_bytes, void *stream_ptr) {
    if (M < 0 || N < 0 || M > INT32_MAX || !norm_type_ok(dtype) || workspace_bytes < 0)
        return TG_ERR_INVALID_VALUE;
    if (N > kNormMaxCols) return TG_ERR_UNSUPPORTED;
    if (!f32_ok(gamma) || !f32_ok(mean) || !f32_ok(rstd) || !f32_ok(dgamma) || !f32_ok(dbeta))
        return TG_ERR_INVALID_VALUE;
    if (N == 0) return M == 0 ? TG_OK : TG_ERR_INVALID_VALUE;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    const int e = type_bytes(dtype);
    if (M > 0) {
        if (!matrix_ok(X, ldx, N, e) || !matrix_ok(dY, lddy, N, e) || !mean || !rstd)
            return TG_ERR_INVALID_VALUE;
        if (dX && !matrix_ok(dX, lddx, N, e)) return TG_ERR_INVALID_VALUE;
    }
    if (!dX && !dgamma && !dbeta) return TG_OK;
    tg::host::Device dev;
    tg_status st = tg::host::device(&dev);
    if (st != TG_OK) return st;
    const bool sums = dgamma || dbeta;
    int64_t groups = 0;
    if (M > 0) {
        groups = backward_groups(M, N, dev.sms);
        if (sums && (!workspace || (uintptr_t)workspace % 4 || workspace_bytes < 2 * 4 * N * groups))
            return TG_ERR_INVALID_VALUE;
        NormParams p = {};
        p.m = M;
        p.n = N;
        p.x = X;
        p.ldx = ldx;
        p.dy = dY;
        p.lddy = lddy;
        p.gamma = gamma;
        p.mean_in = mean;
        p.rstd_in = rstd;
        p.y = dX;
        p.ldy = lddx;
        p.inv_n = 1.0f / (float)N;
        if (dgamma) p.pgamma = static_cast<float *>(workspace);
        if (dbeta) p.pbeta = static_cast<float *>(workspace) + groups * N;
        const NormShape s = norm_shape(N);
        const bool vec = vec_ok(X, ldx, e) && vec_ok(dY, lddy, e) && (!dX || vec_ok(dX, lddx, e));
        if (launch_norm(p, dtype, true, vec, norm_grid(s, M, dev.sms, backward_per_sm(s)), dev.id,
                        stream) !=
            cudaSuccess)
            return TG_ERR_CUDA;
    }
    if (!sums) return TG_OK;
    // M == 0: no groups, the sums are zero.
    const float *w = static_cast<const float *>(workspace);
    return tg::host::colsum_finish(dgamma ? w : w + groups * N, dgamma && dbeta ? w + groups * N : nullptr,
                                   (int32_t)groups, N, dgamma ? dgamma : dbeta,
                                   dgamma && dbeta ? dbeta : nullptr, stream) == cudaSuccess
               ? TG_OK
               : TG_ERR_CUDA;
}
