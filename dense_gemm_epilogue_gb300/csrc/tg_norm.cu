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
// between its statistics and its output, so nothing is read twice; the variance
// is the second moment about the mean just found, not a difference of large
// sums.  A group of 32 to 512 threads takes a row of up to 16 elements each; a
// cluster of 2, 4 or 8 blocks of 512 shares longer rows (to 65536) and adds its
// partial sums through distributed shared memory.  All sums are FP32.
//
// On 16-bit rows what stands between a row and the memory's rate is the number
// of instructions (a build with 8 elements a thread issued 36 per element
// backward, 26 forward, and ran at 0.63 of the copy rate whatever the
// occupancy).  So the arithmetic is on pairs of FP32 values (fma.rn.f32x2), rows
// are copied by pointers that advance by a constant, forward takes two rows per
// step through one reduction, and a thread holds 16 elements, over which a
// reduction's shuffles spread.
//
// Measured (a captured chain of calls, inputs past L2; the copy rate is 6.79 TB/s):
//   16384 x 4096 BF16        forward 42.4 us, 6.3 TB/s; backward 73.8 us, 5.5 TB/s
//   4096 x 16384 BF16        forward 89 us, 3.0 TB/s; backward 119 us, 3.4 TB/s: a
//                            cluster's barriers stand between the steps
//   8 x 4096 BF16            forward 3.1 us: two dependent reductions after a launch
//   4099 x 1001, odd rows    backward FP32 17.6 us, BF16 17.1 us; 16384 x 4097 BF16
//                            forward 155 us: 4-byte copies, single 16-bit loads
//
// Backward keeps each thread's columns fixed over all rows of its group, so
// the column sums dgamma and dbeta accumulate in registers; the block's groups
// add theirs in shared memory in order, and tg_colsum_finish_kernel adds the
// blocks' partials in order.  No atomics: repeated calls agree bit for bit.
// Two steps' rows are in flight behind the one in work (NormRows).
#include <cuda_runtime.h>

#include <atomic>

#include "../../include/tg_gemm.h"
#include "tg_host.h"
#include "tg_rows.cuh"

namespace tg {

constexpr int NORM_PER = 16;   // elements of a row per thread
constexpr int NORM_ROWS = 2;   // rows per step of the forward pass
constexpr int NORM_DEPTH = 3;  // steps in the ring: one in work, two in flight
constexpr int NORM_SM = 512;   // threads a SM (128 registers each)

// Two FP32 values in one 64-bit register, and the arithmetic on both at once.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void f2_split(F2 x, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ float sum2(F2 x) {
    float a, b;
    f2_split(x, a, b);
    return a + b;
}

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

// A thread's elements of a row.  VEC: 16-byte vectors, vector v at column
// (v * THREADS + t) * VW.  Else single elements, element i at i * THREADS + t.
template <class Ty, int THREADS, bool VEC>
struct NormCols {
    static constexpr int VW = Ty::VW;
    __device__ __forceinline__ static int at(int i, int t) {
        return VEC ? ((i / VW) * THREADS + t) * VW + i % VW : i * THREADS + t;
    }
    // Elements 2i, 2i + 1 as pair i.
    __device__ __forceinline__ static void store(typename Ty::T *row, int t, int n, bool whole,
                                                 const F2 (&y)[NORM_PER / 2]) {
        float e[NORM_PER];
#pragma unroll
        for (int i = 0; i < NORM_PER / 2; ++i) f2_split(y[i], e[2 * i], e[2 * i + 1]);
        if constexpr (VEC) {
            typename Ty::T *q = row + t * VW;
#pragma unroll
            for (int v = 0; v < NORM_PER / VW; ++v) {
                const int c = (v * THREADS + t) * VW;
                if (whole) row_store_vec<Ty>(q + v * THREADS * VW, e + v * VW);
                else if (c < n) row_store<Ty>(row, c, n, e + v * VW);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NORM_PER; ++i) {
                const int c = i * THREADS + t;
                if (c < n) row[c] = Ty::down(e[i]);
            }
        }
    }
};

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows on their way: two rows per step (two rows of x, or a row of x and one
// of dy), from pointers that advance by a constant.  Each thread copies its own
// vectors (or FP32 elements) into its own slots of a ring in shared memory
// (cp.async, zero fill past the row's end) and reads them back itself, so no
// barrier is needed and NORM_DEPTH - 1 steps are in flight without a register.
// 16-bit elements of rows that are not 16-byte aligned, which cp.async cannot
// copy, come one step ahead in registers.
template <class Ty, bool VEC>
constexpr bool norm_async() {
    return VEC || sizeof(typename Ty::T) == 4;
}
template <class Ty, int THREADS, int BLOCK, bool VEC>
struct NormRows {
    using T = typename Ty::T;
    static constexpr int VW = Ty::VW, VECS = NORM_PER / VW;
    static constexpr bool ASYNC = norm_async<Ty, VEC>();
    static constexpr int PIECE = VEC ? 16 : 4, PIECES = VEC ? VECS : NORM_PER;
    static constexpr int PIECE_COLS = VEC ? VW : 1;
    static constexpr uint32_t STEP_BYTES = 2 * NORM_PER * BLOCK * (uint32_t)sizeof(T);
    const T *ptr[2];  // this thread's first element of the next rows to ask for
    int64_t hop[2];   // elements to the step after
    int left[2];      // steps that still have such a row
    int n, t;
    uint32_t ring, fill, read;  // shared addresses: this thread's slots; next to fill, to read
    T ahead[2][ASYNC ? 1 : NORM_PER];

    __device__ __forceinline__ void set(int a, const T *base, int64_t ld, int64_t first,
                                        int64_t step, int64_t m) {
        ptr[a] = base + first * ld + t * PIECE_COLS;
        hop[a] = step * ld;
        left[a] = first < m ? (int)((m - first + step - 1) / step) : 0;
    }
    __device__ __forceinline__ void start(void *smem) {
        ring = smem_u32(smem) + threadIdx.x * PIECE;
        fill = read = ring;
#pragma unroll
        for (int d = 0; d < (ASYNC ? NORM_DEPTH - 1 : 1); ++d) ask();
    }
    __device__ __forceinline__ void advance(uint32_t &at) {
        at = at == ring + (NORM_DEPTH - 1) * STEP_BYTES ? ring : at + STEP_BYTES;
    }
    __device__ __forceinline__ void ask() {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            if (left[a] > 0) {
                --left[a];
                if constexpr (ASYNC) {
#pragma unroll
                    for (int v = 0; v < PIECES; ++v) {
                        const int over = n - (v * THREADS + t) * PIECE_COLS;  // columns left here
                        const uint32_t dst = fill + (a * PIECES + v) * BLOCK * PIECE;
                        const T *src = ptr[a] + (over > 0 ? v * THREADS * PIECE_COLS : -t * PIECE_COLS);
                        if constexpr (VEC)
                            cp_async_16(dst, src, over >= VW ? 16u : over > 0 ? over * (uint32_t)sizeof(T) : 0u);
                        else
                            cp_async_4(dst, src, over > 0 ? 4u : 0u);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < NORM_PER; ++i)
                        ahead[a][i] = i * THREADS + t < n ? __ldcs(ptr[a] + i * THREADS) : (T)0;
                }
                ptr[a] += hop[a];
            }
        }
        if constexpr (ASYNC) {
            cp_async_commit();
            advance(fill);
        }
    }
    // The values of the next step, as pairs, with the step after the last one
    // asked for set off.  (A row past the last leaves stale values: the caller
    // drops them.)
    __device__ __forceinline__ void take(F2 (&y)[2][NORM_PER / 2]) {
        if constexpr (ASYNC) {
            cp_async_wait<NORM_DEPTH - 2>();
#pragma unroll
            for (int a = 0; a < 2; ++a) {
#pragma unroll
                for (int v = 0; v < PIECES; ++v) {
                    const uint32_t src = read + (a * PIECES + v) * BLOCK * PIECE;
                    if constexpr (VEC) {
                        uint4 w;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                                     : "r"(src)
                                     : "memory");
                        float e[VW];
                        row_unpack<Ty>(w, e);
#pragma unroll
                        for (int i = 0; i < VW / 2; ++i) y[a][v * VW / 2 + i] = f2(e[2 * i], e[2 * i + 1]);
                    } else if (v % 2 == 0) {
                        float e0, e1;
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(e0) : "r"(src) : "memory");
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(e1) : "r"(src + BLOCK * PIECE) : "memory");
                        y[a][v / 2] = f2(e0, e1);
                    }
                }
            }
            advance(read);
        } else {
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int i = 0; i < NORM_PER / 2; ++i)
                    y[a][i] = f2(Ty::up(ahead[a][2 * i]), Ty::up(ahead[a][2 * i + 1]));
        }
        ask();
    }
};

template <int LANES>
__device__ __forceinline__ float2 lanes_sum2(float2 v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    return v;
}

// Sum of two values over a group of TR threads, times the cluster's CS blocks.
// `turn` alternates between two buffers, so one barrier per call suffices: a
// buffer is written again two calls later, after every reader has passed the
// barrier in between.
template <int TR, int BLOCK, int CS>
struct GroupSum {
    float2 *warps;   // [2][32]
    float2 *blocks;  // [2][8]
    int turn;
    __device__ __forceinline__ float2 operator()(float2 v) {
        v = lanes_sum2<32>(v);
        if constexpr (TR > 32) {
            constexpr int WARPS = TR / 32;
            const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
            if (lane == 0) warps[turn * 32 + w] = v;
            if constexpr (TR < BLOCK) named_bar_sync(1 + threadIdx.x / TR, TR);
            else __syncthreads();
            v = lanes_sum2<WARPS>(warps[turn * 32 + w / WARPS * WARPS + lane % WARPS]);
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

// Threads of a block: forward 256 or a row's group, backward 512 (its groups'
// column sums meet in shared memory).
template <int TR>
constexpr int norm_block() {
    return TR < 256 ? 256 : TR;
}

template <class Ty, int TR, int CS, bool VEC>
__global__ void __launch_bounds__(norm_block<TR>(), NORM_SM / norm_block<TR>())
    tg_norm_kernel(const NormParams p) {
    using T = typename Ty::T;
    extern __shared__ uint4 ring[];
    __shared__ float2 warps[2 * 32];
    __shared__ float2 blocks[2 * 8];
    constexpr int BLOCK = norm_block<TR>(), GROUPS = BLOCK / TR;
    constexpr int THREADS = TR * CS;  // threads that share a row
    using Cols = NormCols<Ty, THREADS, VEC>;
    const int t = (int)(threadIdx.x % TR) + (CS > 1 ? (int)cluster_ctarank() * TR : 0);
    const int64_t group = ((int64_t)blockIdx.x / CS) * GROUPS + threadIdx.x / TR;
    const int64_t groups = ((int64_t)gridDim.x / CS) * GROUPS;
    const int n = (int)p.n;
    GroupSum<TR, BLOCK, CS> sum{warps, blocks, 0};
    griddep_launch();
    if constexpr (CS > 1) cluster_sync_all();  // every block runs before its memory is written
    griddep_wait();
    NormRows<Ty, THREADS, BLOCK, VEC> rows;
    rows.n = n;
    rows.t = t;
#pragma unroll
    for (int k = 0; k < NORM_ROWS; ++k)
        rows.set(k, static_cast<const T *>(p.x), p.ldx, group + k * groups, NORM_ROWS * groups, p.m);
    rows.start(ring);
    // The group's columns never change: gamma and beta stay in registers.
    F2 gam[NORM_PER / 2], bet[NORM_PER / 2];
#pragma unroll
    for (int i = 0; i < NORM_PER / 2; ++i) {
        const int c = Cols::at(2 * i, t), d = Cols::at(2 * i + 1, t);
        gam[i] = f2(p.gamma && c < n ? p.gamma[c] : 1.0f, p.gamma && d < n ? p.gamma[d] : 1.0f);
        bet[i] = f2(p.beta && c < n ? p.beta[c] : 0.0f, p.beta && d < n ? p.beta[d] : 0.0f);
    }
    T *y = static_cast<T *>(p.y);
    const bool whole = n == THREADS * NORM_PER;
    for (int64_t r = group; r < p.m; r += NORM_ROWS * groups) {
        F2 v[NORM_ROWS][NORM_PER / 2];
        rows.take(v);
        float s[NORM_ROWS];
#pragma unroll
        for (int k = 0; k < NORM_ROWS; ++k) {
            F2 a = v[k][0];
#pragma unroll
            for (int i = 1; i < NORM_PER / 2; ++i) a = add2(a, v[k][i]);
            s[k] = sum2(a);
        }
        const float2 total = sum(make_float2(s[0], s[1]));
        const float mean[NORM_ROWS] = {total.x * p.inv_n, total.y * p.inv_n};
#pragma unroll
        for (int k = 0; k < NORM_ROWS; ++k) {
            const F2 minus = f2(-mean[k]);
#pragma unroll
            for (int i = 0; i < NORM_PER / 2; ++i) v[k][i] = add2(v[k][i], minus);
            if (!whole) {
#pragma unroll
                for (int i = 0; i < NORM_PER / 2; ++i) {
                    float a, b;
                    f2_split(v[k][i], a, b);
                    v[k][i] = f2(Cols::at(2 * i, t) < n ? a : 0.0f, Cols::at(2 * i + 1, t) < n ? b : 0.0f);
                }
            }
            F2 q = mul2(v[k][0], v[k][0]);
#pragma unroll
            for (int i = 1; i < NORM_PER / 2; ++i) q = fma2(v[k][i], v[k][i], q);
            s[k] = sum2(q);
        }
        const float2 second = sum(make_float2(s[0], s[1]));
        const float rstd[NORM_ROWS] = {1.0f / sqrtf(second.x * p.inv_n + p.eps),
                                       1.0f / sqrtf(second.y * p.inv_n + p.eps)};
#pragma unroll
        for (int k = 0; k < NORM_ROWS; ++k) {
            const int64_t rr = r + k * groups;
            if (rr >= p.m) break;
            if (t == 0) {
                if (p.mean) p.mean[rr] = mean[k];
                if (p.rstd) p.rstd[rr] = rstd[k];
            }
            const F2 scale = f2(rstd[k]);
#pragma unroll
            for (int i = 0; i < NORM_PER / 2; ++i) v[k][i] = fma2(mul2(v[k][i], scale), gam[i], bet[i]);
            Cols::store(y + rr * p.ldy, t, n, whole, v[k]);
        }
    }
}

template <class Ty, int TR, int CS, bool VEC>
__global__ void __launch_bounds__(NORM_SM, 1) tg_norm_backward_kernel(const NormParams p) {
    using T = typename Ty::T;
    extern __shared__ uint4 ring[];
    __shared__ float2 warps[2 * 32];
    __shared__ float2 blocks[2 * 8];
    constexpr int BLOCK = NORM_SM, GROUPS = BLOCK / TR;
    constexpr int THREADS = TR * CS;
    using Cols = NormCols<Ty, THREADS, VEC>;
    const int t = (int)(threadIdx.x % TR) + (CS > 1 ? (int)cluster_ctarank() * TR : 0);
    const int64_t group = ((int64_t)blockIdx.x / CS) * GROUPS + threadIdx.x / TR;
    const int64_t groups = ((int64_t)gridDim.x / CS) * GROUPS;
    const int n = (int)p.n;
    GroupSum<TR, BLOCK, CS> sum{warps, blocks, 0};
    griddep_launch();
    if constexpr (CS > 1) cluster_sync_all();
    griddep_wait();
    NormRows<Ty, THREADS, BLOCK, VEC> rows;
    rows.n = n;
    rows.t = t;
    rows.set(0, static_cast<const T *>(p.x), p.ldx, group, groups, p.m);
    rows.set(1, static_cast<const T *>(p.dy), p.lddy, group, groups, p.m);
    rows.start(ring);
    T *dx = static_cast<T *>(p.y);
    F2 gam[NORM_PER / 2], sg[NORM_PER / 2], sb[NORM_PER / 2];
#pragma unroll
    for (int i = 0; i < NORM_PER / 2; ++i) {
        const int c = Cols::at(2 * i, t), d = Cols::at(2 * i + 1, t);
        gam[i] = f2(p.gamma && c < n ? p.gamma[c] : 1.0f, p.gamma && d < n ? p.gamma[d] : 1.0f);
        sg[i] = sb[i] = f2(0.0f);
    }
    const bool whole = n == THREADS * NORM_PER;
    float nmean = group < p.m ? p.mean_in[group] : 0.0f;
    float nrstd = group < p.m ? p.rstd_in[group] : 0.0f;
    for (int64_t r = group; r < p.m; r += groups) {
        F2 w[2][NORM_PER / 2];
        rows.take(w);
        F2(&xh)[NORM_PER / 2] = w[0];
        F2(&d)[NORM_PER / 2] = w[1];
        const F2 minus = f2(-nmean), scale = f2(nrstd);
        const float rstd = nrstd;
        if (r + groups < p.m) {
            nmean = p.mean_in[r + groups];
            nrstd = p.rstd_in[r + groups];
        }
        F2 s1 = f2(0.0f), s2 = f2(0.0f);
#pragma unroll
        for (int i = 0; i < NORM_PER / 2; ++i) {
            // Columns past the row's end hold dy = 0 and add nothing.
            xh[i] = mul2(add2(xh[i], minus), scale);
            sg[i] = fma2(d[i], xh[i], sg[i]);
            sb[i] = add2(sb[i], d[i]);
            d[i] = mul2(d[i], gam[i]);
            s1 = add2(s1, d[i]);
            s2 = fma2(d[i], xh[i], s2);
        }
        const float2 s = sum(make_float2(sum2(s1), sum2(s2)));
        if (dx) {
            // rstd (d - c1 - xh c2)
            const F2 k1 = f2(-rstd * s.x * p.inv_n), k2 = f2(-rstd * s.y * p.inv_n);
#pragma unroll
            for (int i = 0; i < NORM_PER / 2; ++i) d[i] = fma2(d[i], scale, fma2(xh[i], k2, k1));
            Cols::store(dx + r * p.ldy, t, n, whole, d);
        }
    }
    // The groups' column sums meet in shared memory, group by group (the ring
    // is done with: every thread has waited for its own copies).
    const int64_t part = blockIdx.x / CS;
    float eg[NORM_PER], eb[NORM_PER];
#pragma unroll
    for (int i = 0; i < NORM_PER / 2; ++i) {
        f2_split(sg[i], eg[2 * i], eg[2 * i + 1]);
        f2_split(sb[i], eb[2 * i], eb[2 * i + 1]);
    }
    if constexpr (GROUPS > 1) {
        float *acc = reinterpret_cast<float *>(ring) + threadIdx.x % TR;  // [2][NORM_PER][TR]
        if constexpr (norm_async<Ty, VEC>()) cp_async_wait<0>();
        for (int g = 0; g < GROUPS; ++g) {
            __syncthreads();
            if ((int)threadIdx.x / TR == g) {
#pragma unroll
                for (int i = 0; i < NORM_PER; ++i) {
                    float *a = acc + i * TR, *b = a + TR * NORM_PER;
                    if (g) {
                        eg[i] = *a + eg[i];
                        eb[i] = *b + eb[i];
                    }
                    *a = eg[i];
                    *b = eb[i];
                }
            }
        }
        if ((int)threadIdx.x / TR != GROUPS - 1) return;  // the last group holds the totals
    }
#pragma unroll
    for (int i = 0; i < NORM_PER; ++i) {
        const int c = Cols::at(i, t);
        if (c < n) {
            if (p.pgamma) p.pgamma[part * p.n + c] = eg[i];
            if (p.pbeta) p.pbeta[part * p.n + c] = eb[i];
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
    for (int tr : {32, 64, 128, 256, 512})
        if (n <= tr * NORM_PER) return {tr, 1};
    for (int cs : {2, 4})
        if (n <= cs * 512 * NORM_PER) return {512, cs};
    return {512, 8};
}

// Clusters of the launch: NORM_SM threads a SM, no more row slots than rows.
int64_t norm_clusters(const NormShape &s, int64_t m, int sms, int block, int rows) {
    const int64_t per = (int64_t)rows * (block / s.tr);  // rows of a cluster's step
    int64_t c = (m + per - 1) / per;
    const int64_t cap = (int64_t)sms * (NORM_SM / block) / s.cs;
    if (c > cap) c = cap;
    return c < 1 ? 1 : c;
}
// Rows of partial column sums that the backward pass leaves.
int64_t backward_parts(int64_t m, int64_t n, int sms) {
    return norm_clusters(norm_shape(n), m, sms, NORM_SM, 1);
}

template <class Ty, int TR, int CS, bool VEC>
cudaError_t launch_shape(const NormParams &p, bool backward, int64_t grid, int device,
                         cudaStream_t stream) {
    constexpr int STEP = 2 * NORM_PER * (int)sizeof(typename Ty::T);  // ring bytes a thread and step
    constexpr bool ASYNC = norm_async<Ty, VEC>();
    constexpr int SMEM = ASYNC ? NORM_DEPTH * STEP * norm_block<TR>() : 0;
    // (without a ring: the groups' column sums)
    constexpr int SMEM_BACK = ASYNC ? NORM_DEPTH * STEP * NORM_SM : 2 * 4 * TR * NORM_PER;
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << device;
    if (!(done.load(std::memory_order_acquire) & bit)) {
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
    cfg.blockDim = dim3(backward ? NORM_SM : norm_block<TR>(), 1, 1);
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
    if (s.tr == 64) return launch_shape<Ty, 64, 1, VEC>(p, backward, grid, device, stream);
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
    const int block = s.tr < 256 ? 256 : s.tr;
    const int64_t grid = s.cs * norm_clusters(s, M, dev.sms, block, NORM_ROWS);
    const bool vec = vec_ok(X, ldx, e) && vec_ok(Y, ldy, e);
    return launch_norm(p, dtype, false, vec, grid, dev.id, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? TG_OK
               : TG_ERR_CUDA;
}

extern "C" int64_t tg_layer_norm_backward_workspace_bytes(int64_t M, int64_t N) {
    if (M < 0 || N < 0 || M > INT32_MAX || N > kNormMaxCols) return -1;
    tg::host::Device dev;
    if (tg::host::device(&dev) != TG_OK) return -1;
    return M == 0 || N == 0 ? 0 : 2 * 4 * N * backward_parts(M, N, dev.sms);
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
    int64_t parts = 0;
    if (M > 0) {
        parts = backward_parts(M, N, dev.sms);
        if (sums && (!workspace || (uintptr_t)workspace % 4 || workspace_bytes < 2 * 4 * N * parts))
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
        if (dbeta) p.pbeta = static_cast<float *>(workspace) + parts * N;
        const NormShape s = norm_shape(N);
        const bool vec = vec_ok(X, ldx, e) && vec_ok(dY, lddy, e) && (!dX || vec_ok(dX, lddx, e));
        if (launch_norm(p, dtype, true, vec, parts * s.cs, dev.id, stream) != cudaSuccess)
            return TG_ERR_CUDA;
    }
    if (!sums) return TG_OK;
    // M == 0: no parts, the sums are zero.
    const float *w = static_cast<const float *>(workspace);
    return tg::host::colsum_finish(dgamma ? w : w + parts * N, dgamma && dbeta ? w + parts * N : nullptr,
                                   (int32_t)parts, N, dgamma ? dgamma : dbeta,
                                   dgamma && dbeta ? dbeta : nullptr, stream) == cudaSuccess
               ? TG_OK
               : TG_ERR_CUDA;
}
