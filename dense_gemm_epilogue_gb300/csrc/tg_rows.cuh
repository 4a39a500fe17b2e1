// Row-wise helpers of the feed-forward operators: 16-byte vectors of typed
// elements, and the fixed-order reduction of per-block column sums.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "tg_ptx.cuh"

namespace tg {

struct TypeF32 {
    using T = float;
    static constexpr int VW = 4;  // elements per 16 bytes
    __device__ static float up(T x) { return x; }
    __device__ static T down(float x) { return x; }
    __device__ static uint32_t down2(float, float) { return 0; }  // 16-bit types only
};
struct TypeBF16 {
    using T = unsigned short;
    static constexpr int VW = 8;
    __device__ static float up(T x) { return __uint_as_float((uint32_t)x << 16); }
    __device__ static float up_high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
    __device__ static T down(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
    __device__ static uint32_t down2(float lo, float hi) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};
struct TypeF16 {
    using T = unsigned short;
    static constexpr int VW = 8;
    __device__ static float up(T x) { return __half2float(__ushort_as_half(x)); }
    __device__ static float up_high(uint32_t w) { return up((T)(w >> 16)); }
    __device__ static T down(float x) { return __half_as_ushort(__float2half_rn(x)); }
    __device__ static uint32_t down2(float lo, float hi) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};

template <class Ty>
__device__ __forceinline__ void row_unpack(const uint4 &v, float *y) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (Ty::VW == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = Ty::up((unsigned short)(w[i] & 0xffffu));
            y[2 * i + 1] = Ty::up_high(w[i]);
        }
    }
}

template <class Ty>
__device__ __forceinline__ void row_store_vec(typename Ty::T *q, const float *y) {
    uint4 v;
    if constexpr (Ty::VW == 4) {
        v = make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                       __float_as_uint(y[3]));
    } else {
        v = make_uint4(Ty::down2(y[0], y[1]), Ty::down2(y[2], y[3]), Ty::down2(y[4], y[5]),
                       Ty::down2(y[6], y[7]));
    }
    *reinterpret_cast<uint4 *>(q) = v;
}

template <class Ty>
__device__ __forceinline__ void row_store(typename Ty::T *row, int64_t c, int64_t n, const float *y) {
    if (c + Ty::VW <= n) {
        row_store_vec<Ty>(row + c, y);
    } else {
#pragma unroll
        for (int i = 0; i < Ty::VW; ++i)
            if (c + i < n) row[c + i] = Ty::down(y[i]);
    }
}

// out[c] = sum over `parts` rows of partial[q][c], q ascending within each of
// the block's row lanes, then the lanes in order: a fixed order, so repeated
// calls agree bit for bit.  Up to two arrays per launch (blockIdx.y).
constexpr int FINISH_COLS = 32, FINISH_ROWS = 16;
static __global__ void __launch_bounds__(FINISH_COLS *FINISH_ROWS)
    tg_colsum_finish_kernel(const float *partial0, const float *partial1, int32_t parts, int64_t n,
                            float *out0, float *out1) {
    __shared__ float sums[FINISH_ROWS][FINISH_COLS];
    griddep_launch();
    griddep_wait();
    const float *partial = blockIdx.y ? partial1 : partial0;
    float *out = blockIdx.y ? out1 : out0;
    const int64_t c = (int64_t)blockIdx.x * FINISH_COLS + threadIdx.x;
    float s = 0.0f;
    if (c < n) {
        int32_t q = threadIdx.y;
        // Eight loads in flight per thread.
        for (; q + 7 * FINISH_ROWS < parts; q += 8 * FINISH_ROWS) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = partial[(int64_t)(q + i * FINISH_ROWS) * n + c];
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[i];
        }
        for (; q < parts; q += FINISH_ROWS) s += partial[(int64_t)q * n + c];
    }
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < n) {
#pragma unroll
        for (int i = 1; i < FINISH_ROWS; ++i) s += sums[i][threadIdx.x];
        out[c] = s;
    }
}

}  // namespace tg
