// Rotary positions: pairs (a, b) of each head's first `rot` values turned by
// position x frequency,
//   a' = amplitude (a cos p - b sin p),  b' = amplitude (a sin p + b cos p),
// and the transposed map for the gradients (sin negated).
//
// The angle is exact at any position: a frequency is held as a fraction of a turn
// in 64 bits, so the product with the position wraps at whole turns by itself,
// and what is left is taken to an eighth of a turn before it becomes FP32 (an
// angle formed in FP32 would be off by 0.03 radians at position 10^6).
//
// Bound: memory; each value is read and written once.  A block takes a run of
// (token, head) rows, computes the angles' sines and cosines of the few tokens
// it touches once, in shared memory, and its threads then each hold eight pairs
// of one place in the head, two rows apart at a time, loads before the table and before
// the stores.  (8192 x 40 heads of 128: 29.7 us, 5.7 TB/s; four rows a thread and four
// blocks an SM, 4.2 waves, 32.9; one row and eight blocks 33.5.  Six blocks an SM hold the
// kernel to 40 registers: vectors of halves spill 24 bytes, 16 in FP32.)
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "../../include/tg_gemm.h"
#include "tg_host.h"
#include "tg_rows.cuh"

namespace tg {

constexpr int ROT_THREADS = 256;
constexpr int ROT_UNROLL = 2;
constexpr int ROT_TABLE_BYTES = 40960;  // sines and cosines of a block

struct RotaryParams {
    int64_t rows;  // tokens x heads
    int32_t heads, dim, rot;
    const void *x;
    int64_t ldx, hx;
    void *y;
    int64_t ldy, hy, y_rows;
    const int64_t *positions, *to;
    const uint64_t *steps;
    float amplitude;
    int32_t transpose;
    int32_t copy;      // 1: values past rot are copied (0: y is x)
    int32_t per;       // items of a row
    int32_t turning;   // items of a row that turn pairs
    int32_t lanes;     // threads side by side on a row: min(per, ROT_THREADS)
    int32_t block_rows;
};

// cos and sin of `phase` / 2^64 turns, to FP32.
__device__ __forceinline__ float2 turn_cos_sin(uint64_t phase) {
    const uint32_t t = (uint32_t)(phase >> 32);
    const uint32_t q = (t + 0x20000000u) >> 30;  // nearest quarter
    float s, c;
    sincospif((float)(int32_t)(t - (q << 30)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
    const float a = q & 1 ? s : c, b = q & 1 ? c : s;
    return make_float2(q == 1 || q == 2 ? -a : a, q >= 2 ? -b : b);
}

// An item: VW pairs in halves (two vectors) or VW / 2 pairs side by side (one
// vector); single elements' rows: one pair.  Past the turning ones, a vector (or
// element) that is copied.  In the table a token's items lie side by side, two pairs'
// cos and sin (16 bytes) at a time, so that neighbouring threads read neighbouring
// words (a pair after the other: four-way bank conflicts).
template <class Ty, bool HALVES, bool VEC>
__global__ void __launch_bounds__(ROT_THREADS, 6) tg_rotary_kernel(const RotaryParams p) {
    using T = typename Ty::T;
    constexpr int VW = VEC ? Ty::VW : 1;
    constexpr int PAIRS = !VEC ? 1 : HALVES ? VW : VW / 2;  // pairs of an item
    constexpr int CHUNK = PAIRS > 1 ? 2 : 1;                // pairs side by side in the table
    extern __shared__ __align__(16) float2 table[];
    griddep_launch();
    griddep_wait();
    const int64_t r0 = (int64_t)blockIdx.x * p.block_rows;
    const int rows = (int)(p.rows - r0 < p.block_rows ? p.rows - r0 : p.block_rows);
    const int64_t t0 = r0 / p.heads;
    const int h0 = (int)(r0 - t0 * p.heads);
    const int half = p.rot / 2;
    const int lane = threadIdx.x % p.lanes, slot = threadIdx.x / p.lanes;
    const int slots = ROT_THREADS / p.lanes;
    const T *x = static_cast<const T *>(p.x) + t0 * p.ldx;
    T *y = static_cast<T *>(p.y);
    const bool in = slot < slots;
    bool ready = false;  // the table
    for (int v = lane; v < p.per || !ready; v += p.lanes) {
        const bool turn = v < p.turning;
        const bool work = in && v < p.per && (turn || p.copy);
        // Offsets of the item's two parts within a head (a copied one: the first).
        const int d = turn ? (HALVES || VEC ? v * VW : 2 * v) : p.rot + (v - p.turning) * VW;
        const int d2 = HALVES ? d + half : d + 1;
        for (int i0 = slot; i0 < rows || !ready; i0 += ROT_UNROLL * slots) {
            uint4 a[ROT_UNROLL], b[ROT_UNROLL];
            T sa[ROT_UNROLL], sb[ROT_UNROLL];
            int64_t to[ROT_UNROLL];
            int tok[ROT_UNROLL];
#pragma unroll
            for (int u = 0; u < ROT_UNROLL; ++u) {
                const int i = i0 + u * slots;
                to[u] = -1;
                tok[u] = 0;
                if (!work || i >= rows) continue;
                const int t = (h0 + i) / p.heads, h = h0 + i - t * p.heads;
                tok[u] = t;
                const int64_t row = p.to ? p.to[t0 + t] : t0 + t;
                if (p.to && (row < 0 || row >= p.y_rows)) continue;
                to[u] = row * p.ldy + h * p.hy;
                const T *src = x + t * p.ldx + h * p.hx;
                if constexpr (VEC) {
                    a[u] = *reinterpret_cast<const uint4 *>(src + d);
                    if (HALVES && turn) b[u] = *reinterpret_cast<const uint4 *>(src + d2);
                } else {
                    sa[u] = src[d];
                    if (turn) sb[u] = src[d2];
                }
            }
            if (!ready) {
                // (while the first values are on their way)
                const int n = ((h0 + rows - 1) / p.heads + 1) * half;
                for (int i = threadIdx.x; i < n; i += ROT_THREADS) {
                    const int t = i / half, f = i - t * half;
                    const int64_t pos = p.positions ? p.positions[t0 + t] : t0 + t;
                    float2 cs = turn_cos_sin((uint64_t)pos * p.steps[f]);
                    cs.x *= p.amplitude;
                    cs.y *= p.transpose ? -p.amplitude : p.amplitude;
                    const int item = f / PAIRS, q = f % PAIRS;
                    table[t * half + (q / CHUNK * p.turning + item) * CHUNK + q % CHUNK] = cs;
                }
                __syncthreads();
                ready = true;
            }
#pragma unroll
            for (int u = 0; u < ROT_UNROLL; ++u) {
                if (to[u] < 0) continue;
                T *dst = y + to[u];
                if (!turn) {
                    if constexpr (VEC) *reinterpret_cast<uint4 *>(dst + d) = a[u];
                    else dst[d] = sa[u];
                    continue;
                }
                const float2 *row = table + tok[u] * half + v * CHUNK;
                if constexpr (!VEC) {
                    const float fa = Ty::up(sa[u]), fb = Ty::up(sb[u]);
                    const float2 cs = row[0];
                    dst[d] = Ty::down(fa * cs.x - fb * cs.y);
                    dst[d2] = Ty::down(fa * cs.y + fb * cs.x);
                } else {
                    float fa[VW], fb[VW];
                    row_unpack<Ty>(a[u], fa);
                    if constexpr (HALVES) row_unpack<Ty>(b[u], fb);
#pragma unroll
                    for (int q = 0; q < PAIRS; q += 2) {
                        const float4 cs = *reinterpret_cast<const float4 *>(row + q / 2 * p.turning * CHUNK);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float c = e ? cs.z : cs.x, s = e ? cs.w : cs.y;
                            float &va = HALVES ? fa[q + e] : fa[(2 * (q + e)) % VW];
                            float &vb = HALVES ? fb[q + e] : fa[(2 * (q + e) + 1) % VW];
                            const float ya = va * c - vb * s;
                            vb = va * s + vb * c;
                            va = ya;
                        }
                    }
                    row_store_vec<Ty>(dst + d, fa);
                    if constexpr (HALVES) row_store_vec<Ty>(dst + d2, fb);
                }
            }
            if (i0 + ROT_UNROLL * slots >= rows) break;
        }
        if (v + p.lanes >= p.per) break;
    }
}

}  // namespace tg

namespace {

using namespace tg;

constexpr int64_t kMaxDim = 4096;
constexpr double kTwoPi = 6.283185307179586;

bool type_ok(tg_out_dtype t) { return t == TG_OUT_F32 || t == TG_OUT_BF16 || t == TG_OUT_F16; }

template <class Ty>
cudaError_t launch_type(RotaryParams p, bool halves, bool aligned, int sms, cudaStream_t stream) {
    const int vw = Ty::VW;
    const bool vec = aligned && p.dim % vw == 0 && (halves ? p.rot % (2 * vw) == 0 : p.rot % vw == 0);
    p.turning = vec ? p.rot / (halves ? 2 * vw : vw) : p.rot / 2;
    p.per = p.turning + (p.copy ? (p.dim - p.rot) / (vec ? vw : 1) : 0);
    if (p.per == 0) return cudaSuccess;
    p.lanes = p.per < ROT_THREADS ? p.per : ROT_THREADS;
    // ROT_UNROLL rows a thread where that still leaves two blocks an SM; no more tokens
    // than the table holds (a run of n rows touches up to (n - 1) / heads + 2).
    const int64_t slots = ROT_THREADS / p.lanes;
    int64_t n = p.rows >= 2 * sms * ROT_UNROLL * slots ? ROT_UNROLL * slots : slots;
    const int64_t token_bytes = 4 * (int64_t)p.rot;
    if (token_bytes) {
        const int64_t most = (ROT_TABLE_BYTES / token_bytes - 2) * p.heads + 1;
        if (n > most) n = most;
    }
    p.block_rows = (int32_t)n;
    const int64_t grid = (p.rows + n - 1) / n;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    const int64_t tokens = (n - 1) / p.heads + 2;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(ROT_THREADS, 1, 1);
    cfg.dynamicSmemBytes = (size_t)(tokens * token_bytes);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (vec)
        return halves ? cudaLaunchKernelEx(&cfg, tg_rotary_kernel<Ty, true, true>, p)
                      : cudaLaunchKernelEx(&cfg, tg_rotary_kernel<Ty, false, true>, p);
    return halves ? cudaLaunchKernelEx(&cfg, tg_rotary_kernel<Ty, true, false>, p)
                  : cudaLaunchKernelEx(&cfg, tg_rotary_kernel<Ty, false, false>, p);
}

tg_status rotary(int64_t tokens, int64_t heads, int64_t dim, int64_t rot, const void *X, int64_t ldx,
                 int64_t hx, void *Y, int64_t ldy, int64_t hy, int64_t y_rows, const int64_t *positions,
                 const int64_t *rows, const uint64_t *steps, tg_rotary_layout layout, float amplitude,
                 tg_out_dtype dtype, bool transpose, void *stream) {
    if (tokens < 0 || heads < 0 || dim < 0 || rot < 0 || rot > dim || rot % 2 || !type_ok(dtype))
        return TG_ERR_INVALID_VALUE;
    if (tokens > INT32_MAX || heads > 65536) return TG_ERR_INVALID_VALUE;
    if (layout != TG_ROTARY_HALVES && layout != TG_ROTARY_PAIRS) return TG_ERR_INVALID_VALUE;
    if (!std::isfinite(amplitude) || (rows && y_rows < 0)) return TG_ERR_INVALID_VALUE;
    if (dim > kMaxDim) return TG_ERR_UNSUPPORTED;
    if (tokens == 0 || heads == 0 || dim == 0) return TG_OK;
    const int e = dtype == TG_OUT_F32 ? 4 : 2;
    if (!X || !Y || (uintptr_t)X % e || (uintptr_t)Y % e || ldx < dim || ldy < dim ||
        (heads > 1 && (hx < dim || hy < dim)))
        return TG_ERR_INVALID_VALUE;
    if (ldx >= (int64_t)1 << 38 || ldy >= (int64_t)1 << 38 ||
        (heads > 1 && (hx >= (int64_t)1 << 38 || hy >= (int64_t)1 << 38)))
        return TG_ERR_INVALID_VALUE;
    // In place: value for value.
    if (X == Y && !rows && ((tokens > 1 && ldx != ldy) || (heads > 1 && hx != hy))) return TG_ERR_INVALID_VALUE;
    // Y's rows and heads may not run into each other.
    const int64_t out_rows = rows ? y_rows : tokens;
    if (heads > 1 && out_rows > 1 && ldy < (heads - 1) * hy + dim && (double)hy < (double)(out_rows - 1) * ldy + dim)
        return TG_ERR_INVALID_VALUE;
    if (((uintptr_t)positions | (uintptr_t)rows | (uintptr_t)steps) % 8 || (rot > 0 && !steps))
        return TG_ERR_INVALID_VALUE;
    if (heads == 1) hx = hy = 0;
    tg::host::Device dev;
    const tg_status st = tg::host::device(&dev);
    if (st != TG_OK) return st;
    RotaryParams p = {};
    p.rows = tokens * heads;
    p.heads = (int32_t)heads;
    p.dim = (int32_t)dim;
    p.rot = (int32_t)rot;
    p.x = X;
    p.ldx = ldx;
    p.hx = hx;
    p.y = Y;
    p.ldy = ldy;
    p.hy = hy;
    p.y_rows = y_rows;
    p.positions = positions;
    p.to = rows;
    p.steps = steps;
    p.amplitude = amplitude;
    p.transpose = transpose;
    p.copy = X != Y || rows != nullptr;
    const bool aligned = !(((uintptr_t)X | (uintptr_t)Y) % 16) && !((ldx | ldy | hx | hy) * e % 16);
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool halves = layout == TG_ROTARY_HALVES;
    const cudaError_t err = dtype == TG_OUT_F32    ? launch_type<TypeF32>(p, halves, aligned, dev.sms, cs)
                            : dtype == TG_OUT_BF16 ? launch_type<TypeBF16>(p, halves, aligned, dev.sms, cs)
                                                   : launch_type<TypeF16>(p, halves, aligned, dev.sms, cs);
    return err == cudaSuccess ? TG_OK : TG_ERR_CUDA;
}

}  // namespace

extern "C" tg_status tg_rotary_steps(int64_t rot, double base, tg_rotary_scaling scaling, double factor,
                                     double low, double high, double original, uint64_t *steps) {
    if (rot <= 0 || rot % 2 || rot > kMaxDim || !steps) return TG_ERR_INVALID_VALUE;
    if (!(base > 0.0) || !std::isfinite(base) || !(factor > 0.0) || !std::isfinite(factor))
        return TG_ERR_INVALID_VALUE;
    if (scaling < TG_ROTARY_NONE || scaling > TG_ROTARY_BANDS) return TG_ERR_INVALID_VALUE;
    if (scaling == TG_ROTARY_BASE && rot < 4) return TG_ERR_INVALID_VALUE;
    if (scaling == TG_ROTARY_BANDS &&
        (!(low < high) || !std::isfinite(low) || !std::isfinite(high) || !(original > 0.0) ||
         !std::isfinite(original)))
        return TG_ERR_INVALID_VALUE;
    if (scaling == TG_ROTARY_BASE) base *= std::pow(factor, (double)rot / (double)(rot - 2));
    // (with an infinite base all pairs but the first would stand still)
    if (!(base > 0.0) || !std::isfinite(base)) return TG_ERR_INVALID_VALUE;
    for (int64_t i = 0; i < rot / 2; ++i) {
        double f = std::pow(base, -(double)(2 * i) / (double)rot);
        if (scaling == TG_ROTARY_LINEAR) f /= factor;
        if (scaling == TG_ROTARY_BANDS) {
            double g = (original * f / kTwoPi - low) / (high - low);
            g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
            f = g * f + (1.0 - g) * f / factor;
        }
        double turns = f / kTwoPi;
        turns -= std::floor(turns);
        if (!(turns >= 0.0)) return TG_ERR_INVALID_VALUE;  // an overflow above
        // To the nearest step: truncated, low frequencies would lose twice as much a position.
        // (The largest double below 1 times 2^64 is a whole number below 2^64.)
        steps[i] = turns >= 1.0 ? 0 : (uint64_t)std::nearbyint(std::ldexp(turns, 64));
    }
    return TG_OK;
}

extern "C" tg_status tg_rotary(int64_t tokens, int64_t heads, int64_t dim, int64_t rot, const void *X,
                               int64_t ldx, int64_t hx, void *Y, int64_t ldy, int64_t hy, int64_t y_rows,
                               const int64_t *positions, const int64_t *rows, const uint64_t *steps,
                               tg_rotary_layout layout, float amplitude, tg_out_dtype dtype,
                               void *stream) {
    return rotary(tokens, heads, dim, rot, X, ldx, hx, Y, ldy, hy, y_rows, positions, rows, steps, layout,
                  amplitude, dtype, false, stream);
}

extern "C" tg_status tg_rotary_backward(int64_t tokens, int64_t heads, int64_t dim, int64_t rot,
                                        const void *dY, int64_t lddy, int64_t hdy, void *dX, int64_t lddx,
                                        int64_t hdx, const int64_t *positions, const uint64_t *steps,
                                        tg_rotary_layout layout, float amplitude, tg_out_dtype dtype,
                                        void *stream) {
    return rotary(tokens, heads, dim, rot, dY, lddy, hdy, dX, lddx, hdx, 0, positions, nullptr, steps,
                  layout, amplitude, dtype, true, stream);
}
