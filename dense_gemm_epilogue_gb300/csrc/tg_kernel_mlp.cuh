// Tile GEMM of the feed-forward operators: row-major outputs, operands
// contiguous along either axis, and epilogues that need more than the
// accumulator.
//
// Role space: out(r, c) = f(sum_k A(r, k) B(c, k)), r < m, c < n, row-major.
// A team of CG CTAs computes 128 CG rows x BN accumulator columns with
// tcgen05.mma.cta_group::CG: a pair on neighbouring SMs (CG = 2, half the B
// bytes per SM), or a single CTA (CG = 1, for products whose 256-row tiles
// would leave SMs idle or rows empty).  The persistent schedule, the barriers
// between a pair, the ticket ring and the bounded waits are those of the
// CTA-pair GEMM (tg_kernel_pair.cuh).  What differs:
//
//   operands  Each of A and B is either K-major (rows of K) or MN-major (rows
//             of the reduction index, the role-space row index contiguous):
//             dX = dZ W reads W by columns, dW = dZ^T X reads both operands
//             by columns.  An MN-major operand lands as 64 x 64 boxes (64
//             reduction rows of 128 bytes, 128-byte swizzle), 8 KB apart
//             along the role-space rows, and the MMA's transpose bits take it
//             from there; nothing is transposed in memory.
//   two pairs The reduction may run over two operand pairs in turn (dX = dG
//             Wg + dU Wu): K blocks from k_blocks0 on come from the second
//             pair of maps, into the same accumulator.
//   dual      The gated unit's forward tile holds BN/2 gate columns and BN/2
//             up columns of the same features: Wg rows and Wu rows are halves
//             of the B stage (a pair's leader stages the one, its peer the
//             other), one MMA serves both, and one thread of the epilogue owns
//             g and u of the same element.
//   entries   A second problem of the same shape in the same launch (dWg and
//             dWu share X): tiles from tiles_per_batch on use the second A map
//             and the second output.
//   epilogue  A thread holds one row's consecutive columns.  Its warp stages 32
//             rows x 64 bytes in shared memory (swizzled, two 2 KB buffers, so
//             that one is filled while the other drains) and stores them by TMA,
//             which clips at the rows' and columns' end.  The residual comes in
//             through the same buffers by TMA, the first box before the
//             accumulator is ready and each next one while the last is in work.
//             Against plain 16-byte stores from a single staged box (calls back
//             to back on the same inputs): 1111 x 8200 x 2056 with GELU and saved
//             Z 41.7 us, 43.7; gated 333 x 5640 x 2048 19.3, 20.1; gated 8192 x
//             14336 x 4096 with G and U 1172, 1187; without an activation no
//             difference.  Rows that are not 16-byte
//             aligned, and boxes that end inside 16 bytes (there a TMA store
//             wrote into the row's padding), go through the same buffers with
//             4-byte stores.
//
// Bound: tensor throughput for token counts above about 300 (arithmetic
// intensity 256 x 256 / (256 + 256) = 128 FLOP per byte of L2 traffic).  8192 x
// 4096 x 14336 with bias and residual: 573 us in a chain of launches, 1.68 PFLOP/s,
// 593 us in a long run at the power limit (1.62; cuBLAS sustains 1.71 there).
#pragma once

#include <cstdint>
#include <type_traits>
#include "tg_kernel_pair.cuh"

namespace tg {

enum MlpAct : int32_t { MLP_NONE = 0, MLP_RELU = 1, MLP_SILU = 2, MLP_GELU = 3, MLP_ACTS = 4 };

// The activations and their derivatives all come from one logistic function,
// sigmoid(v) = 1 / (1 + 2^u), u = -v log2 e, by the hardware's base-2 exponential
// and reciprocal: relative error about 2^-21 for the |v| that matter, far
// below a 16-bit output's 2^-9, and below the 1e-6 that an FP32 column sum over
// it is held to.  The error grows with |u| (u's own rounding), to about 2^-17 at
// the tail's end.
//
// Both instructions flush subnormal results, and 2^u overflows from u = 128 on,
// while y sigmoid(y) stays a normal FP32 and BF16 number down to y = -91.8 (u =
// 132).  So 2^u is the square of h = 2^(u/2), and the denominator carries a factor
// 2^-64, 2^-64 (1 + h^2), whose reciprocal stays normal up to u = 190; the last
// product rounds to a subnormal where the value is one.  Beyond, the limit 0 is
// right to FP32's smallest subnormal.  (Two more multiplications than 1 / (1 +
// 2^u), which flushes: 55.0 us for the column sums of 4096 x 16384 with GELU, 52.5
// without; a select between the two forms, five more instructions, 59.1.)
constexpr float kLog2E = 1.4426950408889634f;
__device__ __forceinline__ float mlp_sigmoid_half(float v) {  // v = u / 2
    constexpr float SCALE = 5.421010862427522e-20f;  // 2^-64
    float h, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(v));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(fmaf(h * SCALE, h, SCALE)));
    return s * SCALE;
}

// The tanh form of GELU is y/2 (1 + tanh(v)) = y sigmoid(2v), v =
// sqrt(2/pi) (y + 0.044715 y^3): no cancellation in 1 + tanh(v) for negative
// v.  y^2 is held to 256 inside the argument (for |y| >= 16 sigmoid is 0 or 1
// to all FP32 digits), which keeps it and the derivative's product finite.
constexpr float kGelu2C = 1.5957691216057308f;  // 2 sqrt(2/pi)
__device__ __forceinline__ float mlp_gelu_sigmoid(float y, float y2) {
    return mlp_sigmoid_half(y * fmaf(-0.5f * kLog2E * kGelu2C * 0.044715f, y2, -0.5f * kLog2E * kGelu2C));
}

template <int ACT>
__device__ __forceinline__ float mlp_act(float y) {
    if constexpr (ACT == MLP_RELU) return (!(y > 0.0f) && !(y != y)) ? 0.0f : y;
    else if constexpr (ACT == MLP_SILU) return y * mlp_sigmoid_half(-0.5f * kLog2E * y);
    else if constexpr (ACT == MLP_GELU) return y * mlp_gelu_sigmoid(y, fminf(y * y, 256.0f));
    else return y;
}

// Activation and its derivative.  ReLU'(0) = 0.
template <int ACT>
__device__ __forceinline__ void mlp_act_grad(float y, float &a, float &d) {
    if constexpr (ACT == MLP_RELU) {
        const bool on = y > 0.0f || y != y;
        a = on ? y : 0.0f;
        d = on ? 1.0f : 0.0f;
    } else if constexpr (ACT == MLP_SILU) {
        const float s = mlp_sigmoid_half(-0.5f * kLog2E * y);
        a = y * s;
        d = fmaf(a, 1.0f - s, s);
    } else if constexpr (ACT == MLP_GELU) {
        const float y2 = fminf(y * y, 256.0f);
        const float s = mlp_gelu_sigmoid(y, y2);
        a = y * s;
        d = fmaf(a * (1.0f - s), fmaf(kGelu2C * 0.134145f, y2, kGelu2C), s);
    } else {
        a = y;
        d = 1.0f;
    }
}

// f(integral constant of the activation) for a runtime one: the branch is
// taken once around a loop, not per element.
template <class F>
__device__ __forceinline__ void mlp_with_act(int act, F f) {
    switch (act) {
    case MLP_RELU: f(std::integral_constant<int, MLP_RELU>{}); return;
    case MLP_SILU: f(std::integral_constant<int, MLP_SILU>{}); return;
    case MLP_GELU: f(std::integral_constant<int, MLP_GELU>{}); return;
    default: f(std::integral_constant<int, MLP_NONE>{}); return;
    }
}

template <Kind KD>
__device__ __forceinline__ float mlp_to_float(uint32_t half_bits) {
    if constexpr (KD == Kind::BF16) return __uint_as_float(half_bits << 16);
    else return __half2float(__ushort_as_half((unsigned short)half_bits));
}
template <Kind KD>
__device__ __forceinline__ uint32_t mlp_pack2(float lo, float hi) {
    if constexpr (KD == Kind::BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

// TMA store of a swizzled shared-memory box; bounds are the map's.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t src, int32_t c0,
                                             int32_t c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(src), "r"(c0), "r"(c1)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the issuing thread's last LEFT stores have read their shared memory;
// all its stores are complete.
template <int LEFT>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(LEFT) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Descriptor of an MN-major operand tile: 64-element rows of 128 bytes along
// the role-space rows, one per reduction index, 128-byte swizzle.  Leading
// byte offset: the next 64 role-space rows (one 64 x 64 box, 8 KB); stride
// byte offset: the next 8 reduction indexes (1 KB).
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(8192u >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// K segments of a split tile, less the finisher's own: at most this many.
constexpr int SPLIT_PARTS = 3;

enum class MlpEpi : int { LINEAR = 0, GATED = 1, PLAIN = 2 };

struct MlpOut {
    void *ptr;       // row-major output (NULL: not wanted)
    int64_t ld;      // elements between rows
    int32_t tma;     // 1: stored by TMA through its map
    int32_t pad_;
};

struct MlpMaps {
    CUtensorMap a[2], b[2], out[3], r;
};

struct MlpParams {
    GemmParams g;             // schedule, split, status (m, n: rows and columns of one output)
    int32_t k_blocks0;        // K blocks of the first operand pair (rest: the second)
    int32_t act;
    const float *bias;        // n values or NULL
    const void *r;            // residual (m x n) or NULL
    int64_t ldr;
    int32_t r_tma;            // 1: loaded by TMA through its map
    int32_t out_f32;          // PLAIN: outputs are FP32 (else the operands' type)
    int32_t clip;             // 1: a row's bytes are a multiple of 16, so TMA may clip a box there
    // 1: this product reads nothing that the kernel before it writes (a weight
    // gradient after the input gradient), so it starts without waiting for that
    // kernel and waits at its end, for whatever comes next on the stream.  Only
    // one of the two may use the stream's workspace.
    int32_t late_wait;
    // What makes the kernels before that one visible to it (NULL: neither side).
    // The input gradient raises the gate (a release) once its own wait has
    // returned, and only then lets its successor start; a thread of each of the
    // weight gradient's CTAs acquires it while the others set the CTA up.  A gate
    // found down, which that order all but rules out (the first CTA takes it down
    // after its wait, when a late one may still be starting), costs the producer
    // the wait itself.
    uint32_t *gate;
    MlpOut out[3];            // LINEAR: Y, Z; GATED: H, G, U; PLAIN: one per entry
};

// AM, BM: 0 = K-major, 1 = MN-major operand.  CG: CTAs per team.
template <Kind KD, int CG, int BN, int AM, int BM, MlpEpi EP>
struct MlpConfig {
    using T = KindTraits<KD>;
    static constexpr int BK = T::block_k;
    static constexpr int TILE_M = CG * BLOCK_M;
    static constexpr int B_ROWS = BN / CG;  // B-role rows staged by each CTA
    static constexpr bool DUAL = EP == MlpEpi::GATED;
    static constexpr int OUT_N = DUAL ? BN / 2 : BN;  // output columns per tile
    static constexpr int A_BYTES = BLOCK_M * ROW_BYTES;
    static constexpr int B_BYTES = B_ROWS * ROW_BYTES;
    static constexpr int EPI_WARPS = 8;
    static constexpr int COLS = OUT_N / 2;            // output columns of an epilogue warp
    static constexpr int STG_ROW = 64;                // a staged row: 32 16-bit columns
    static constexpr int STG_BYTES = 32 * STG_ROW;    // one staging buffer, two per warp
    static constexpr int FIT = (SMEM_LIMIT - 3072 - 2 * EPI_WARPS * STG_BYTES) / (A_BYTES + B_BYTES);
    static constexpr int STAGES = FIT > 8 ? 8 : FIT;
    static constexpr int A_OFF = 0;
    static constexpr int B_OFF = STAGES * A_BYTES;
    static constexpr int STG_OFF = B_OFF + STAGES * B_BYTES;
    static constexpr int BIAS_OFF = STG_OFF + 2 * EPI_WARPS * STG_BYTES;
    static constexpr int BAR_OFF = BIAS_OFF + EPI_WARPS * 128;  // 32 floats per warp
    static constexpr int FULL0 = 0, EMPTY0 = STAGES;
    static constexpr int ACCF0 = 2 * STAGES, ACCE0 = ACCF0 + 2, DRAIN = ACCE0 + 2;
    static constexpr int SLOTS = 4;
    static constexpr int TKF0 = DRAIN + 1, TKE0 = TKF0 + SLOTS;
    static constexpr int RES0 = TKE0 + SLOTS;  // two per epilogue warp: residual box landed
    static constexpr int NUM_BARS = RES0 + 2 * EPI_WARPS;
    static constexpr int MISC_OFF = BAR_OFF + NUM_BARS * 8;
    static constexpr int TK_OFF = (MISC_OFF + 16 + 15) / 16 * 16;
    static constexpr int TICKET_OFF = TK_OFF + 16 * SLOTS;
    static constexpr int SMEM_BYTES = TICKET_OFF + 16 * SLOTS + 1024;
    static constexpr int TMEM_COLS = 2 * BN;
    static constexpr int NUM_WARPS = 2 + EPI_WARPS;
    static constexpr int NUM_THREADS = NUM_WARPS * 32;
    static constexpr int MMAS_PER_STAGE = BK / T::umma_k;
    static constexpr int READERS = CG * (1 + EPI_WARPS) + 1;
    static constexpr uint32_t IDESC = (1u << 4) | (T::fmt << 7) | (T::fmt << 10) |
                                      ((uint32_t)AM << 15) | ((uint32_t)BM << 16) |
                                      ((uint32_t)(BN >> 3) << 17) |
                                      ((uint32_t)(TILE_M >> 4) << 24);
    static_assert(T::mma == MmaKind::F16, "16-bit kinds");
    static_assert(SMEM_BYTES <= SMEM_LIMIT, "shared memory budget");
    static_assert(BN == 256 || (BN == 128 && (CG == 1 || EP == MlpEpi::PLAIN)), "tile shapes");
};

// Byte `b` of row `r` of a staging buffer: 64-byte rows with TMA's 64-byte
// swizzle (the 16-byte piece's index xor row bits 1-2).
__device__ __forceinline__ int stg_offset(int r, int b) {
    return r * 64 + ((((b >> 4) ^ ((r >> 1) & 3)) << 4) | (b & 15));
}

// A staged box (32 rows x 64 bytes) of 16-bit values to output rows that TMA
// does not store: two rows per step, half a warp each, neighbouring lanes on
// neighbouring four-byte words from the row's first 4-byte boundary on (element
// 0 or 1), and single elements where one is left over; eight steps' reads before
// their stores.  Out of line, so that the usual path keeps its registers.
static __device__ __noinline__ void stg_to_global_odd(const uint8_t *stg, uint16_t *dst, int64_t ld,
                                                      int32_t rows_left, int32_t cols_left, int lane) {
    const int left = cols_left < 32 ? cols_left : 32;
    const int even = (int)((uintptr_t)dst >> 1), step = (int)(ld & 1);
    const int r0 = lane >> 4, l = lane & 15;
#pragma unroll 1
    for (int g = 0; g < 32 && g < rows_left; g += 16) {
        uint32_t w[8], first[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = g + 2 * i + r0, c = 2 * l + ((even + r * step) & 1);
            const int c1 = c + 1 < 32 ? c + 1 : 0;
            const uint32_t lo = *reinterpret_cast<const uint16_t *>(stg + stg_offset(r, 2 * c));
            const uint32_t hi = *reinterpret_cast<const uint16_t *>(stg + stg_offset(r, 2 * c1));
            first[i] = *reinterpret_cast<const uint16_t *>(stg + stg_offset(r, 0));
            w[i] = lo | (hi << 16);
        }
        uint16_t *q = dst + (int64_t)(g + r0) * ld;
#pragma unroll
        for (int i = 0; i < 8; ++i, q += 2 * ld) {
            const int r = g + 2 * i + r0, odd = (even + r * step) & 1, c = 2 * l + odd;
            if (r < rows_left) {
                if (c + 1 < left) *reinterpret_cast<uint32_t *>(q + c) = w[i];
                else if (c < left) q[c] = (uint16_t)w[i];
                if (odd && l == 0) q[0] = (uint16_t)first[i];
            }
        }
    }
}
// The same for FP32 values: two rows a step, half a warp each.
static __device__ __noinline__ void stg_to_global_f32(const uint8_t *stg, float *dst, int64_t ld,
                                                      int32_t rows_left, int32_t cols_left, int lane) {
    const int c = lane & 15;
#pragma unroll 4
    for (int r = lane >> 4; r < 32; r += 2)
        if (r < rows_left && c < cols_left)
            dst[(int64_t)r * ld + c] = *reinterpret_cast<const float *>(stg + stg_offset(r, c * 4));
}

// The residual's box (32 rows x 32 values), zero outside, from rows that TMA
// cannot address.
__device__ __forceinline__ void residual_to_stg(uint8_t *stg, const uint16_t *src, int64_t ld,
                                                int32_t row0, int32_t col0, int32_t rows,
                                                int32_t cols, int lane) {
#pragma unroll 8
    for (int r = 0; r < 32; ++r) {
        const bool in = row0 + r < rows && col0 + lane < cols;
        *reinterpret_cast<uint16_t *>(stg + stg_offset(r, lane * 2)) =
            in ? src[(int64_t)(row0 + r) * ld + col0 + lane] : (uint16_t)0;
    }
}

template <Kind KD, int CG, int BN, int AM, int BM, MlpEpi EP>
__global__ void __launch_bounds__(MlpConfig<KD, CG, BN, AM, BM, EP>::NUM_THREADS, 1)
    tg_mlp_kernel(const __grid_constant__ MlpMaps maps, const __grid_constant__ MlpParams mp) {
    using C = MlpConfig<KD, CG, BN, AM, BM, EP>;
    constexpr int S = C::STAGES;
    const GemmParams &p = mp.g;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_ctarank() : 0;  // 0: leader, 1: a pair's peer
    const bool leader = rank == 0;
    const int64_t pair = blockIdx.x / CG;  // this team
    const int64_t num_pairs = gridDim.x / CG;

    auto bar = [&](int i) -> uint32_t { return sbase + C::BAR_OFF + 8 * i; };
    auto a_stage = [&](int s) -> uint32_t { return sbase + C::A_OFF + s * C::A_BYTES; };
    auto b_stage = [&](int s) -> uint32_t { return sbase + C::B_OFF + s * C::B_BYTES; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 4);
    volatile int *fin_ready = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 8);
    volatile uint32_t *gate_seen = reinterpret_cast<volatile uint32_t *>(smem + C::MISC_OFF + 12);
    const PairWaitCtl ctl{abort_flag, map_shared_rank(smem_u32(smem + C::MISC_OFF + 4), rank ^ (CG - 1u)),
                          p.status, p.wait_limit_ns};
    const int nkb = p.num_k_blocks;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(bar(C::FULL0 + s), 1);
            mbar_init(bar(C::EMPTY0 + s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar(C::ACCF0 + a), 1);
            mbar_init(bar(C::ACCE0 + a), CG * C::EPI_WARPS);
        }
        mbar_init(bar(C::DRAIN), 1);
        for (int c = 0; c < C::SLOTS; ++c) {
            mbar_init(bar(C::TKF0 + c), 1);
            mbar_init(bar(C::TKE0 + c), C::READERS);
        }
        for (int w = 0; w < 2 * C::EPI_WARPS; ++w) mbar_init(bar(C::RES0 + w), 1);
        *abort_flag = 0;
        fence_mbar_init();
        if (nkb > 0) {
            prefetch_tensormap(&maps.a[0]);
            prefetch_tensormap(&maps.b[0]);
        }
        if (mp.out[0].tma) prefetch_tensormap(&maps.out[0]);
    }
    if (warp == 1) {
        if constexpr (CG == 2) {
            tmem_alloc_pair(smem_u32(tmem_slot), C::TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
            tmem_relinquish();
        }
    }
    if (mp.late_wait && threadIdx.x == 64) {
        *gate_seen = ld_acquire_gpu_u32(mp.gate);
        fence_proxy_async();  // TMA's reads after it (the barrier below passes that on)
    }
    tc_fence_before();
    if constexpr (CG == 2) cluster_sync_all();
    else __syncthreads();
    tc_fence_after();
    // The kernel before this one: waited for here, or (late_wait) at the end.
    auto wait_before = [&] {
        if (!mp.late_wait) griddep_wait();
    };
    // The same for a producer, whose loads everything else follows (through the
    // stage barriers): with late_wait the gate, acquired above, stands for it.
    auto wait_inputs = [&] {
        if (!mp.late_wait || *gate_seen == 0u) griddep_wait();
    };
    // The next kernel may be set up beside this one from here on; an input
    // gradient holds it back until its own wait (see late_wait, gate).
    constexpr bool HOLD = AM == 0 && BM == 1;
    if (!HOLD) griddep_launch();
    const uint32_t tmem_base = *tmem_slot;
    const UnitPlan up = make_unit_plan(p, num_pairs);
    // Tickets as in the CTA-pair GEMM: the first unit static, later ones
    // claimed in order; the launch's last claim resets the counter.
    const bool tick = p.ticket != nullptr && up.units >= num_pairs;
    auto tk_read = [&](int64_t step) -> int64_t {
        const int slot = (int)(step % C::SLOTS);
        int64_t next = -2;
        if (pair_wait(bar(C::TKF0 + slot), (uint32_t)((step / C::SLOTS) & 1), ctl, SITE_SCHED)) {
            const volatile uint64_t *r =
                reinterpret_cast<const volatile uint64_t *>(smem + C::TK_OFF + 16 * slot);
            next = (int64_t)r[0];
        }
        if (leader) mbar_arrive(bar(C::TKE0 + slot));
        else mbar_arrive_cluster(map_shared_rank(bar(C::TKE0 + slot), 0));
        return next;
    };
    auto tk_read_warp = [&](int64_t step) -> int64_t {
        int64_t next = 0;
        if (lane == 0) next = tk_read(step);
        return __shfl_sync(0xffffffffu, next, 0);
    };

    if (warp == 0) {
        // ------------------------------------------------------ producer (both CTAs)
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            int64_t issued = 0;
            bool ok = true;
            int64_t step = 0;
            bool waited = false;
            for (int64_t u = pair; ok && u >= 0 && u < up.units;) {
                const Unit un = decode_unit(up, u, nkb);
                int bt, mb, nb;
                batch_tile_coords(un.tile, p, bt, mb, nb);
                if (!waited) {
                    wait_inputs();
                    waited = true;
                }
                if (tick) {
                    const int slot = (int)(step % C::SLOTS);
                    mbar_arrive_expect_tx(bar(C::TKF0 + slot), 16);
                    if (leader) {
                        if (step >= C::SLOTS &&
                            !pair_wait(bar(C::TKE0 + slot),
                                       (uint32_t)(((step / C::SLOTS) - 1) & 1), ctl, SITE_SCHED)) {
                            ok = false;
                            break;
                        }
                        const uint32_t v = atomicAdd(p.ticket, 1u);
                        int64_t next = num_pairs + (int64_t)v;
                        if (next >= up.units) {
                            next = -1;
                            if ((int64_t)v == up.units - 1) atomicExch(p.ticket, 0u);
                        }
                        volatile int64_t *stg =
                            reinterpret_cast<volatile int64_t *>(smem + C::TICKET_OFF + 16 * slot);
                        stg[0] = next;
                        stg[1] = 0;
                        fence_proxy_async_smem();
                        const uint32_t src = sbase + C::TICKET_OFF + 16 * slot;
                        const uint32_t dst = sbase + C::TK_OFF + 16 * slot;
                        const uint32_t fb = bar(C::TKF0 + slot);
                        bulk_copy_s2cluster(map_shared_rank(dst, 0), src, 16,
                                            map_shared_rank(fb, 0));
                        if constexpr (CG == 2)
                            bulk_copy_s2cluster(map_shared_rank(dst, 1), src, 16,
                                                map_shared_rank(fb, 1));
                    }
                }
                const int32_t arow = mb * C::TILE_M + (int32_t)rank * BLOCK_M;
                const int32_t brow = nb * C::OUT_N + (C::DUAL ? 0 : (int32_t)rank * C::B_ROWS);
                const bool down = p.k_snake && ((un.tile / num_pairs) & 1);
                for (int i = 0; i < un.k1 - un.k0; ++i) {
                    const int kb = down ? un.k1 - 1 - i : un.k0 + i;
                    const bool second = kb >= mp.k_blocks0;
                    const int32_t kc = (second ? kb - mp.k_blocks0 : kb) * C::BK;
                    const CUtensorMap *ma = &maps.a[second || bt ? 1 : 0];
                    const CUtensorMap *mb_ = &maps.b[(C::DUAL ? rank != 0 : second) ? 1 : 0];
                    if (!pair_wait(bar(C::EMPTY0 + s), ph ^ 1, ctl, SITE_EMPTY)) { ok = false; break; }
                    const uint32_t full =
                        CG == 2 ? map_shared_rank(bar(C::FULL0 + s), 0) : bar(C::FULL0 + s);
                    if (leader)
                        mbar_arrive_expect_tx(bar(C::FULL0 + s), CG * (C::A_BYTES + C::B_BYTES));
                    auto load = [&](uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y) {
                        if constexpr (CG == 2) tma_load_2d_pair(dst, map, full, x, y);
                        else tma_load_2d(dst, map, full, x, y);
                    };
                    if constexpr (AM == 0) {
                        load(a_stage(s), ma, kc, arow);
                    } else {
#pragma unroll
                        for (int q = 0; q < BLOCK_M / 64; ++q)
                            load(a_stage(s) + q * 8192, ma, arow + q * 64, kc);
                    }
                    if constexpr (BM == 0) {
                        load(b_stage(s), mb_, kc, brow);
                        if constexpr (C::DUAL && CG == 1)
                            load(b_stage(s) + C::B_BYTES / 2, &maps.b[1], kc, brow);
                    } else {
#pragma unroll
                        for (int q = 0; q < C::B_ROWS / 64; ++q)
                            load(b_stage(s) + q * 8192, mb_, brow + q * 64, kc);
                    }
                    ++issued;
                    if (++s == S) { s = 0; ph ^= 1; }
                }
                if (!ok) break;
                u = tick ? tk_read(step++) : u + num_pairs;
            }
            // Copies already issued land within microseconds; their barriers
            // may be the peer's, which this thread cannot poll.
            if (!ok && issued) pair_pause_ns(200000);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer (leader)
        wait_before();
        if (HOLD) {
            if (mp.gate && blockIdx.x == 0 && lane == 0) st_release_gpu_u32(mp.gate, 1u);
            __syncwarp();
            griddep_launch();
        }
        if (leader && lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            uint32_t tl = 0;
            bool ok = true;
            int64_t step = 0;
            auto commit = [&](uint32_t b) {  // an arrival in every CTA of the team
                if constexpr (CG == 2) mma_commit_pair_mcast(b, (uint16_t)0x3);
                else mma_commit(b);
            };
            for (int64_t u = pair; ok && u >= 0 && u < up.units; ++tl) {
                const Unit un = decode_unit(up, u, nkb);
                const uint32_t acc = tl & 1, use = tl >> 1;
                if (!pair_wait(bar(C::ACCE0 + acc), (use & 1) ^ 1, ctl, SITE_ACC_EMPTY)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * BN;
                for (int i = 0; i < un.k1 - un.k0; ++i) {
                    if (!pair_wait(bar(C::FULL0 + s), ph, ctl, SITE_FULL)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a0 = a_stage(s), b0 = b_stage(s);
#pragma unroll
                    for (int kk = 0; kk < C::MMAS_PER_STAGE; ++kk) {
                        // 16 reduction indexes: 32 bytes of a K-major row, 16
                        // rows of 128 bytes of an MN-major box.
                        const uint64_t ad = AM ? smem_desc_mn_sw128(a0 + kk * 2048)
                                               : smem_desc_sw128(a0 + kk * 32);
                        const uint64_t bd = BM ? smem_desc_mn_sw128(b0 + kk * 2048)
                                               : smem_desc_sw128(b0 + kk * 32);
                        if constexpr (CG == 2) mma_f16_pair(d_tmem, ad, bd, C::IDESC, (i != 0) || (kk != 0));
                        else mma_f16(d_tmem, ad, bd, C::IDESC, (i != 0) || (kk != 0));
                    }
                    commit(bar(C::EMPTY0 + s));
                    if (++s == S) { s = 0; ph ^= 1; }
                }
                if (!ok) break;
                commit(bar(C::ACCF0 + acc));
                u = tick ? tk_read(step++) : u + num_pairs;
            }
            if (!ok) {
                if constexpr (CG == 2) mma_commit_pair_mcast(bar(C::DRAIN), (uint16_t)1);
                else mma_commit(bar(C::DRAIN));
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(bar(C::DRAIN), 0)) {
                    if (globaltimer_ns() - t0 > p.wait_limit_ns) {
                        atomicCAS(p.status, 0u, (uint32_t)SITE_DRAIN);
                        break;
                    }
                }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ epilogue (both CTAs)
        wait_before();
        const int q = warp & 3;
        const int ew = warp - 2;
        constexpr int EPI_THREADS = C::EPI_WARPS * 32;
        const int etid = threadIdx.x - 64;
        constexpr int COLS = C::COLS;
        const int cbase = (ew / 4) * COLS;
        // Two staging buffers, used in turn: `cur` is the next one to fill.
        uint8_t *const stg0 = smem + C::STG_OFF + ew * 2 * C::STG_BYTES;
        float4 *const bias_s = reinterpret_cast<float4 *>(smem + C::BIAS_OFF + ew * 128);
        uint32_t cur = 0;
        uint32_t res_phase = 0;  // one bit per buffer
        uint32_t tl = 0;
        int64_t step = 0;
        bool alive = true;
        for (int64_t u = pair;; ++tl) {
            // With split tiles the epilogue warps meet on named barriers, so
            // they leave together: a warp whose wait gave up takes all along.
            if (up.segs > 1 ? named_bar_any(2, EPI_THREADS, u == -2 || !alive)
                            : (u == -2 || !alive))
                break;
            if (u < 0 || u >= up.units) break;
            const Unit un = decode_unit(up, u, nkb);
            int bt, mb, nb;
            batch_tile_coords(un.tile, p, bt, mb, nb);
            const uint32_t acc = tl & 1, use = tl >> 1;
            const int32_t row0 = mb * C::TILE_M + (int32_t)rank * BLOCK_M + q * 32;
            const int32_t colw = nb * C::OUT_N + cbase;  // first output column of this warp
            const bool writer = un.seg >= 0 && un.seg < up.segs - 1;
            const bool finisher = un.seg >= 0 && !writer;

            // Ask for the residual box at column `col` into buffer `at`, whose
            // last store, if any, must have left it (wait: all stores so far).
            auto ask_residual = [&](int32_t col, uint32_t at) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bulk_wait_read<0>();
                    const uint32_t b = bar(C::RES0 + 2 * ew + at);
                    mbar_arrive_expect_tx(b, C::STG_BYTES);
                    tma_load_2d(smem_u32(stg0 + at * C::STG_BYTES), &maps.r, b, col, row0);
                }
            };
            bool asked = false;
            if constexpr (EP == MlpEpi::LINEAR) {
                if (mp.r && mp.r_tma && !mp.out[1].ptr && !writer && row0 < p.m && colw < p.n) {
                    ask_residual(colw, cur);
                    asked = true;
                }
            }

            const bool got = pair_wait(bar(C::ACCF0 + acc), use & 1, ctl, SITE_ACC_FULL);
            if (up.segs > 1 ? named_bar_any(2, EPI_THREADS, !got) : !__all_sync(0xffffffffu, got)) {
                alive = false;
            }
            if (!alive) {
                if (asked) pair_pause_ns(200000);  // the box may still be landing
                break;
            }
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * BN;
            auto part = [&](int32_t k) -> float * {
                const int64_t pidx = un.tail * (up.segs - 1) + k;
                return p.ws + ((pidx * CG + rank) * BN) * (int64_t)BLOCK_M + q * 32 + lane;
            };
            auto flag = [&](int32_t k) -> uint32_t * {
                return p.flags + (un.tail * (up.segs - 1) + k) * CG + rank;
            };
            if (writer) {
                float *dst = part(un.seg);
                constexpr int ACOLS = BN / 2;
                const int a0 = (ew / 4) * ACOLS;
#pragma unroll 1
                for (int c0 = a0; c0 < a0 + ACOLS; c0 += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(taddr + c0, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        __stcg(dst + (int64_t)(c0 + j) * BLOCK_M, __uint_as_float(v[j]));
                }
                __threadfence();
                named_bar_sync(1, EPI_THREADS);
                if (etid == 0) st_release_gpu_u32(flag(un.seg), 1u);
            } else {
                bool ready = true;
                if (finisher) {
                    if (etid == 0) {
                        const uint64_t t0 = globaltimer_ns();
                        for (int32_t k = 0; k < up.segs - 1 && ready; ++k) {
                            while (ld_acquire_gpu_u32(flag(k)) == 0u) {
                                if (*abort_flag || globaltimer_ns() - t0 > p.wait_limit_ns) {
                                    if (!*abort_flag) pair_raise_abort(ctl, SITE_PARTIAL);
                                    ready = false;
                                    break;
                                }
                            }
                        }
                        *fin_ready = ready ? 1 : 0;
                    }
                    named_bar_sync(1, EPI_THREADS);
                    ready = *fin_ready != 0;
                    if (ready)
                        for (int32_t k = 0; k < up.segs - 1; ++k) (void)ld_acquire_gpu_u32(flag(k));
                }
                // 32 accumulator columns of this thread's row (plus the other
                // segments' partial sums, in segment order).
                auto load_acc = [&](int c0, float (&y)[32]) {
                    if (nkb == 0) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) y[j] = 0.0f;
                        return;
                    }
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(taddr + c0, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) y[j] = __uint_as_float(v[j]);
                    if (finisher) {
                        // All segments' loads of these columns at once: one
                        // round trip to L2, not one per segment.
                        const int32_t parts = up.segs - 1;
                        float w[SPLIT_PARTS][32];
#pragma unroll
                        for (int k = 0; k < SPLIT_PARTS; ++k) {
                            const float *src = part(k < parts ? k : 0) + (int64_t)c0 * BLOCK_M;
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                w[k][j] = k < parts ? __ldcg(src + (int64_t)j * BLOCK_M) : 0.0f;
                        }
#pragma unroll
                        for (int k = 0; k < SPLIT_PARTS; ++k)
#pragma unroll
                            for (int j = 0; j < 32; ++j) y[j] += w[k][j];
                    }
                };
                auto stg16 = [&](int piece) -> uint4 * {
                    return reinterpret_cast<uint4 *>(stg0 + cur * C::STG_BYTES +
                                                     stg_offset(lane, piece * 16));
                };
                // Buffer `cur` may be written: its store, the one before the
                // last, has left it.
                auto free_stg = [&]() {
                    if (lane == 0) bulk_wait_read<1>();
                    __syncwarp();
                };
                // Buffer `cur` goes out as columns col.. of output o.
                auto send = [&](int o, int32_t col) {
                    const bool f32 = EP == MlpEpi::PLAIN && mp.out_f32;
                    uint8_t *stg = stg0 + cur * C::STG_BYTES;
                    if (mp.out[o].tma && (mp.clip || col + (f32 ? 16 : 32) <= p.n)) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) tma_store_2d(&maps.out[o], smem_u32(stg), col, row0);
                    } else {
                        __syncwarp();
                        if (f32)
                            stg_to_global_f32(stg, static_cast<float *>(mp.out[o].ptr) +
                                                       (int64_t)row0 * mp.out[o].ld + col,
                                              mp.out[o].ld, p.m - row0, p.n - col, lane);
                        else
                            stg_to_global_odd(stg, static_cast<uint16_t *>(mp.out[o].ptr) +
                                                       (int64_t)row0 * mp.out[o].ld + col,
                                              mp.out[o].ld, p.m - row0, p.n - col, lane);
                        __syncwarp();
                    }
                    if (lane == 0) bulk_commit();  // one group per buffer filled
                    cur ^= 1;
                };
                // 32 values as a 16-bit staged row.
                auto put = [&](const float (&y)[32]) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *stg16(j) = make_uint4(mlp_pack2<KD>(y[8 * j], y[8 * j + 1]),
                                               mlp_pack2<KD>(y[8 * j + 2], y[8 * j + 3]),
                                               mlp_pack2<KD>(y[8 * j + 4], y[8 * j + 5]),
                                               mlp_pack2<KD>(y[8 * j + 6], y[8 * j + 7]));
                };
                const bool rows_in = ready && row0 < p.m;
                if constexpr (EP == MlpEpi::LINEAR) {
#pragma unroll 1
                    for (int c = 0; c < COLS && rows_in && colw + c < p.n; c += 32) {
                        const int32_t col = colw + c;
                        float y[32];
                        if (mp.bias) {
                            __syncwarp();
                            reinterpret_cast<float *>(bias_s)[lane] =
                                col + lane < p.n ? mp.bias[col + lane] : 0.0f;
                            __syncwarp();
                        }
                        load_acc(cbase + c, y);
                        if (mp.bias) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float4 b = bias_s[j];
                                y[4 * j] += b.x;
                                y[4 * j + 1] += b.y;
                                y[4 * j + 2] += b.z;
                                y[4 * j + 3] += b.w;
                            }
                        }
                        if (mp.out[1].ptr) {
                            free_stg();
                            put(y);
                            send(1, col);
                        }
                        const bool r_tma = mp.r && mp.r_tma;
                        if (r_tma) {
                            // With Z both buffers turn over every 32 columns, so
                            // the box is asked for here; else it was asked for one
                            // step ago, and the next one goes out now.
                            if (!asked) ask_residual(col, cur);
                            asked = !mp.out[1].ptr && c + 32 < COLS && col + 32 < p.n;
                            if (asked) ask_residual(col + 32, cur ^ 1);
                        }
                        mlp_with_act(mp.act, [&](auto a) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) y[j] = mlp_act<a.value>(y[j]);
                        });
                        if (r_tma) {
                            const bool landed = pair_wait(bar(C::RES0 + 2 * ew + cur),
                                                          (res_phase >> cur) & 1, ctl, SITE_RESIDUAL);
                            res_phase ^= 1u << cur;
                            if (!__all_sync(0xffffffffu, landed)) {
                                pair_pause_ns(200000);
                                asked = false;
                                alive = false;
                                break;
                            }
                        } else {
                            free_stg();
                            if (mp.r) {
                                residual_to_stg(stg0 + cur * C::STG_BYTES,
                                                static_cast<const uint16_t *>(mp.r), mp.ldr, row0, col,
                                              p.m, p.n, lane);
                                __syncwarp();
                            }
                        }
                        if (mp.r) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint4 w = *stg16(j);
                                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    y[8 * j + 2 * e] += mlp_to_float<KD>(ws[e] & 0xffffu);
                                    y[8 * j + 2 * e + 1] += mlp_to_float<KD>(ws[e] >> 16);
                                }
                            }
                        }
                        put(y);
                        send(0, col);
                    }
                } else if constexpr (EP == MlpEpi::GATED) {
                    constexpr int UP = BN / 2;  // accumulator column of the up half
#pragma unroll 1
                    for (int c = 0; c < COLS && rows_in && colw + c < p.n; c += 32) {
                        const int32_t col = colw + c;
                        float y[32], w[32];
                        load_acc(cbase + c, y);
                        load_acc(UP + cbase + c, w);
                        if (mp.out[1].ptr) {
                            free_stg();
                            put(y);
                            send(1, col);
                        }
                        if (mp.out[2].ptr) {
                            free_stg();
                            put(w);
                            send(2, col);
                        }
                        mlp_with_act(mp.act, [&](auto a) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) y[j] = mlp_act<a.value>(y[j]) * w[j];
                        });
                        free_stg();
                        put(y);
                        send(0, col);
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < COLS && rows_in && colw + c < p.n; c += 32) {
                        float y[32];
                        load_acc(cbase + c, y);
                        if (mp.out_f32) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                if (colw + c + 16 * h >= p.n) break;
                                free_stg();
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    *stg16(j) = make_uint4(__float_as_uint(y[16 * h + 4 * j]),
                                                           __float_as_uint(y[16 * h + 4 * j + 1]),
                                                           __float_as_uint(y[16 * h + 4 * j + 2]),
                                                           __float_as_uint(y[16 * h + 4 * j + 3]));
                                send(bt, colw + c + 16 * h);
                            }
                        } else {
                            free_stg();
                            put(y);
                            send(bt, colw + c);
                        }
                    }
                }
                if (finisher) {
                    named_bar_sync(1, EPI_THREADS);
                    if (etid == 0 && ready)
                        for (int32_t k = 0; k < up.segs - 1; ++k) *flag(k) = 0u;
                }
            }
            if (asked) pair_pause_ns(200000);  // an unread box (the finisher gave up): let it land
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(bar(C::ACCE0 + acc));
                else mbar_arrive_cluster_relaxed(map_shared_rank(bar(C::ACCE0 + acc), 0));
            }
            u = tick ? tk_read_warp(step++) : u + num_pairs;
        }
        if (lane == 0) bulk_wait_all();
    }

    if (mp.late_wait) {
        griddep_wait();
        if (blockIdx.x == 0 && threadIdx.x == 0) *reinterpret_cast<volatile uint32_t *>(mp.gate) = 0u;
    }
    tc_fence_before();
    if constexpr (CG == 2) cluster_sync_all();
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (CG == 2) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
        else tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

}  // namespace tg
