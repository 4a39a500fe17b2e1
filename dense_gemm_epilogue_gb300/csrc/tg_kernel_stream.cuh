// Feed-forward products for few tokens: the weights stream through the
// tensor cores once, at the memory's rate.
//
//   out(j, f) = epi(sum_k W(f, k) X(j, k)),  j < tokens <= NT, f < features
//
// With few tokens a product reads N K weights for 2 M N K operations, so the
// weights' bytes bound it (M = 1: 1 FLOP a byte).  Here the weights are the
// 128-row operand and the tokens the NT-column one (NT = 16, 32 or, not gated,
// 64, zero rows beyond the tokens), so every weight byte crosses shared memory
// once and the accumulator wastes columns, which cost nothing, instead of
// rows.  One CTA per SM keeps a ring of 100 or 200 KB of TMA loads in flight: 6.7
// TB/s at about 1 us of latency needs 44 KB per SM.  With the small ring the next
// kernel's CTA fits beside this one: its set-up and, for short shares, an L2
// prefetch of its first weights run under this kernel's end.  What a call costs
// above its bytes is about 5.5 us of start, join and end; in between the weights
// arrive at 6.6 TB/s (1 x 4096 x 4096 10.7 us, 1 x 16384 x 4096 25.8; these and the
// times below are of a captured chain of calls, inputs past L2).
//
// Work split: the (tile, K block) iterations of all 128-feature tiles are cut
// into equal contiguous shares, one per CTA, so that 112 tiles (say) load 152
// SMs evenly.  A CTA walks its share from the end to the start.  Its first
// unit may end short of a tile's last K block: it writes the FP32 partial
// sums and raises a flag.  The CTA that holds a tile's last K block finishes
// it: it adds the partials of the CTAs before it, nearest first (a fixed
// order), and runs the epilogue.  It reaches such a tile last, when the
// partials, which their owners computed first, are long there; and it waits
// only for CTAs of lower index, so no two wait on each other.
//
// Gated: each stage holds 128 gate rows and the same 128 up rows; two MMAs
// share the token operand and one thread holds g and u of its feature.
// Transposed (the input gradient, dX = dZ W or dG Wg + dU Wu): the streamed
// operand's rows are the products' reduction index, so its 128 features lie
// along its rows (MN-major, two 64 x 64 boxes a stage), and the K blocks may
// run over two operand pairs in turn.
#pragma once

#include <cstdint>
#include "tg_kernel_mlp.cuh"

namespace tg {

enum class StreamOp : int { LINEAR = 0, GATED = 1, DGRAD = 2 };

template <Kind KD, int NT, StreamOp OP>
struct StreamConfig {
    using T = KindTraits<KD>;
    static constexpr bool DUAL = OP == StreamOp::GATED, TRANS = OP == StreamOp::DGRAD;
    static constexpr int BK = T::block_k;
    static constexpr int MATS = DUAL ? 2 : 1;
    static constexpr int A_BYTES = BLOCK_M * ROW_BYTES;
    static constexpr int B_BYTES = NT * ROW_BYTES;
    static constexpr int STAGE_BYTES = MATS * A_BYTES + B_BYTES;
    // One weight matrix and up to 32 tokens: a ring of about 100 KB, two CTAs to
    // an SM (1 x 4096 x 4096 10.7 us, 11.0 with all of shared memory; 1 x 16384 x
    // 4096 25.8, 27.2); else all of it (gated, 4 x 14336 x 4096: 42.2 us either way).
    static constexpr bool SMALL = NT <= 32 && !DUAL;
    static constexpr int BUDGET = SMALL ? SMEM_LIMIT / 2 - 1024 : SMEM_LIMIT;
    static constexpr int FIT = (BUDGET - 2048) / STAGE_BYTES;
    static constexpr int STAGES = FIT > 12 ? 12 : FIT;
    // K blocks prefetched into L2 ahead of the first load (256 KB a CTA), and the
    // longest share that this pays for: 1 x 4096 x 4096 (13 blocks a CTA) 10.7 us
    // with it and 11.0 without, 1 x 16384 x 4096 (54) 27.0 and 25.8.
    static constexpr int PREFETCH = 16 / MATS, PREFETCH_SHARE = 32;
    static constexpr int BAR_OFF = STAGES * STAGE_BYTES;
    static constexpr int FULL0 = 0, EMPTY0 = STAGES, ACCF0 = 2 * STAGES, ACCE0 = ACCF0 + 2,
                         DRAIN = ACCE0 + 2, NUM_BARS = DRAIN + 1;
    static constexpr int MISC_OFF = BAR_OFF + NUM_BARS * 8;
    static constexpr int SMEM_BYTES = MISC_OFF + 16 + 1024;
    static constexpr int ACC_COLS = MATS * NT;
    static constexpr int TMEM_COLS = 2 * ACC_COLS;
    static constexpr int EPI_WARPS = 8;  // two per tensor-memory lane quarter
    static constexpr int NUM_THREADS = (2 + EPI_WARPS) * 32;
    static constexpr int MMAS_PER_STAGE = BK / T::umma_k;
    static constexpr uint32_t IDESC = (1u << 4) | (T::fmt << 7) | (T::fmt << 10) |
                                      ((uint32_t)TRANS << 15) | ((uint32_t)(NT >> 3) << 17) |
                                      ((uint32_t)(BLOCK_M >> 4) << 24);
    static_assert(SMEM_BYTES <= SMEM_LIMIT, "shared memory budget");
    static_assert(TMEM_COLS >= 32 && TMEM_COLS <= 512, "tensor-memory allocation");
};

struct StreamMaps {
    CUtensorMap w[2], x[2];
};

struct StreamParams {
    int32_t tokens, features, tiles, num_k_blocks;
    int32_t k_blocks0;  // K blocks of the first operand pair (DGRAD)
    int32_t act;
    const float *bias;
    const void *r;
    int64_t ldr;
    MlpOut out[3];  // LINEAR: Y, Z; GATED: H, G, U
    float *ws;      // one slot of 128 x 256 floats per CTA
    uint32_t *flags;  // eight per CTA (one per epilogue warp), zero between launches
    uint32_t *gate;   // DGRAD: as MlpParams::gate
    uint32_t *status;
    uint64_t wait_limit_ns;
};

// This CTA's units, highest tile first.
struct StreamUnits {
    int64_t lo, pos;
    int32_t t, k0, k1;
    __device__ __forceinline__ StreamUnits(const StreamParams &p) {
        const int64_t total = (int64_t)p.tiles * p.num_k_blocks;
        lo = sk_start(total, blockIdx.x, gridDim.x);
        pos = sk_start(total, blockIdx.x + 1, gridDim.x);
        t = k0 = k1 = 0;
    }
    __device__ __forceinline__ bool next(const StreamParams &p) {
        if (pos <= lo) return false;
        const int nkb = p.num_k_blocks;
        t = (int32_t)((pos - 1) / nkb);
        const int64_t base = (int64_t)t * nkb;
        k1 = (int32_t)(pos - base);
        k0 = lo > base ? (int32_t)(lo - base) : 0;
        pos = base + k0;
        return true;
    }
};

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

template <Kind KD>
__device__ __forceinline__ uint16_t mlp_narrow(float y) {
    if constexpr (KD == Kind::BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(y));
    else return __half_as_ushort(__float2half_rn(y));
}

template <Kind KD, int NT, StreamOp OP>
__global__ void __launch_bounds__(StreamConfig<KD, NT, OP>::NUM_THREADS,
                                  StreamConfig<KD, NT, OP>::SMALL ? 2 : 1)
    tg_stream_kernel(const __grid_constant__ StreamMaps maps, const StreamParams p) {
    using C = StreamConfig<KD, NT, OP>;
    constexpr bool DUAL = C::DUAL, TRANS = C::TRANS;
    constexpr int S = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    auto bar = [&](int i) -> uint32_t { return sbase + C::BAR_OFF + 8 * i; };
    // A stage: the token rows after the weight rows (16 KB each, so every
    // part starts on a swizzle atom).
    auto stage = [&](int s) -> uint32_t { return sbase + s * C::STAGE_BYTES; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 4);
    const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns};

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(bar(C::FULL0 + s), 1);
            mbar_init(bar(C::EMPTY0 + s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar(C::ACCF0 + a), 1);
            mbar_init(bar(C::ACCE0 + a), C::EPI_WARPS);
        }
        mbar_init(bar(C::DRAIN), 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&maps.w[0]);
        if (DUAL) prefetch_tensormap(&maps.w[1]);
        prefetch_tensormap(&maps.x[0]);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (an input gradient holds its successor back until its own wait: see
    // MlpParams::late_wait and gate)
    if (!TRANS) griddep_launch();
    const uint32_t tmem_base = *tmem_slot;
    const int nkb = p.num_k_blocks;

    if (warp == 0) {
        if (lane == 0) {
            // The first weights on their way into L2 while the kernel before
            // this one ends: a prefetch consumes no value, so it may run ahead
            // of whatever that kernel still writes.
            {
                StreamUnits un(p);
                for (int left = un.pos - un.lo <= C::PREFETCH_SHARE ? C::PREFETCH : 0;
                     left > 0 && un.next(p);)
                    for (int kb = un.k0; kb < un.k1 && left > 0; ++kb, --left) {
                        const int second = TRANS && kb >= p.k_blocks0;
                        const int32_t kc = (kb - (second ? p.k_blocks0 : 0)) * C::BK;
                        const int32_t f = un.t * BLOCK_M;
                        if constexpr (TRANS) {
                            tma_prefetch_l2_2d(&maps.w[second], f, kc);
                            tma_prefetch_l2_2d(&maps.w[second], f + 64, kc);
                        } else {
                            tma_prefetch_l2_2d(&maps.w[0], kc, f);
                            if (DUAL) tma_prefetch_l2_2d(&maps.w[1], kc, f);
                        }
                    }
            }
            griddep_wait();
            int s = 0;
            uint32_t ph = 0;
            int64_t issued = 0;
            bool ok = true;
            StreamUnits un(p);
            while (ok && un.next(p)) {
                for (int kb = un.k0; kb < un.k1; ++kb) {
                    if (!wait_phase(bar(C::EMPTY0 + s), ph ^ 1, ctl, SITE_EMPTY)) { ok = false; break; }
                    const uint32_t full = bar(C::FULL0 + s);
                    mbar_arrive_expect_tx(full, C::STAGE_BYTES);
                    const int second = TRANS && kb >= p.k_blocks0;
                    const int32_t kc = (kb - (second ? p.k_blocks0 : 0)) * C::BK;
                    const int32_t f = un.t * BLOCK_M;
                    if constexpr (TRANS) {
                        tma_load_2d(stage(s), &maps.w[second], full, f, kc);
                        tma_load_2d(stage(s) + 8192, &maps.w[second], full, f + 64, kc);
                    } else {
                        tma_load_2d(stage(s), &maps.w[0], full, kc, f);
                        if (DUAL) tma_load_2d(stage(s) + C::A_BYTES, &maps.w[1], full, kc, f);
                    }
                    tma_load_2d(stage(s) + C::MATS * C::A_BYTES, &maps.x[second], full, kc, 0);
                    ++issued;
                    if (++s == S) { s = 0; ph ^= 1; }
                }
            }
            if (!ok) {
                for (int st = 0; st < S && st < issued; ++st) {
                    const int64_t last = st + (int64_t)S * ((issued - 1 - st) / S);
                    wait_phase_drain(bar(C::FULL0 + st), (uint32_t)((last / S) & 1), ctl);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        griddep_wait();
        if (TRANS) {
            if (p.gate && blockIdx.x == 0 && lane == 0) st_release_gpu_u32(p.gate, 1u);
            __syncwarp();
            griddep_launch();
        }
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            uint32_t tl = 0;
            bool ok = true;
            StreamUnits un(p);
            while (ok && un.next(p)) {
                const uint32_t acc = tl & 1, use = tl >> 1;
                ++tl;
                if (!wait_phase(bar(C::ACCE0 + acc), (use & 1) ^ 1, ctl, SITE_ACC_EMPTY)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + acc * C::ACC_COLS;
                for (int kb = un.k0; kb < un.k1; ++kb) {
                    if (!wait_phase(bar(C::FULL0 + s), ph, ctl, SITE_FULL)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t a0 = stage(s), b0 = stage(s) + C::MATS * C::A_BYTES;
#pragma unroll
                    for (int kk = 0; kk < C::MMAS_PER_STAGE; ++kk) {
                        const uint64_t bd = smem_desc_sw128(b0 + kk * 32);
                        const uint32_t keep = (kb != un.k0) || (kk != 0);
                        mma_f16(d, TRANS ? smem_desc_mn_sw128(a0 + kk * 2048) : smem_desc_sw128(a0 + kk * 32),
                                bd, C::IDESC, keep);
                        if (DUAL)
                            mma_f16(d + NT, smem_desc_sw128(a0 + C::A_BYTES + kk * 32), bd,
                                    C::IDESC, keep);
                    }
                    mma_commit(bar(C::EMPTY0 + s));
                    if (++s == S) { s = 0; ph ^= 1; }
                }
                if (!ok) break;
                mma_commit(bar(C::ACCF0 + acc));
            }
            if (!ok) {
                mma_commit(bar(C::DRAIN));
                wait_phase_drain(bar(C::DRAIN), 0, ctl);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ epilogue
        griddep_wait();
        // Warp: lane quarter q, tokens [16 h, 16 h + 16), [16 h + 32, ...).
        const int q = warp & 3, h = (warp - 2) >> 2;
        const int ew = warp - 2;
        uint32_t tl = 0;
        bool ok = true;
        StreamUnits un(p);
        while (ok && un.next(p)) {
            const uint32_t acc = tl & 1, use = tl >> 1;
            ++tl;
            ok = __all_sync(0xffffffffu, wait_phase(bar(C::ACCF0 + acc), use & 1, ctl, SITE_ACC_FULL));
            if (!ok) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + acc * C::ACC_COLS;
            float *slot0 = p.ws + q * 32 + lane;  // row of this thread in slot 0
            if (un.k1 < nkb) {
                float *dst = slot0 + (int64_t)blockIdx.x * SK_SLOT_FLOATS;
#pragma unroll 1
                for (int j0 = 16 * h; j0 < p.tokens; j0 += 32) {
                    uint32_t v[C::MATS][16];
#pragma unroll
                    for (int a = 0; a < C::MATS; ++a) tmem_ld_32x32b_x16(taddr + a * NT + j0, v[a]);
                    tmem_ld_wait();
#pragma unroll
                    for (int a = 0; a < C::MATS; ++a)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (j0 + j < p.tokens)
                                __stcg(dst + (int64_t)(a * NT + j0 + j) * BLOCK_M,
                                       __uint_as_float(v[a][j]));
                }
                __threadfence();
                __syncwarp();
                // (a warp without tokens has no reader to put its flag back)
                if (lane == 0 && 16 * h < p.tokens)
                    st_release_gpu_u32(p.flags + blockIdx.x * 8 + ew, 1u);
            } else {
                // The CTAs before this one that hold the tile's first K blocks.
                const int me = (int)blockIdx.x;
                int first = me;
                if (un.k0 > 0 && 16 * h < p.tokens) {
                    const int64_t total = (int64_t)p.tiles * nkb, base = (int64_t)un.t * nkb;
                    do {
                        --first;
                    } while (sk_start(total, first, gridDim.x) > base);
                    // One lane per flag.
                    const uint64_t t0 = globaltimer_ns();
                    for (int c = me - 1 - lane; c >= first && ok; c -= 32) {
                        while (ld_acquire_gpu_u32(p.flags + c * 8 + ew) == 0u) {
                            if (*abort_flag || globaltimer_ns() - t0 > p.wait_limit_ns) {
                                if (!*abort_flag) {
                                    *abort_flag = 1;
                                    atomicCAS(p.status, 0u, (uint32_t)SITE_PARTIAL);
                                }
                                ok = false;
                                break;
                            }
                        }
                    }
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    __threadfence();
                    __syncwarp();
                }
                const int32_t f = un.t * BLOCK_M + q * 32 + lane;
                const bool in = f < p.features;
                const float b = (p.bias && in) ? p.bias[f] : 0.0f;
                // The epilogue of TC tokens from j0 on.
                auto finish = [&](auto tc, int j0) {
                    constexpr int TC = tc.value;
                    // The tokens' sums: this CTA's and the partials, nearest
                    // first, WAYS CTAs' loads in flight at once.
                    constexpr int WAYS = TC == 4 ? 8 : C::SMALL ? 2 : 4;
                    auto load_acc = [&](int a, float (&y)[TC]) {
                        uint32_t v[16];
                        tmem_ld_32x32b_x16(taddr + a * NT + j0, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < TC; ++j) y[j] = __uint_as_float(v[j]);
#pragma unroll 1
                        for (int c = me - 1; c >= first; c -= WAYS) {
                            float w[WAYS][TC];
#pragma unroll
                            for (int i = 0; i < WAYS; ++i) {
                                const float *src = slot0 + (int64_t)(c - i) * SK_SLOT_FLOATS +
                                                   (int64_t)(a * NT + j0) * BLOCK_M;
#pragma unroll
                                for (int j = 0; j < TC; ++j)
                                    w[i][j] = c - i >= first && j0 + j < p.tokens
                                                  ? __ldcg(src + (int64_t)j * BLOCK_M)
                                                  : 0.0f;
                            }
#pragma unroll
                            for (int i = 0; i < WAYS; ++i)
#pragma unroll
                                for (int j = 0; j < TC; ++j) y[j] += w[i][j];
                        }
                    };
                    auto store = [&](int o, const float (&y)[TC]) {
                        if (!in) return;
                        uint16_t *dst = static_cast<uint16_t *>(p.out[o].ptr) + (int64_t)j0 * p.out[o].ld + f;
#pragma unroll
                        for (int j = 0; j < TC; ++j)
                            if (j0 + j < p.tokens) dst[(int64_t)j * p.out[o].ld] = mlp_narrow<KD>(y[j]);
                    };
                    float y[TC];
                    if constexpr (DUAL) {
                        float w[TC];
                        load_acc(0, y);
                        load_acc(1, w);
                        if (p.out[1].ptr) store(1, y);
                        if (p.out[2].ptr) store(2, w);
                        mlp_with_act(p.act, [&](auto a) {
#pragma unroll
                            for (int j = 0; j < TC; ++j) y[j] = mlp_act<a.value>(y[j]) * w[j];
                        });
                    } else {
                        uint16_t rr[TC];
                        if (p.r) {
                            const uint16_t *src = static_cast<const uint16_t *>(p.r) + (int64_t)j0 * p.ldr + f;
#pragma unroll
                            for (int j = 0; j < TC; ++j)
                                rr[j] = in && j0 + j < p.tokens ? src[(int64_t)j * p.ldr] : (uint16_t)0;
                        }
                        load_acc(0, y);
#pragma unroll
                        for (int j = 0; j < TC; ++j) y[j] += b;
                        if (p.out[1].ptr) store(1, y);
                        mlp_with_act(p.act, [&](auto a) {
#pragma unroll
                            for (int j = 0; j < TC; ++j) y[j] = mlp_act<a.value>(y[j]);
                        });
                        if (p.r) {
#pragma unroll
                            for (int j = 0; j < TC; ++j) y[j] += mlp_to_float<KD>(rr[j]);
                        }
                    }
                    store(0, y);
                };
                if (p.tokens <= 4) {
                    if (h == 0) finish(std::integral_constant<int, 4>{}, 0);
                } else {
#pragma unroll 1
                    for (int j0 = 16 * h; j0 < p.tokens; j0 += 32)
                        finish(std::integral_constant<int, 16>{}, j0);
                }
                __syncwarp();
                for (int c = me - 1 - lane; c >= first; c -= 32) p.flags[c * 8 + ew] = 0u;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::ACCE0 + acc));
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

}  // namespace tg
