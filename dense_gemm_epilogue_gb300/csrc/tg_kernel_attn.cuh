// Attention forward: O = softmax(scale Q K^T) V over packed sequences.
//
// A tile is 128 rows: `tokens` consecutive tokens of a sequence times the
// `group` query heads that share a key head, so that every key and value that
// comes in serves the whole group.  Over blocks of 128 keys, for each row,
//   s_j = q . k_j,  p_j = 2^(c s_j - r),  c = scale log2 e
//   l' = l 2^(r - r') + sum p_j,  o' = o 2^(r - r') + sum p_j v_j
// and in the end o / l: one pass, with O and S in tensor memory and a thread
// for each row.  Any reference r' >= r near the row's maximum (times c) will do;
// it is raised, and O rescaled, in a few blocks only.  p is rounded to 16 bits for
// the second product, whose operand it is; l sums it unrounded in FP32.  (That rounding
// is O's distance from FP32 probabilities, 0.0022 of its norm in BF16 and 0.00025 in FP16:
// to a form that rounds p likewise it is 0.00013 and 0.00003.)
//
// NQ = 2 (many tiles): two tiles a CTA, four warps each for the softmax, a warp for
// the loads, a thread for each tile's MMAs.  While the warps of one tile work on
// their scores the tensor core runs the other tile's two products.  P overwrites
// S (128-wide heads; the tensor core runs a CTA's MMAs in the order of issue,
// so the next S waits for P V), or has columns of its own (64-wide).
// NQ = 1 (few rows, long keys; short sequences): one tile, S doubled, so that
// the next block's S runs while the softmax is on this one's, and a deep ring
// of keys and values; the keys may be cut into `splits` ranges of `chunk`
// blocks, whose rows go unnormalised, in FP32, to the workspace, where
// tg_attn_join_kernel adds them.
//
// Bound, many tiles: the tensor core in principle (4 x 128 x 128 x 128 multiply-adds
// a block of two tiles, 2048 cycles), in fact the chain S, softmax, P V of a tile,
// whose next S has no columns before P V is through: 2950 cycles a block.  8192
// tokens, 32 heads over 8 of 128, causal: 336 us alone, 1.64 PFLOP/s; 356 (1.54) in
// long runs at the power limit.  Tried and slower there: eight softmax warps a tile
// (378 to 405), the loads' registers given to the softmax, and blocks of 64 keys with S
// twice (377; S of 128 x 64 reads its operands at 48 cycles a step for 32 of
// arithmetic).  Bound, single tokens: memory (32 tokens over 355 to 11800 keys, 91
// us, 5.9 TB/s; one over 131072 keys 88.5, 6.06).
#pragma once

#include "tg_attn_work.cuh"

namespace tg {

template <Kind KD, int DT, int NQ>
struct AttnConfig {
    using T = KindTraits<KD>;
    static constexpr int HALVES = DT / 64;                // 64-value boxes of a row
    static constexpr int TILE_BYTES = HALVES * 128 * 128;  // 128 rows
    static constexpr int FIT = (SMEM_LIMIT - 2048 - NQ * TILE_BYTES) / TILE_BYTES;
    static constexpr int STAGES = FIT > 12 ? 12 : FIT;
    static constexpr int Q_OFF = 0;
    static constexpr int KV_OFF = NQ * TILE_BYTES;
    static constexpr int BAR_OFF = KV_OFF + STAGES * TILE_BYTES;
    static constexpr int QF = 0, FULL0 = 1, EMPTY0 = FULL0 + STAGES, SF0 = EMPTY0 + STAGES, PR0 = SF0 + 2,
                         PH0 = PR0 + 2, PVA0 = PH0 + 2, OD0 = PVA0 + 2, PVD = OD0 + 2, TURN0 = PVD + 1, DRAIN0 = TURN0 + 2,
                         QE = DRAIN0 + 2, OE0 = QE + 1, WF0 = OE0 + 2, WE0 = WF0 + 2, NEXT = WE0 + 2,
                         NUM_BARS = NEXT + 1;
    static constexpr int NEXT_OFF = (BAR_OFF + NUM_BARS * 8 + 15) / 16 * 16;  // launch control's answer
    static constexpr int MISC_OFF = NEXT_OFF + 16;
    static constexpr int WORK_OFF = MISC_OFF + 16;  // two pieces of work
    static constexpr int SMEM_BYTES = WORK_OFF + 2 * sizeof(AttnWork) + 1024;
    static constexpr int SOFT_WARPS = 4 * NQ;
    static constexpr int LOAD_WARP = SOFT_WARPS, MMA_WARP = SOFT_WARPS + 1;
    static constexpr int NUM_THREADS = 32 * (SOFT_WARPS + 1 + NQ);  // an MMA warp a tile
    static constexpr int TMEM_COLS = 512;
    static constexpr int O_COL = 256;
    static constexpr int P_COL = DT == 64 ? O_COL + NQ * DT : 0;  // (DT == 128: over S)
    static constexpr int P_STEP = DT == 64 ? 64 : 128;
    static constexpr uint32_t ID_BASE = (1u << 4) | (T::fmt << 7) | (T::fmt << 10) | ((128u >> 4) << 24);
    static constexpr uint32_t ID_S = ID_BASE | ((128u >> 3) << 17);
    static constexpr uint32_t ID_PV = ID_BASE | (1u << 16) | ((uint32_t)(DT >> 3) << 17);
    static_assert(SMEM_BYTES <= SMEM_LIMIT && STAGES >= 4, "shared memory budget");
};

// S (128 x 128) = A (rows of DT) B^T (rows of DT), both K-major tiles of 64-value boxes
// (the 16-value steps K0 to K1 of the reduction).
template <int K0, int K1>
__device__ __forceinline__ void attn_mma_rows(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
    const uint64_t da = smem_desc_sw128(a), db = smem_desc_sw128(b);
#pragma unroll
    for (int kk = K0; kk < K1; ++kk) {
        const int at = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
        mma_f16(d, da + at, db + at, idesc, kk != 0);
    }
}
// D (128 x N) (+)= A (tensor memory) B (MN-major tile of 128 rows), over the
// reduction values 16 K0 to 16 K1; HALF: columns from A's value 0 to its value 64.
template <int K0, int K1, int HALF>
__device__ __forceinline__ void attn_mma_ta(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                            bool accumulate) {
    const uint64_t db = smem_desc_mn_rows128(b);
#pragma unroll
    for (int kk = K0; kk < K1; ++kk)
        mma_f16_ta(d, a + (kk >> 2) * HALF + (kk & 3) * 8, db + kk * (2048 >> 4), idesc, kk ? 1 : accumulate);
}

// Zeroes a row of a tile: rows behind a sequence's end hold others' values, and 0
// times an infinity or a NaN would reach the sums.
template <int HALVES>
__device__ __forceinline__ void attn_zero_row(uint8_t *tile, int row) {
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
        uint4 *q = reinterpret_cast<uint4 *>(tile + h * 16384 + row * 128);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = make_uint4(0, 0, 0, 0);
    }
}

// COLS columns from tensor memory, times f, to a 16-bit row of which `left` values
// exist; zeros where a thread has none.  (A warp loads when any has: `load`.)
template <Kind KD, int COLS>
__device__ __forceinline__ void attn_store_row(uint32_t at, bool some, bool load, float f, bool valid,
                                               int left, uint16_t *dst) {
#pragma unroll 1
    for (int i = 0; i < COLS; i += 32) {
        uint32_t o[32];
        if (load) {
            tmem_ld_row32(at + i, o);
            tmem_ld_wait();
        }
        if (!valid) continue;
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
            if (i + e >= left) break;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (some) {
                uint32_t y[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    y[q] = pack_half2<KD>(__uint_as_float(o[e + 2 * q]) * f, __uint_as_float(o[e + 2 * q + 1]) * f);
                v = make_uint4(y[0], y[1], y[2], y[3]);
            }
            *reinterpret_cast<uint4 *>(dst + i + e) = v;
        }
    }
}

// Key blocks of a piece of work: from jb, to je[t] for tile t; `all` together.
template <int NQ>
struct AttnBlocks {
    int jb, je[NQ], all;
    __device__ __forceinline__ AttnBlocks(const AttnForward &p, const AttnWork &w) {
        jb = w.split * p.chunk;
        int last = jb;
#pragma unroll
        for (int t = 0; t < NQ; ++t) {
            const int end = w.first + (t + 1) * p.h.tokens;  // tokens before it are in tiles up to t
            const int tokens = end < w.lq ? end : w.lq;
            const int seen = tokens > w.first + t * p.h.tokens ? attn_seen(p.s, w, tokens - 1) : 0;
            je[t] = (seen + ATTN_KEYS - 1) / ATTN_KEYS;
            if (je[t] > jb + p.chunk) je[t] = jb + p.chunk;
            if (je[t] < jb) je[t] = jb;
            if (je[t] > last) last = je[t];
        }
        all = last - jb;
    }
};

template <Kind KD, int DT, int NQ>
__global__ void __launch_bounds__(AttnConfig<KD, DT, NQ>::NUM_THREADS, 1)
    tg_attn_kernel(const __grid_constant__ AttnForward p) {
    using C = AttnConfig<KD, DT, NQ>;
    constexpr int S = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](int i) -> uint32_t { return sbase + C::BAR_OFF + 8 * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 4);
    const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns};

    if (threadIdx.x == 0) {
        mbar_init(bar(C::QF), 1);
        mbar_init(bar(C::QE), NQ);
        for (int s = 0; s < S; ++s) {
            mbar_init(bar(C::FULL0 + s), 1);
            mbar_init(bar(C::EMPTY0 + s), NQ);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(C::SF0 + i), 1);
            mbar_init(bar(C::PR0 + i), 4);
            mbar_init(bar(C::PH0 + i), 4);
            mbar_init(bar(C::PVA0 + i), 1);
            mbar_init(bar(C::OD0 + i), 1);
            mbar_init(bar(C::OE0 + i), 4);
            mbar_init(bar(C::TURN0 + i), 1);
            mbar_init(bar(C::DRAIN0 + i), 1);
            mbar_init(bar(C::WF0 + i), 1);
            mbar_init(bar(C::WE0 + i), C::SOFT_WARPS + NQ);
        }
        mbar_init(bar(C::PVD), 1);
        mbar_init(bar(C::NEXT), 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&p.q);
        prefetch_tensormap(&p.k);
        prefetch_tensormap(&p.v);
    }
    if (warp == C::MMA_WARP) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch();
    griddep_wait();
    const uint32_t tmem = *tmem_slot;
    // Piece `step` of this CTA's work, from LOAD_WARP.
    auto work_at = [&](int step) -> volatile AttnWork * {
        return reinterpret_cast<volatile AttnWork *>(smem + C::WORK_OFF) + (step & 1);
    };
    auto read_work = [&](int step) -> AttnWork {
        const volatile AttnWork *v = work_at(step);
        AttnWork w;
        w.seq = v->seq;
        w.first = v->first;
        w.q0 = v->q0;
        w.lq = v->lq;
        w.k0 = v->k0;
        w.lk = v->lk;
        w.head = v->head;
        w.split = v->split;
        return w;
    };

    int asked = 0, loads = 0, tiles_q = 0;  // LOAD_WARP: answers, ring items, Q tiles asked for so far
    if (warp == C::LOAD_WARP) {
        // ------------------------------------------------------ work and loads
        // A CTA that is done takes over the work of one that has not started (launch
        // control), so that only its first piece waits for its set-up: the next piece
        // is asked for, found and loaded while the ring's last blocks are in work.  (Asked
        // for earlier, the last pieces went to CTAs that were not the first to be free.)
        int item = blockIdx.x, step = 0;
        bool ok = true;
        while (ok) {
            AttnWork w;
            w.head = -1;
            if (item >= 0) {
                // Pieces count down through the tiles: the last tokens of a sequence see
                // the most keys, and the long work is better begun first.
                const int rest = item / p.splits;
                w = attn_find<false>(p.s, p.tiles - 1 - rest / p.h.kv_heads, NQ * p.h.tokens, lane);
                w.head = rest % p.h.kv_heads;
                w.split = item % p.splits;
            }
            if (w.seq >= 0) {
                if (!wait_warp(bar(C::WE0 + (step & 1)), (uint32_t)(step >> 1 & 1) ^ 1, ctl, SITE_SCHED)) break;
                if (lane == 0) {
                    volatile AttnWork *v = work_at(step);
                    v->seq = w.seq;
                    v->first = w.first;
                    v->q0 = w.q0;
                    v->lq = w.lq;
                    v->k0 = w.k0;
                    v->lk = w.lk;
                    v->head = w.head;
                    v->split = w.split;
                    mbar_arrive(bar(C::WF0 + (step & 1)));
                }
                ++step;
                __syncwarp();
                const AttnBlocks<NQ> b(p, w);
                if (b.all > 0) {
                    if (elect_one()) {
                        ok = wait_phase(bar(C::QE), (uint32_t)(tiles_q & 1) ^ 1, ctl, SITE_EMPTY);
                        if (ok) {
                            mbar_arrive_expect_tx(bar(C::QF), NQ * C::HALVES * p.h.tokens * p.h.group * 128);
#pragma unroll
                            for (int t = 0; t < NQ; ++t)
#pragma unroll
                                for (int h = 0; h < C::HALVES; ++h)
                                    tma_load_4d(sbase + C::Q_OFF + t * C::TILE_BYTES + h * 16384, &p.q, bar(C::QF),
                                                h * 64, 0, w.head, w.q0 + w.first + t * p.h.tokens);
                            ++tiles_q;
                        }
                        int s = loads % S;
                        uint32_t ph = (uint32_t)(loads / S) & 1;
                        for (int it = 0; ok && it < 2 * b.all; ++it) {
                            if (!wait_phase(bar(C::EMPTY0 + s), ph ^ 1, ctl, SITE_EMPTY)) { ok = false; break; }
                            mbar_arrive_expect_tx(bar(C::FULL0 + s), C::TILE_BYTES);
                            const int row = w.k0 + (b.jb + (it >> 1)) * ATTN_KEYS;
#pragma unroll
                            for (int h = 0; h < C::HALVES; ++h)
                                tma_load_3d(sbase + C::KV_OFF + s * C::TILE_BYTES + h * 16384, it & 1 ? &p.v : &p.k,
                                            bar(C::FULL0 + s), h * 64, w.head, row);
                            ++loads;
                            if (++s == S) { s = 0; ph ^= 1; }
                        }
                    }
                    // (the counts of the lane that loaded, the only one that counted)
                    loads = __reduce_max_sync(0xffffffffu, loads);
                    tiles_q = __reduce_max_sync(0xffffffffu, tiles_q);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                }
            }
            if (lane == 0) {
                fence_proxy_async_smem();
                mbar_arrive_expect_tx(bar(C::NEXT), 16);
                clc_try_cancel(sbase + C::NEXT_OFF, bar(C::NEXT));
            }
            ++asked;
            __syncwarp();
            ok = wait_warp(bar(C::NEXT), (uint32_t)(asked - 1) & 1, ctl, SITE_SCHED);
            if (!ok) break;
            const volatile uint64_t *answer = reinterpret_cast<const volatile uint64_t *>(smem + C::NEXT_OFF);
            item = clc_cancelled_x(answer[0], answer[1]);
            __syncwarp();
            if (item < 0) {
                if (!wait_warp(bar(C::WE0 + (step & 1)), (uint32_t)(step >> 1 & 1) ^ 1, ctl, SITE_SCHED)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    work_at(step)->head = -1;
                    mbar_arrive(bar(C::WF0 + (step & 1)));
                }
                break;
            }
        }
    } else if (warp >= C::MMA_WARP) {
        // A thread for each tile's products: while one waits for its probabilities
        // the other's are in the tensor core's queue, which holds only a few (with
        // one thread for both, 0.3 of the time was between a wait and the next MMA).
        // They take turns, a tile's P V and next S at a time: mixed, both tiles'
        // scores would be ready at once and both tiles' softmax stand idle at once.
        const int t = warp - C::MMA_WARP;
        if (elect_one()) {
            const uint32_t q = sbase + C::Q_OFF + t * C::TILE_BYTES;
            const uint32_t o = tmem + C::O_COL + t * DT;
            // The ring's items in order: K, V, K, V, ...
            struct Ring {
                int s = 0;
                uint32_t ph = 0;
                __device__ void next() {
                    if (++s == S) { s = 0; ph ^= 1; }
                }
            } k, v;  // the next K, the next V
            v.next();
            auto tile = [&](const Ring &r) -> uint32_t { return sbase + C::KV_OFF + r.s * C::TILE_BYTES; };
            auto full = [&](const Ring &r) -> bool {
                const bool ok = wait_phase(bar(C::FULL0 + r.s), r.ph, ctl, SITE_FULL);
                tc_fence_after();
                return ok;
            };
            auto release = [&](Ring &r) {
                mma_commit(bar(C::EMPTY0 + r.s));
                r.next();
                r.next();
            };
            uint32_t turns = t;  // of the other thread's awaited so far, odd for t = 1
            auto turn = [&]() -> bool {
                if (NQ == 1) return true;
                const uint32_t n = turns++;  // (t = 0 begins: it awaits the other's n - 1)
                return n == 0 || wait_phase(bar(C::TURN0 + t), (n - 1) & 1, ctl, SITE_ACC_EMPTY);
            };
            auto pass = [&] {
                if (NQ == 2) mbar_arrive(bar(C::TURN0 + (t ^ 1)));
            };
            bool ok = true;
            uint32_t g = 0;             // blocks of this tile so far
            uint32_t pieces = 0, o_used = 0;  // pieces with keys; those with keys for this tile
            for (int step = 0; ok; ++step) {
                ok = wait_phase(bar(C::WF0 + (step & 1)), (uint32_t)(step >> 1) & 1, ctl, SITE_SCHED);
                if (!ok) break;
                const AttnWork w = read_work(step);
                mbar_arrive(bar(C::WE0 + (step & 1)));
                if (w.head < 0) break;
                const AttnBlocks<NQ> b(p, w);
                const int all = b.all, mine = (NQ == 2 && t ? b.je[NQ - 1] : b.je[0]) - b.jb;
                if (all == 0) continue;
                auto scores = [&](int n) {
                    const int slot = NQ == 2 ? t : (int)((g + n) & 1);
                    attn_mma_rows<0, DT / 16>(tmem + slot * 128, q, tile(k), C::ID_S);
                    mma_commit(bar(C::SF0 + slot));
                    if (n + 1 == mine) mma_commit(bar(C::QE));
                };
                ok = wait_phase(bar(C::QF), pieces & 1, ctl, SITE_FULL) && full(k) && turn();
                if (!ok) break;
                ++pieces;
                if (mine > 0) scores(0);
                else mma_commit(bar(C::QE));
                release(k);
                pass();
                for (int n = 0; n < all; ++n) {
                    const int slot = NQ == 2 ? t : (int)((g + n) & 1);
                    const uint32_t phase = NQ == 2 ? (g + n) & 1 : ((g + n) >> 1) & 1;
                    // (Waits that can be before the turn are: one on shared memory takes
                    // 150 cycles under the MMAs' reads even when its phase is over.)
                    ok = full(v) && (n + 1 == all || full(k));
                    if (!ok) break;
                    if (NQ == 1 && n + 1 < all) {
                        scores(n + 1);
                        release(k);
                    }
                    if (n == 0 && mine > 0 && o_used > 0)  // (O is still the piece's before)
                        ok = wait_phase(bar(C::OE0 + t), (o_used - 1) & 1, ctl, SITE_ACC_EMPTY);
                    ok = ok && (n >= mine || wait_phase(bar(C::PH0 + slot), phase, ctl, SITE_PROBABILITIES)) && turn();
                    if (!ok) break;
                    if (n < mine) {
                        const uint32_t pr = tmem + C::P_COL + slot * C::P_STEP;
                        tc_fence_after();
                        attn_mma_ta<0, 4, 32>(o, pr, tile(v), C::ID_PV, n > 0);
                        mma_commit(bar(C::PVA0 + t));
                        ok = wait_phase(bar(C::PR0 + slot), phase, ctl, SITE_PROBABILITIES);
                        if (!ok) break;
                        tc_fence_after();
                        attn_mma_ta<4, 8, 32>(o, pr, tile(v), C::ID_PV, true);
                    }
                    release(v);
                    if (NQ == 1) mma_commit(bar(C::PVD));
                    if (n + 1 == mine) mma_commit(bar(C::OD0 + t));
                    // (P over S: these scores overwrite what P V above still reads.  No barrier is
                    // between them, only the tensor core's order, that of issue by one thread: the
                    // two stay in this thread and in this order.)
                    if (NQ == 2 && n + 1 < all) {
                        if (n + 1 < mine) scores(n + 1);
                        release(k);
                    }
                    pass();
                }
                if (mine > 0) {
                    g += mine;
                    ++o_used;
                }
            }
            if (!ok) {
                mma_commit(bar(C::DRAIN0 + t));
                wait_phase_drain(bar(C::DRAIN0 + t), 0, ctl);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ softmax: a row a thread
        const int t = NQ == 2 ? warp >> 2 : 0;
        const int row = threadIdx.x & 127;
        const uint32_t lane_base = (uint32_t)(warp & 3) << 21;  // lane field: bits 16 up
        // The reference r, in units of log2, is the maximum of the first block; later
        // it stands until a half block's sum of 2^(c s - r) says that it is too small
        // (the sum is needed anyway, the maximum would cost a quarter of the softmax's
        // time).  FP32 sums and BF16 probabilities are as exact far above 1 as below; in
        // FP16 the limit keeps them from overflow.
        constexpr float LIMIT = KD == Kind::BF16 ? 1073741824.0f : 16384.0f;
        const float c = p.h.scale_log2;
        const uint64_t cc = pair2(c, c);
        const uint32_t o_at = tmem + lane_base + C::O_COL + t * DT;
        bool ok = true;
        uint32_t g = 0, o_used = 0;  // blocks of this tile so far; pieces with any
        int ring = 0;                // ring items of the pieces so far
        for (int step = 0; ok; ++step) {
            ok = wait_warp(bar(C::WF0 + (step & 1)), (uint32_t)(step >> 1) & 1, ctl, SITE_SCHED);
            if (!ok) break;
            const AttnWork w = read_work(step);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::WE0 + (step & 1)));
            if (w.head < 0) break;
            const AttnBlocks<NQ> b(p, w);
            const int head = w.head, jb = b.jb;
            const int token = w.first + t * p.h.tokens + row / p.h.group;
            const int qh = head * p.h.group + row % p.h.group;
            const bool valid = row < p.h.tokens * p.h.group && token < w.lq;
            const int seen = valid ? attn_seen(p.s, w, token) : 0;
            const int first_seen = attn_seen(p.s, w, w.first + t * p.h.tokens);  // the tile's least
            const int end = NQ == 2 && t ? b.je[NQ - 1] : b.je[0];
            // A row that is not the sequence's (another's, or one that no load wrote) has no say
            // in when its warp raises: the others' last bits would go by what it holds.
            float r = 0.0f, l = 0.0f, limit = valid ? LIMIT : INFINITY;
            for (int j = jb; j < end; ++j) {
                const int n = j - jb;
                const int slot = NQ == 2 ? t : (int)((g + n) & 1);
                const uint32_t phase = NQ == 2 ? (g + n) & 1 : ((g + n) >> 1) & 1;
                if (!wait_warp(bar(C::SF0 + slot), phase, ctl, SITE_SCORES)) { ok = false; break; }
                tc_fence_after();
                const uint32_t s_at = tmem + lane_base + slot * 128;
                const bool cut = (j + 1) * ATTN_KEYS > first_seen;
                const int lim = cut ? seen - j * ATTN_KEYS : ATTN_KEYS;
                // Half the row's scores at a time: all 128 at once leave the CTA's
                // registers short.
                auto half = [&](int h, uint32_t *s) {
                    tmem_ld_row32(s_at + h, s);
                    tmem_ld_row32(s_at + h + 32, s + 32);
                    tmem_ld_wait();
                    if (cut) {
#pragma unroll
                        for (int i = 0; i < 64; ++i)
                            if (h + i >= lim) s[i] = 0xff800000u;
                    }
                };
                auto largest = [&](const uint32_t *s) -> float {
                    float mx[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mx[i] = max3(__uint_as_float(s[3 * i]), __uint_as_float(s[3 * i + 1]), __uint_as_float(s[3 * i + 2]));
#pragma unroll
                    for (int i = 12; i < 64; i += 2)
                        mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
                    return max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
                };
                uint32_t s[64], y[32];
                auto exponentials = [&]() -> float {
                    const uint64_t rr = pair2(-r, -r);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float a, b;
                        unpair2(fma_pair(pair2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), cc, rr), a, b);
                        a = exp2_approx(a);
                        b = exp2_approx(b);
                        sum[i & 1] = add_pair(sum[i & 1], pair2(a, b));
                        y[i] = pack_half2<KD>(a, b);
                    }
                    float a, b;
                    unpair2(add_pair(sum[0], sum[1]), a, b);
                    return a + b;
                };
                // A reference that is not below `top`, and what was summed by the old one.
                // (A row whose scores were all -infinity so far has summed nothing: `top`
                // is its first reference, however low.)
                auto raise = [&](float top) {
                    const bool first = limit < 0.0f;
                    const float to = first ? (top == -INFINITY ? 0.0f : top) : fmaxf(r, top);
                    const float f = first ? 0.0f : exp2_approx(r - to);
                    if (first && top != -INFINITY) limit = LIMIT;
                    r = to;
                    l *= f;
#pragma unroll 1
                    for (int i = 0; i < DT; i += 32) {
                        uint32_t o[32];
                        tmem_ld_row32(o_at + i, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st_32x32b_x32(o_at + i, o);
                    }
                };
                auto put = [&](int h, uint32_t arrived) {
                    tmem_st_32x32b_x32(tmem + lane_base + C::P_COL + slot * C::P_STEP + h / 2, y);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(arrived + slot));
                };
                if (n == 0) {
                    half(64, s);
                    const float mx = largest(s);
                    half(0, s);
                    const float top = fmaxf(mx, largest(s));
                    r = top * c;
                    if (top == -INFINITY) {
                        r = 0.0f;
                        if (valid && lim > 0) limit = -1.0f;
                    }
                } else {
                    half(0, s);
                }
                float sum = exponentials();
                if (n > 0 && __any_sync(0xffffffffu, sum > limit)) {
                    // (P over S: the first half is not stored before this is known.)
                    if (NQ == 1 && !wait_warp(bar(C::PVD), (g + n - 1) & 1, ctl, SITE_ACC_FULL)) { ok = false; break; }
                    tc_fence_after();
                    half(64, s);
                    const float mx = largest(s);
                    half(0, s);
                    raise(fmaxf(mx, largest(s)) * c);
                    sum = exponentials();
                }
                // Values behind the sequence's end: zero (see attn_zero_row).  (The barrier is
                // at most one phase behind: the thread that issued these scores has waited
                // for the slot's earlier items.)
                if (w.lk - j * ATTN_KEYS < ATTN_KEYS) {
                    const int it = ring + 2 * n + 1;
                    if (!wait_warp(bar(C::FULL0 + it % S), (uint32_t)(it / S) & 1, ctl, SITE_FULL)) { ok = false; break; }
                    if (row >= w.lk - j * ATTN_KEYS) {
                        attn_zero_row<C::HALVES>(smem + C::KV_OFF + (it % S) * C::TILE_BYTES, row);
                        fence_proxy_async_smem();
                    }
                }
                put(0, C::PH0);
                l += sum;
                half(64, s);
                sum = exponentials();
                if (n > 0 && __any_sync(0xffffffffu, sum > limit)) {
                    // The first half's product is under way by the old reference.  With one tile
                    // S runs ahead: these scores say that P V(n - 2) is over, and another warp may
                    // still keep P V(n - 1) waiting, so PVA0 may be a phase behind, whose parity
                    // would pass for this one's.  P V(n - 1) first.
                    if (NQ == 1 && !wait_warp(bar(C::PVD), (g + n - 1) & 1, ctl, SITE_ACC_FULL)) { ok = false; break; }
                    if (!wait_warp(bar(C::PVA0 + t), (g + n) & 1, ctl, SITE_ACC_FULL)) { ok = false; break; }
                    tc_fence_after();
                    raise(largest(s) * c);
                    sum = exponentials();
                }
                put(64, C::PR0);
                l += sum;
            }
            const bool some = end > jb;
            if (ok && some) {
                ok = wait_warp(bar(C::OD0 + t), o_used & 1, ctl, SITE_ACC_FULL);
                tc_fence_after();
            }
            if (!ok) break;
            {
                const int64_t at = (int64_t)qh * p.s.q_rows + w.q0 + token;
                if (p.splits > 1) {
                    const int64_t slot = (int64_t)w.split * p.h.heads * p.s.q_rows + at;
                    if (valid) p.part_ml[slot] = make_float2(r, l);
                    float4 *dst = reinterpret_cast<float4 *>(p.part_o + slot * p.h.dim);
                    if (some) {
#pragma unroll 1
                        for (int i = 0; i < DT; i += 32) {
                            uint32_t o[32];
                            tmem_ld_row32(o_at + i, o);
                            tmem_ld_wait();
                            if (valid && l != 0.0f) {
#pragma unroll
                                for (int e = 0; e < 32; e += 4)
                                    if (i + e < p.h.dim)
                                        dst[(i + e) >> 2] = make_float4(
                                            __uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                            __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
                            }
                        }
                    }
                } else {
                    if (valid && p.lse) p.lse[at] = l == 0.0f ? -INFINITY : (r + log2f(l)) * 0.6931471805599453f;
                    attn_store_row<KD, DT>(o_at, some && l != 0.0f, some, l == 0.0f ? 0.0f : 1.0f / l, valid, p.h.dim,
                                           static_cast<uint16_t *>(p.o.ptr) + (w.q0 + (int64_t)token) * p.o.ld +
                                               qh * p.o.hd);
                }
            }
            if (some) {
                // (the next piece may use O)
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::OE0 + t));
                g += end - jb;
                ++o_used;
            }
            ring += 2 * b.all;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag && warp == C::LOAD_WARP && lane == 0) {
        // What was asked for lands before the CTA exits.
        if (asked) wait_phase_drain(bar(C::NEXT), (uint32_t)(asked - 1) & 1, ctl);
        if (tiles_q) wait_phase_drain(bar(C::QF), (uint32_t)(tiles_q - 1) & 1, ctl);
        for (int i = loads > S ? loads - S : 0; i < loads; ++i)
            wait_phase_drain(bar(C::FULL0 + i % S), (uint32_t)(i / S) & 1, ctl);
    }
    if (warp == C::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// The rows of a tile from their key ranges: with M the largest reference,
//   L = sum l_s 2^(m_s - M),  O = sum o_s 2^(m_s - M) / L,  LSE = (M + log2 L) ln 2,
// always in the same order.  WIDE: the block's eight warps share a row's ranges (a
// few rows with many ranges); else a warp a row.  blockIdx.y: which rows of the tile.
// Bound: its launch and two dependent reads (32 single tokens: 7.6 us by itself).
constexpr int JOIN_WARPS = 8;
template <Kind KD, bool WIDE>
__global__ void __launch_bounds__(32 * JOIN_WARPS) tg_attn_join_kernel(const __grid_constant__ AttnForward p) {
    __shared__ float4 part[WIDE ? JOIN_WARPS : 1][32];
    __shared__ float sums[WIDE ? JOIN_WARPS : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_launch();
    griddep_wait();
    const int head = blockIdx.x % p.h.kv_heads;
    const AttnWork w = attn_find<false>(p.s, blockIdx.x / p.h.kv_heads, p.join_tokens, lane);
    const int row = WIDE ? blockIdx.y : blockIdx.y * JOIN_WARPS + warp;
    const int token = w.first + row / p.h.group, qh = head * p.h.group + row % p.h.group;
    if (w.seq < 0 || row >= p.join_tokens * p.h.group || token >= w.lq) return;  // (WIDE: the whole block)
    const int64_t stride = (int64_t)p.h.heads * p.s.q_rows;
    const int64_t at = (int64_t)qh * p.s.q_rows + w.q0 + token;
    // Lane i looks at ranges i, i + 32, ...
    float m = -INFINITY;
    for (int s = lane; s < p.splits; s += 32) {
        const float2 ml = p.part_ml[s * stride + at];
        if (ml.y != 0.0f) m = fmaxf(m, ml.x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int step = WIDE ? JOIN_WARPS : 1;
#pragma unroll 4
    for (int s = WIDE ? warp : 0; s < p.splits; s += step) {
        const float2 ml = p.part_ml[s * stride + at];
        if (ml.y == 0.0f) continue;  // (nothing was stored)
        const float g = exp2_approx(ml.x - m);
        l += ml.y * g;
        if (4 * lane < p.h.dim) {
            const float4 v = reinterpret_cast<const float4 *>(p.part_o + (s * stride + at) * p.h.dim)[lane];
            o[0] += v.x * g;
            o[1] += v.y * g;
            o[2] += v.z * g;
            o[3] += v.w * g;
        }
    }
    if constexpr (WIDE) {
        part[warp][lane] = make_float4(o[0], o[1], o[2], o[3]);
        if (lane == 0) sums[warp] = l;
        __syncthreads();
        if (warp) return;
        for (int i = 1; i < JOIN_WARPS; ++i) {
            const float4 v = part[i][lane];
            o[0] += v.x;
            o[1] += v.y;
            o[2] += v.z;
            o[3] += v.w;
            l += sums[i];
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (lane == 0 && p.lse) p.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    if (4 * lane < p.h.dim) {
        uint16_t *dst = static_cast<uint16_t *>(p.o.ptr) + (w.q0 + token) * p.o.ld + qh * p.o.hd;
        *reinterpret_cast<uint2 *>(dst + 4 * lane) =
            make_uint2(pack_half2<KD>(o[0] * inv, o[1] * inv), pack_half2<KD>(o[2] * inv, o[3] * inv));
    }
}

}  // namespace tg
