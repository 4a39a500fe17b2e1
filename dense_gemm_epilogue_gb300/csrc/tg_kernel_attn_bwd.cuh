// Attention backward over packed sequences:
//   P = 2^(c s - LSE log2 e),  dP = dO V^T,  dS = P (dP - delta),  delta = sum_d dO O,
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K
// (s = q . k, c = scale log2 e), the heads of a group summed in dK and dV.
//
// Two kinds of CTAs, each with its sums in tensor memory from the first term to the
// last: one owns 128 keys and goes over the rows that see them (dK, dV: four
// products a tile), one owns a tile of 128 rows and goes over its keys (dQ: three).
// S and dP are computed in both, seven products where five are the least, and
// for that no sum is added to memory by several CTAs: repeated calls agree bit
// for bit, and nothing is cleared before or converted after.
//
// A row tile is the forward kernel's: `tokens` tokens x the group's heads, so the
// keys' CTA adds up a group's heads as it adds up tokens.  P and dS are rounded
// to 16 bits, as tensor-core operands; they stay in tensor memory.  (Those roundings are
// the gradients' distance from FP32 ones, 0.0026 of their norms in BF16 and 0.0003 in
// FP16: to a form that rounds likewise it is 0.0006 and 0.00006 at most.)
//
// Bound: the chain S, dP, dS, products of a tile, like the forward kernel's: keys'
// CTAs 2900 cycles a tile for 2176 of MMAs, rows' CTAs 1800 for 1536 (128-wide
// heads).  8192 tokens, 32 heads over 8 of 128, causal: 1171 us alone, 1260 in long
// runs at the power limit, 1.09 PFLOP/s of the five products (1.53 of the seven).  CTAs
// that stay for several tiles took 1441, halves of P 720 for 693 in the keys' part.
#pragma once

#include "tg_kernel_attn.cuh"

namespace tg {

// delta = sum over d of dO O.  Bound: memory (4096 tokens x 32 heads of 128: 14.5 us with
// a cold L2, 4.6 TB/s).
template <Kind KD>
__global__ void __launch_bounds__(DELTA_THREADS) tg_attn_delta_kernel(const __grid_constant__ AttnDelta p) {
    griddep_launch();
    griddep_wait();
    // 16 lanes a row and head (8 values each): 16 of them a block, heads innermost.
    const int lane = threadIdx.x & 15;
    const int64_t i = (int64_t)blockIdx.x * (DELTA_THREADS / 16) + (threadIdx.x >> 4);
    const int64_t row = i / p.heads;
    const int head = (int)(i - row * p.heads);
    float s = 0.0f;
    if (row < p.rows && 8 * lane < p.dim) {
        const uint4 a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.o) + row * p.ldo +
                                                         head * p.ho + 8 * lane);
        const uint4 b = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.dy) + row * p.lddy +
                                                         head * p.hdy + 8 * lane);
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float a0, a1, b0, b1;
            unpack_half2<KD>(aw[q], a0, a1);
            unpack_half2<KD>(bw[q], b0, b1);
            s = fmaf(a0, b0, s);
            s = fmaf(a1, b1, s);
        }
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0 && row < p.rows) p.delta[(int64_t)head * p.rows + row] = s;
}

template <Kind KD, int DT>
struct AttnBackConfig {
    using T = KindTraits<KD>;
    static constexpr int HALVES = DT / 64;
    static constexpr int TILE_BYTES = HALVES * 128 * 128;
    static constexpr int SOFT_WARPS = 8;
    static constexpr int LOAD_WARP = 8, MMA_WARP = 9, MMA2_WARP = 10, ROWS_WARP = 11;
    static constexpr int NUM_THREADS = 32 * 12;
    static constexpr int TMEM_COLS = 512;
    static constexpr uint32_t ID_BASE = (1u << 4) | (T::fmt << 7) | (T::fmt << 10) | ((128u >> 4) << 24);
    static constexpr uint32_t ID_S = ID_BASE | ((128u >> 3) << 17);
    static constexpr uint32_t ID_PV = ID_BASE | (1u << 16) | ((uint32_t)(DT >> 3) << 17);
    static constexpr uint32_t ID_64 = ID_BASE | (1u << 16) | ((64u >> 3) << 17);  // half the columns
};

// -LSE/scale and -delta come into S and dP as products: a keys' CTA has a key a
// thread, and reading 64 rows' values from shared memory for every tile took 1100
// of its 3500 cycles, against MMAs that read shared memory all the time.  Instead
// one more MMA (16 values of the reduction index) adds weights x parts: a value in
// up to four parts v = sum w_i v_i, each a 16-bit number, good to 2^-24 of v
// (BF16: w = 1; FP16: 2^15, 2^5, 2^-5, 2^-15, for |v| below 2^31).
template <Kind KD>
__device__ __forceinline__ uint4 attn_parts(float v) {
    constexpr bool BF = KD == Kind::BF16;
    float part[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float w = BF ? 1.0f : i == 0 ? 32768.0f : i == 1 ? 32.0f : i == 2 ? 0.03125f : 3.0517578125e-5f;
        const uint32_t h = pack_half2<KD>(v / w, 0.0f);
        float lo, hi;
        unpack_half2<KD>(h, lo, hi);
        part[i] = lo;
        // (an infinity is all in the first part)
        v = fabsf(lo) == INFINITY ? 0.0f : v - lo * w;
    }
    return make_uint4(pack_half2<KD>(part[0], part[1]), pack_half2<KD>(part[2], part[3]), 0u, 0u);
}
template <Kind KD>
__device__ __forceinline__ uint4 attn_weights() {
    return KD == Kind::BF16 ? make_uint4(pack_half2<KD>(1.0f, 1.0f), pack_half2<KD>(1.0f, 1.0f), 0u, 0u)
                            : make_uint4(pack_half2<KD>(32768.0f, 32.0f), pack_half2<KD>(0.03125f, 3.0517578125e-5f),
                                         0u, 0u);
}

// The keys' CTAs: shared memory and tensor memory.
template <Kind KD, int DT>
struct AttnKeysConfig : AttnBackConfig<KD, DT> {
    using B = AttnBackConfig<KD, DT>;
    // Tiles of Q, and of dO.  Two of 128-wide heads fit.  A tile of Q stays from S(n)
    // to dK(n), almost two rounds, and the next but one has a third of a round to
    // arrive in, so its two 64-wide boxes are loaded and given back one by one.
    static constexpr int STAGES = DT == 64 ? 4 : 2;
    static constexpr int QB = STAGES * B::HALVES;  // boxes of Q
    static constexpr int ROW_SLOTS = DT == 64 ? 6 : 3;  // rows' LSE, delta (16 bytes of parts each), keys seen
    static constexpr int ROW_SLOT_BYTES = 2048 + 2048 + 512;
    static constexpr int K_OFF = 0, V_OFF = B::TILE_BYTES, Q_OFF = 2 * B::TILE_BYTES;
    static constexpr int DY_OFF = Q_OFF + STAGES * B::TILE_BYTES;
    static constexpr int ROWS_OFF = DY_OFF + STAGES * B::TILE_BYTES;
    static constexpr int WEIGHTS_OFF = ROWS_OFF + ROW_SLOTS * ROW_SLOT_BYTES;  // 128 rows of 16 bytes
    static constexpr int ZERO_OFF = WEIGHTS_OFF + 2048;                    // 128 rows of 16 zero bytes
    static constexpr int BAR_OFF = ZERO_OFF + 2048;
    static constexpr int KVF = 0, QF0 = 1, QE0 = QF0 + QB, DF0 = QE0 + QB, DE0 = DF0 + STAGES,
                         SF0 = DE0 + STAGES, DPF = SF0 + 2, PR0 = DPF + 1, DSR = PR0 + 2, RF0 = DSR + 1,
                         RE0 = RF0 + ROW_SLOTS, LAST = RE0 + ROW_SLOTS, OD = LAST + 3, TURN = OD + 1, DRAIN = TURN + 2,
                         NUM_BARS = DRAIN + 2;
    static constexpr int MISC_OFF = BAR_OFF + NUM_BARS * 8;
    static constexpr int SMEM_BYTES = MISC_OFF + 64 + 1024;
    // P over S, dS over dP (each thread over the columns it has read).  64-wide heads
    // leave room for S twice, a tile ahead of the warps (which may then be a tile ahead
    // of the thread that awaits P: a barrier for each slot, of S and of P).
    static constexpr int S_SLOTS = DT == 64 ? 2 : 1;
    static constexpr int S_COL = 0, DP_COL = 128 * S_SLOTS, DV_COL = DP_COL + 128, DK_COL = DV_COL + DT;
    static constexpr int P_HALF = 64;  // columns from rows 0-63 to rows 64-127
    static_assert(DK_COL + DT <= 512, "tensor memory");
    static_assert(SMEM_BYTES <= SMEM_LIMIT, "shared memory budget");
};

// 64 FP32 values to 16 bits in 32 columns.
template <Kind KD>
__device__ __forceinline__ void attn_store_half(uint32_t at, const float *y) {
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = pack_half2<KD>(y[2 * i], y[2 * i + 1]);
    tmem_st_32x32b_x32(at, w);
    tmem_st_wait();
}

// COLS columns from tensor memory as FP32 to a row of which `left` values exist.
template <int COLS>
__device__ __forceinline__ void attn_store_part(uint32_t at, bool valid, int left, float *dst) {
#pragma unroll 1
    for (int i = 0; i < COLS; i += 32) {
        uint32_t o[32];
        tmem_ld_row32(at + i, o);
        tmem_ld_wait();
        if (!valid) continue;
#pragma unroll
        for (int e = 0; e < 32; e += 4)
            if (i + e < left)
                *reinterpret_cast<float4 *>(dst + i + e) =
                    make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                                __uint_as_float(o[e + 3]));
    }
}

// The first token that sees a key of the block, and the row tiles from there on.
__device__ __forceinline__ int attn_key_tiles(const AttnBackward &p, const AttnWork &w, int &i0) {
    i0 = p.s.causal ? w.first - w.lk + w.lq : 0;
    if (i0 < 0) i0 = 0;
    return w.seq >= 0 && i0 < w.lq ? (w.lq - i0 + p.h.tokens - 1) / p.h.tokens : 0;
}
// The key blocks that a row tile sees.
__device__ __forceinline__ int attn_row_blocks(const AttnBackward &p, const AttnWork &w) {
    const int end = w.first + p.h.tokens < w.lq ? w.first + p.h.tokens : w.lq;
    const int seen = w.seq >= 0 ? attn_seen(p.s, w, end - 1) : 0;
    return (seen + ATTN_KEYS - 1) / ATTN_KEYS;
}

template <Kind KD, int DT>
__device__ __forceinline__ void attn_keys(const AttnBackward &p, const int block) {
    using C = AttnKeysConfig<KD, DT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](int i) -> uint32_t { return sbase + C::BAR_OFF + 8 * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 4);
    AttnWork *shared_work = reinterpret_cast<AttnWork *>(smem + C::MISC_OFF + 8);
    const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns};
    const int box = p.h.tokens * p.h.group;  // rows of a tile that loads write

    if (threadIdx.x == 0) {
        mbar_init(bar(C::KVF), 1);
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(bar(C::DF0 + s), 1);
            mbar_init(bar(C::DE0 + s), 2);
        }
        for (int s = 0; s < C::QB; ++s) {
            mbar_init(bar(C::QF0 + s), 1);
            mbar_init(bar(C::QE0 + s), 1);
        }
        mbar_init(bar(C::SF0), 1);
        mbar_init(bar(C::SF0 + 1), 1);
        mbar_init(bar(C::DPF), 1);
        mbar_init(bar(C::PR0), C::SOFT_WARPS);
        mbar_init(bar(C::PR0 + 1), C::SOFT_WARPS);
        mbar_init(bar(C::DSR), C::SOFT_WARPS);
        for (int s = 0; s < C::ROW_SLOTS; ++s) {
            mbar_init(bar(C::RF0 + s), 32);
            mbar_init(bar(C::RE0 + s), C::SOFT_WARPS);
        }
        for (int i = 0; i < 3; ++i) mbar_init(bar(C::LAST + i), 1);
        mbar_init(bar(C::OD), 2);
        mbar_init(bar(C::TURN), 1);
        mbar_init(bar(C::TURN + 1), 1);
        mbar_init(bar(C::DRAIN), 1);
        mbar_init(bar(C::DRAIN + 1), 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&p.q);
        prefetch_tensormap(&p.dy);
    }
    // Rows that no load writes stay zero.
    for (int i = threadIdx.x; i < 2 * C::STAGES * (ATTN_ROWS - box); i += C::NUM_THREADS)
        attn_zero_row<C::HALVES>(smem + C::Q_OFF + (i / (ATTN_ROWS - box)) * C::TILE_BYTES,
                                 box + i % (ATTN_ROWS - box));
    if (threadIdx.x < 128) {
        *reinterpret_cast<uint4 *>(smem + C::WEIGHTS_OFF + 16 * threadIdx.x) = attn_weights<KD>();
        *reinterpret_cast<uint4 *>(smem + C::ZERO_OFF + 16 * threadIdx.x) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    if (warp == C::MMA_WARP) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    griddep_wait();
    const int part = block % p.key_parts, rest = block / p.key_parts;
    const int head = rest % p.h.kv_heads;
    if (warp == C::LOAD_WARP) {
        const AttnWork w = attn_find<true>(p.s, rest / p.h.kv_heads, ATTN_KEYS, lane);
        if (lane == 0) *shared_work = w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch();
    const uint32_t tmem = *tmem_slot;
    const AttnWork w = *shared_work;
    int i0;  // the first token of this part
    int tiles = attn_key_tiles(p, w, i0) - part * p.key_tiles;
    tiles = tiles < 0 ? 0 : tiles < p.key_tiles ? tiles : p.key_tiles;
    if (tiles > 0) i0 += part * p.key_tiles * p.h.tokens;
    const int tail = tiles > 0 ? attn_tail_rows(w.lq, i0, tiles, p.h.tokens, p.h.group) : box;  // rows of the last tile
    const bool fix = tail < box;
    auto q_tile = [&](int n) -> int { return C::Q_OFF + n % C::STAGES * C::TILE_BYTES; };
    auto dy_tile = [&](int n) -> int { return C::DY_OFF + n % C::STAGES * C::TILE_BYTES; };
    auto parity = [&](int n) -> uint32_t { return (uint32_t)(n / C::STAGES) & 1; };
    auto s_col = [&](int n) -> int { return C::S_COL + n % C::S_SLOTS * 128; };
    auto q_box = [&](int n, int h) -> int { return n % C::STAGES * C::HALVES + h; };
    // Where the loads of tile n report: a last tile that ends inside reports to
    // ROWS_WARP, which passes it on once the rest is zero.
    const int last = fix ? tiles - 1 : tiles;
    auto q_landed = [&](int n, int h) -> uint32_t { return bar(n == last ? C::LAST + h : C::QF0 + q_box(n, h)); };
    auto dy_landed = [&](int n) -> uint32_t { return bar(n == last ? C::LAST + 2 : C::DF0 + n % C::STAGES); };
    auto landed_parity = [&](int n) -> uint32_t { return n == last ? 0 : parity(n); };

    if (warp == C::LOAD_WARP) {
        if (tiles > 0 && elect_one()) {
            const uint32_t bytes = box * 128;  // of a box
            mbar_arrive_expect_tx(bar(C::KVF), 2 * C::TILE_BYTES);
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h) {
                tma_load_3d(sbase + C::K_OFF + h * 16384, &p.k, bar(C::KVF), h * 64, head, w.k0 + w.first);
                tma_load_3d(sbase + C::V_OFF + h * 16384, &p.v, bar(C::KVF), h * 64, head, w.k0 + w.first);
            }
            int q_n = 0, dy_n = 0;  // boxes of Q, tiles of dO under way
            bool ok = true;
            for (int n = 0; ok && n < tiles; ++n) {
                const int row = w.q0 + i0 + n * p.h.tokens;
                // (dO first: its stage is free half a round before Q's.)
                ok = wait_phase(bar(C::DE0 + n % C::STAGES), parity(n) ^ 1, ctl, SITE_EMPTY);
                if (!ok) break;
                mbar_arrive_expect_tx(dy_landed(n), C::HALVES * bytes);
#pragma unroll
                for (int h = 0; h < C::HALVES; ++h)
                    tma_load_4d(sbase + dy_tile(n) + h * 16384, &p.dy, dy_landed(n), h * 64, 0, head, row);
                ++dy_n;
#pragma unroll
                for (int h = 0; ok && h < C::HALVES; ++h) {
                    ok = wait_phase(bar(C::QE0 + q_box(n, h)), parity(n) ^ 1, ctl, SITE_EMPTY);
                    if (!ok) break;
                    mbar_arrive_expect_tx(q_landed(n, h), bytes);
                    tma_load_4d(sbase + q_tile(n) + h * 16384, &p.q, q_landed(n, h), h * 64, 0, head, row);
                    ++q_n;
                }
            }
            if (!ok) {
                // Every copy already issued lands before the CTA exits.
                wait_phase_drain(bar(C::KVF), 0, ctl);
                for (int i = q_n > C::QB ? q_n - C::QB : 0; i < q_n; ++i)
                    wait_phase_drain(q_landed(i / C::HALVES, i % C::HALVES), landed_parity(i / C::HALVES), ctl);
                for (int n = dy_n > C::STAGES ? dy_n - C::STAGES : 0; n < dy_n; ++n)
                    wait_phase_drain(dy_landed(n), landed_parity(n), ctl);
            }
        }
        __syncwarp();
    } else if (warp == C::MMA_WARP || warp == C::MMA2_WARP) {
        // Two threads, for the products that wait for P (dV, then the next S, over
        // the same columns) and those that wait for dS (dK, then the next dP): while
        // one waits, the other's are in the tensor core's short queue.  The warps turn
        // S into P while dK and dP run, and dP into dS while dV and S do; the threads
        // take turns, so that one pair is done before the other begins.
        const bool first = warp == C::MMA_WARP;
        if (tiles > 0 && elect_one()) {
            // The rows' own terms (attn_parts) of S, and 2 KB on, of dP.
            auto terms = [&](uint32_t d, int n, int at) {
                const uint32_t rows = sbase + C::ROWS_OFF + n % C::ROW_SLOTS * C::ROW_SLOT_BYTES + at;
                mma_f16(d, smem_desc_k2(sbase + C::WEIGHTS_OFF, C::ZERO_OFF - C::WEIGHTS_OFF),
                        smem_desc_k2(rows, sbase + C::ZERO_OFF - rows), C::ID_S, 1);
            };
            auto rows_ready = [&](int n) -> bool {
                const bool ok = wait_phase(bar(C::RF0 + n % C::ROW_SLOTS), (uint32_t)(n / C::ROW_SLOTS) & 1, ctl,
                                           SITE_FULL);
                tc_fence_after();
                return ok;
            };
            // S(n), each half of its reduction as its box of Q comes.
            auto scores = [&](int n) -> bool {
#pragma unroll
                for (int h = 0; h < C::HALVES; ++h) {
                    if (!wait_phase(bar(C::QF0 + q_box(n, h)), parity(n), ctl, SITE_FULL)) return false;
                    tc_fence_after();
                    if (h == 0) attn_mma_rows<0, 4>(tmem + s_col(n), sbase + C::K_OFF, sbase + q_tile(n), C::ID_S);
                    else attn_mma_rows<4, 8>(tmem + s_col(n), sbase + C::K_OFF, sbase + q_tile(n), C::ID_S);
                }
                terms(tmem + s_col(n), n, 0);
                mma_commit(bar(C::SF0 + n % C::S_SLOTS));
                return true;
            };
            auto gradients = [&](int n) {
                attn_mma_rows<0, DT / 16>(tmem + C::DP_COL, sbase + C::V_OFF, sbase + dy_tile(n), C::ID_S);
                terms(tmem + C::DP_COL, n, 2048);
                mma_commit(bar(C::DPF));
                mma_commit(bar(C::DE0 + n % C::STAGES));
            };
            // Turn n of either (S(0), then dV(n - 1) and the next S; dP(0), then dK and dP).
            auto turn = [&](int n) -> bool {
                const bool ok = first ? n == 0 || wait_phase(bar(C::TURN), (n - 1) & 1, ctl, SITE_ACC_EMPTY)
                                      : wait_phase(bar(C::TURN + 1), n & 1, ctl, SITE_ACC_EMPTY);
                tc_fence_after();
                return ok;
            };
            auto pass = [&] { mbar_arrive(bar(first ? C::TURN + 1 : C::TURN)); };
            // Under the MMAs' own reads a wait on shared memory takes 150 cycles even
            // when its phase is over: what comes early is awaited early, and what
            // the other thread has awaited before its turn is not awaited again (dO
            // for dV, Q for dK, the rows' terms for dP).
            constexpr int AHEAD = C::S_SLOTS - 1;  // S(n + AHEAD) goes with dV(n - 1)
            bool ok = wait_phase(bar(C::KVF), 0, ctl, SITE_FULL);
            for (int n = 0; first && ok && n < AHEAD && n < tiles; ++n) ok = rows_ready(n) && scores(n);
            for (int n = 0; ok && n <= tiles; ++n) {
                if (first && n + AHEAD < tiles) ok = rows_ready(n + AHEAD);
                if (!first && n < tiles) ok = wait_phase(bar(C::DF0 + n % C::STAGES), parity(n), ctl, SITE_FULL);
                if (ok && n > 0)
                    ok = first ? wait_phase(bar(C::PR0 + (n - 1) % C::S_SLOTS),
                                            (uint32_t)((n - 1) / C::S_SLOTS) & 1, ctl, SITE_PROBABILITIES)
                               : wait_phase(bar(C::DSR), (n - 1) & 1, ctl, SITE_PROBABILITIES);
                if (!ok || !turn(n)) {
                    ok = false;
                    break;
                }
                // (S over P, and dP over dS, are issued behind the products that read what they
                // overwrite by the same thread: the tensor core's order is that of issue, and
                // nothing else keeps them apart.)
                if (first) {
                    if (n > 0) {
                        attn_mma_ta<0, 8, C::P_HALF>(tmem + C::DV_COL, tmem + s_col(n - 1), sbase + dy_tile(n - 1),
                                                     C::ID_PV, n > 1);
                        mma_commit(bar(C::DE0 + (n - 1) % C::STAGES));
                    }
                    if (n + AHEAD < tiles) ok = scores(n + AHEAD);
                } else {
                    if (n > 0) {
#pragma unroll
                        for (int h = 0; h < C::HALVES; ++h) {
                            attn_mma_ta<0, 8, C::P_HALF>(tmem + C::DK_COL + 64 * h, tmem + C::DP_COL,
                                                         sbase + q_tile(n - 1) + h * 16384, C::ID_64, n > 1);
                            mma_commit(bar(C::QE0 + q_box(n - 1, h)));
                        }
                    }
                    if (n < tiles) gradients(n);
                }
                pass();
            }
            const uint32_t end = bar(ok ? C::OD : C::DRAIN + (first ? 0 : 1));
            mma_commit(end);
            if (!ok) wait_phase_drain(end, 0, ctl);
        }
        __syncwarp();
    } else if (warp == C::ROWS_WARP) {
        // ------------------------------------------------------ the rows' LSE, delta, keys seen
        // (the next tile's values are on their way while this one's are written)
        const float over_scale = 1.0f / p.h.scale;
        float z[4], d[4];
        auto fetch = [&](int n) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = lane + 32 * q, token = i0 + n * p.h.tokens + row / p.h.group;
                z[q] = -INFINITY;
                d[q] = 0.0f;
                if (row < box && token < w.lq) {
                    const int64_t at =
                        (int64_t)(head * p.h.group + row % p.h.group) * p.s.q_rows + w.q0 + token;
                    z[q] = p.lse[at];
                    d[q] = p.delta[at];
                }
            }
        };
        if (tiles > 0) fetch(0);
        for (int n = 0; n < tiles; ++n) {
            const int s = n % C::ROW_SLOTS;
            if (!wait_warp(bar(C::RE0 + s), (uint32_t)(n / C::ROW_SLOTS + 1) & 1, ctl, SITE_EMPTY)) break;
            uint8_t *rows = smem + C::ROWS_OFF + s * C::ROW_SLOT_BYTES;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = lane + 32 * q, token = i0 + n * p.h.tokens + row / p.h.group;
                // A row that is none, or sees nothing: P = 2^(-infinity) = 0.
                *reinterpret_cast<uint4 *>(rows + 16 * row) =
                    attn_parts<KD>(z[q] == -INFINITY ? -INFINITY : -z[q] * over_scale);
                *reinterpret_cast<uint4 *>(rows + 2048 + 16 * row) = attn_parts<KD>(-d[q]);
                *reinterpret_cast<int *>(rows + 4096 + 4 * row) =
                    row < box && token < w.lq ? attn_seen(p.s, w, token) : 0;
            }
            if (n + 1 < tiles) fetch(n + 1);
            fence_proxy_async_smem();
            mbar_arrive(bar(C::RF0 + s));
            if (fix && n == tiles - 1) {
                // Rows of other sequences, in the last tile, become zero.
#pragma unroll
                for (int h = 0; h < C::HALVES + 1; ++h) {
                    const bool q = h < C::HALVES;
                    if (!wait_warp(bar(q ? C::LAST + h : C::LAST + 2), 0, ctl, SITE_FULL)) break;
                    for (int row = tail + lane; row < box; row += 32) {
                        if (q) attn_zero_row<1>(smem + q_tile(n) + h * 16384, row);
                        else attn_zero_row<C::HALVES>(smem + dy_tile(n), row);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(q ? C::QF0 + q_box(n, h) : C::DF0 + n % C::STAGES));
                }
            }
        }
        __syncwarp();
    } else if (w.seq >= 0) {
        // ------------------------------------------------------ a key a thread, 64 rows of it
        const int half = warp >> 2;
        const uint32_t lane_base = (uint32_t)(warp & 3) << 21;
        const int key = w.first + (threadIdx.x & 127);
        const float c = p.h.scale_log2;
        const uint64_t cc = pair2(c, c);
        bool ok = true;
        for (int n = 0; n < tiles; ++n) {
            const int s = n % C::ROW_SLOTS;
            ok = wait_warp(bar(C::SF0 + n % C::S_SLOTS), (uint32_t)(n / C::S_SLOTS) & 1, ctl, SITE_SCORES);
            if (!ok) break;
            tc_fence_after();
            float y[64];
            uint32_t *yw = reinterpret_cast<uint32_t *>(y);
#pragma unroll
            for (int i = 0; i < 2; ++i) tmem_ld_row32(tmem + lane_base + s_col(n) + 64 * half + 32 * i, yw + 32 * i);
            tmem_ld_wait();
            // Some rows of the tile do not see all of the keys.
            const bool cut = p.s.causal && attn_seen(p.s, w, i0 + n * p.h.tokens) < w.first + ATTN_KEYS;
            if (cut) {
                ok = wait_warp(bar(C::RF0 + s), (uint32_t)(n / C::ROW_SLOTS) & 1, ctl, SITE_FULL);
                if (!ok) break;
            }
            const int *seen = reinterpret_cast<const int *>(smem + C::ROWS_OFF + s * C::ROW_SLOT_BYTES + 4096) + 64 * half;
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
                unpair2(mul_pair(pair2(y[i], y[i + 1]), cc), y[i], y[i + 1]);
                y[i] = exp2_approx(y[i]);
                y[i + 1] = exp2_approx(y[i + 1]);
            }
            if (cut) {
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    if (key >= seen[i]) y[i] = 0.0f;
            }
            attn_store_half<KD>(tmem + lane_base + s_col(n) + C::P_HALF * half, y);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::PR0 + n % C::S_SLOTS));

            ok = wait_warp(bar(C::DPF), n & 1, ctl, SITE_SCORES);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < 64; i += 32) {
                uint32_t d[32];
                tmem_ld_row32(tmem + lane_base + C::DP_COL + 64 * half + i, d);
                tmem_ld_wait();
                const float *f = reinterpret_cast<const float *>(d);
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    unpair2(mul_pair(pair2(y[i + e], y[i + e + 1]), pair2(f[e], f[e + 1])), y[i + e], y[i + e + 1]);
            }
            attn_store_half<KD>(tmem + lane_base + C::DP_COL + C::P_HALF * half, y);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(C::DSR));
                mbar_arrive(bar(C::RE0 + s));
            }
        }
        if (ok && tiles > 0) {
            ok = wait_warp(bar(C::OD), 0, ctl, SITE_ACC_FULL);
            tc_fence_after();
        }
        const AttnOut &out = half ? p.dk : p.dv;
        const uint32_t at = tmem + lane_base + (half ? C::DK_COL : C::DV_COL);
        if (ok && out.ptr) {
            if (p.key_parts == 1)
                attn_store_row<KD, DT>(at, tiles > 0, tiles > 0, half ? p.h.scale : 1.0f, key < w.lk, p.h.dim,
                                       static_cast<uint16_t *>(out.ptr) + (w.k0 + (int64_t)key) * out.ld +
                                           head * out.hd);
            else if (tiles > 0)
                attn_store_part<DT>(at, key < w.lk, p.h.dim,
                                    p.part_keys + ((((int64_t)part * 2 + half) * p.h.kv_heads + head) * p.s.k_rows +
                                                   w.k0 + key) * p.h.dim);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == C::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// The rows' CTAs.
template <Kind KD, int DT>
struct AttnRowsConfig : AttnBackConfig<KD, DT> {
    using B = AttnBackConfig<KD, DT>;
    static constexpr int FIT = (SMEM_LIMIT - 2048 - 2 * B::TILE_BYTES) / B::TILE_BYTES;
    static constexpr int STAGES = FIT > 8 ? 8 : FIT;
    // Rings of their own: values are done with after dP, keys only after dQ, and a
    // common ring held up the next values' load behind them.
    static constexpr int KS = (STAGES + 1) / 2, VS = STAGES / 2;
    static constexpr int Q_OFF = 0, DY_OFF = B::TILE_BYTES, KV_OFF = 2 * B::TILE_BYTES;
    static constexpr int BAR_OFF = KV_OFF + STAGES * B::TILE_BYTES;
    static constexpr int QF = 0, FULL0 = 1, EMPTY0 = FULL0 + STAGES, SF = EMPTY0 + STAGES, SE = SF + 1,
                         DPF = SE + 1, DSR = DPF + 1, LAST = DSR + 1, OD = LAST + 2, DRAIN = OD + 1,
                         NUM_BARS = DRAIN + 2;
    static constexpr int MISC_OFF = BAR_OFF + NUM_BARS * 8;
    static constexpr int SMEM_BYTES = MISC_OFF + 64 + 1024;
    static constexpr int S_COL = 0, DP_COL = 128, DQ_COL = 256, DS_COL = 384;  // dS twice, 64 columns each
    static_assert(SMEM_BYTES <= SMEM_LIMIT && STAGES >= 5, "shared memory budget");
};

template <Kind KD, int DT>
__device__ __forceinline__ void attn_rows(const AttnBackward &p, const int block) {
    using C = AttnRowsConfig<KD, DT>;
    constexpr int S = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](int i) -> uint32_t { return sbase + C::BAR_OFF + 8 * i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::MISC_OFF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::MISC_OFF + 4);
    AttnWork *shared_work = reinterpret_cast<AttnWork *>(smem + C::MISC_OFF + 8);
    const WaitCtl ctl{abort_flag, p.status, p.wait_limit_ns};

    if (threadIdx.x == 0) {
        mbar_init(bar(C::QF), 1);
        for (int s = 0; s < S; ++s) {
            mbar_init(bar(C::FULL0 + s), 1);
            mbar_init(bar(C::EMPTY0 + s), 1);
        }
        mbar_init(bar(C::SF), 1);
        mbar_init(bar(C::SE), C::SOFT_WARPS);
        mbar_init(bar(C::DPF), 1);
        mbar_init(bar(C::DSR), C::SOFT_WARPS);
        mbar_init(bar(C::LAST), 1);
        mbar_init(bar(C::LAST + 1), 1);
        mbar_init(bar(C::OD), 1);
        mbar_init(bar(C::DRAIN), 1);
        mbar_init(bar(C::DRAIN + 1), 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&p.k);
        prefetch_tensormap(&p.v);
    }
    if (warp == C::MMA_WARP) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    griddep_wait();
    const int part = block % p.row_parts, rest = block / p.row_parts;
    const int head = rest % p.h.kv_heads;
    if (warp == C::LOAD_WARP) {
        const AttnWork w = attn_find<false>(p.s, p.tiles - 1 - rest / p.h.kv_heads, p.h.tokens, lane);
        if (lane == 0) *shared_work = w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch();
    const uint32_t tmem = *tmem_slot;
    const AttnWork w = *shared_work;
    const int b0 = part * p.row_blocks;  // the first block of this part
    int blocks = attn_row_blocks(p, w) - b0;
    blocks = blocks < 0 ? 0 : blocks < p.row_blocks ? blocks : p.row_blocks;
    const int tail = w.lk - (b0 + blocks - 1) * ATTN_KEYS;  // keys of the sequence from the last block on
    const bool fix = blocks > 0 && tail < ATTN_KEYS;
    // Item 2n is block n's keys, 2n + 1 its values.
    auto slot = [&](int it) -> int { return it & 1 ? C::KS + (it >> 1) % C::VS : (it >> 1) % C::KS; };
    auto tile = [&](int it) -> int { return C::KV_OFF + slot(it) * C::TILE_BYTES; };
    auto parity = [&](int it) -> uint32_t {
        return (uint32_t)(it & 1 ? (it >> 1) / C::VS : (it >> 1) / C::KS) & 1;
    };
    // Where item `it`'s loads report: a last block that ends inside reports to
    // ROWS_WARP, which passes it on once the rest is zero.
    auto landed = [&](int it) -> uint32_t {
        return bar(fix && (it >> 1) == blocks - 1 ? C::LAST + (it & 1) : C::FULL0 + slot(it));
    };

    if (warp == C::LOAD_WARP) {
        if (blocks > 0 && elect_one()) {
            mbar_arrive_expect_tx(bar(C::QF), 2 * C::HALVES * p.h.tokens * p.h.group * 128);
#pragma unroll
            for (int h = 0; h < C::HALVES; ++h) {
                tma_load_4d(sbase + C::Q_OFF + h * 16384, &p.q, bar(C::QF), h * 64, 0, head, w.q0 + w.first);
                tma_load_4d(sbase + C::DY_OFF + h * 16384, &p.dy, bar(C::QF), h * 64, 0, head, w.q0 + w.first);
            }
            int issued = 0;
            bool ok = true;
            for (int it = 0; it < 2 * blocks; ++it) {
                if (!wait_phase(bar(C::EMPTY0 + slot(it)), parity(it) ^ 1, ctl, SITE_EMPTY)) { ok = false; break; }
                mbar_arrive_expect_tx(landed(it), C::TILE_BYTES);
#pragma unroll
                for (int h = 0; h < C::HALVES; ++h)
                    tma_load_3d(sbase + tile(it) + h * 16384, it & 1 ? &p.v : &p.k, landed(it), h * 64,
                                head, w.k0 + (b0 + (it >> 1)) * ATTN_KEYS);
                ++issued;
            }
            if (!ok) {
                wait_phase_drain(bar(C::QF), 0, ctl);
                for (int it = issued > 2 * C::KS ? issued - 2 * C::KS : 0; it < issued; ++it)
                    if (it + 2 * (it & 1 ? C::VS : C::KS) >= issued)
                        wait_phase_drain(landed(it), fix && (it >> 1) == blocks - 1 ? 0 : parity(it), ctl);
            }
        }
        __syncwarp();
    } else if (warp == C::MMA_WARP || warp == C::MMA2_WARP) {
        // Two threads: one for S, a block ahead, one for dP and dQ.
        const bool first = warp == C::MMA_WARP;
        if (blocks > 0 && elect_one()) {
            auto full = [&](int it) -> bool {
                const bool ok = wait_phase(bar(C::FULL0 + slot(it)), parity(it), ctl, SITE_FULL);
                tc_fence_after();
                return ok;
            };
            bool ok = wait_phase(bar(C::QF), 0, ctl, SITE_FULL);
            if (first) {
                for (int n = 0; ok && n < blocks; ++n) {
                    // (once the warps hold the scores of the block before)
                    ok = full(2 * n) && (n == 0 || wait_phase(bar(C::SE), (n - 1) & 1, ctl, SITE_PROBABILITIES));
                    if (!ok) break;
                    tc_fence_after();
                    attn_mma_rows<0, DT / 16>(tmem + C::S_COL, sbase + C::Q_OFF, sbase + tile(2 * n), C::ID_S);
                    mma_commit(bar(C::SF));
                }
            } else {
                for (int n = 0; ok && n <= blocks; ++n) {
                    if (n < blocks) ok = full(2 * n + 1);
                    if (ok && n > 0) ok = wait_phase(bar(C::DSR), (n - 1) & 1, ctl, SITE_PROBABILITIES);
                    if (!ok) break;
                    tc_fence_after();
                    if (n < blocks) {
                        attn_mma_rows<0, DT / 16>(tmem + C::DP_COL, sbase + C::DY_OFF, sbase + tile(2 * n + 1), C::ID_S);
                        mma_commit(bar(C::DPF));
                        mma_commit(bar(C::EMPTY0 + slot(2 * n + 1)));
                    }
                    if (n > 0) {
                        const int m = n - 1;
                        attn_mma_ta<0, 8, 32>(tmem + C::DQ_COL, tmem + C::DS_COL + (m & 1) * 64, sbase + tile(2 * m),
                                              C::ID_PV, m > 0);
                        mma_commit(bar(C::EMPTY0 + slot(2 * m)));
                    }
                }
            }
            if (!ok || !first) {
                const uint32_t end = bar(ok ? C::OD : C::DRAIN + (first ? 0 : 1));
                mma_commit(end);
                if (!ok) wait_phase_drain(end, 0, ctl);
            }
        }
        __syncwarp();
    } else if (warp == C::ROWS_WARP) {
        // Keys and values behind the sequence's end become zero.
        for (int i = 0; fix && i < 2; ++i) {
            const int it = 2 * (blocks - 1) + i;
            if (!wait_warp(bar(C::LAST + i), 0, ctl, SITE_FULL)) break;
            for (int row = tail + lane; row < ATTN_KEYS; row += 32) attn_zero_row<C::HALVES>(smem + tile(it), row);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::FULL0 + slot(it)));
        }
        __syncwarp();
    } else if (w.seq >= 0) {
        // ------------------------------------------------------ a row a thread, 64 keys of a block
        const int half = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lane_base = (uint32_t)(warp & 3) << 21;
        const int token = w.first + row / p.h.group, qh = head * p.h.group + row % p.h.group;
        const bool valid = row < p.h.tokens * p.h.group && token < w.lq;
        const int seen = valid ? attn_seen(p.s, w, token) : 0;
        const int first_seen = attn_seen(p.s, w, w.first);
        float lse = -INFINITY, delta = 0.0f;
        if (valid) {
            const int64_t at = (int64_t)qh * p.s.q_rows + w.q0 + token;
            const float z = p.lse[at];
            if (z != -INFINITY) lse = -z * 1.4426950408889634f;
            delta = -p.delta[at];
        }
        const uint64_t cc = pair2(p.h.scale_log2, p.h.scale_log2), ll = pair2(lse, lse), dd = pair2(delta, delta);
        bool ok = true;
        for (int n = 0; n < blocks; ++n) {
            ok = wait_warp(bar(C::SF), n & 1, ctl, SITE_SCORES);
            if (!ok) break;
            tc_fence_after();
            float y[64];
            uint32_t *yw = reinterpret_cast<uint32_t *>(y);
#pragma unroll
            for (int i = 0; i < 2; ++i) tmem_ld_row32(tmem + lane_base + C::S_COL + 64 * half + 32 * i, yw + 32 * i);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::SE));
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
                unpair2(fma_pair(pair2(y[i], y[i + 1]), cc, ll), y[i], y[i + 1]);
                y[i] = exp2_approx(y[i]);
                y[i + 1] = exp2_approx(y[i + 1]);
            }
            if ((b0 + n + 1) * ATTN_KEYS > first_seen) {
                const int lim = seen - (b0 + n) * ATTN_KEYS - 64 * half;
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    if (i >= lim) y[i] = 0.0f;
            }
            ok = wait_warp(bar(C::DPF), n & 1, ctl, SITE_SCORES);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < 64; i += 32) {
                uint32_t d[32];
                tmem_ld_row32(tmem + lane_base + C::DP_COL + 64 * half + i, d);
                tmem_ld_wait();
                const float *f = reinterpret_cast<const float *>(d);
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    unpair2(mul_pair(pair2(y[i + e], y[i + e + 1]), add_pair(pair2(f[e], f[e + 1]), dd)), y[i + e],
                            y[i + e + 1]);
            }
            attn_store_half<KD>(tmem + lane_base + C::DS_COL + (n & 1) * 64 + 32 * half, y);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::DSR));
        }
        if (ok && blocks > 0) {
            ok = wait_warp(bar(C::OD), 0, ctl, SITE_ACC_FULL);
            tc_fence_after();
        }
        const uint32_t at = tmem + lane_base + C::DQ_COL + half * (DT / 2);
        const int left = p.h.dim - half * (DT / 2);
        if (ok && p.row_parts == 1)
            attn_store_row<KD, DT / 2>(at, blocks > 0, blocks > 0, p.h.scale, valid, left,
                                       static_cast<uint16_t *>(p.dq.ptr) + (w.q0 + (int64_t)token) * p.dq.ld +
                                           qh * p.dq.hd + half * (DT / 2));
        else if (ok && blocks > 0)
            attn_store_part<DT / 2>(at, valid, left,
                                    p.part_rows + (((int64_t)part * p.h.heads + qh) * p.s.q_rows + w.q0 + token) *
                                                      p.h.dim + half * (DT / 2));
    }

    tc_fence_before();
    __syncthreads();
    if (warp == C::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// Both in one launch, the keys' CTAs (the longer work) first: the rows' fill in
// where the keys' run out.
template <Kind KD, int DT>
__global__ void __launch_bounds__(AttnBackConfig<KD, DT>::NUM_THREADS, 1)
    tg_attn_backward_kernel(const __grid_constant__ AttnBackward p) {
    if ((int)blockIdx.x < p.key_ctas) attn_keys<KD, DT>(p, blockIdx.x);
    else attn_rows<KD, DT>(p, blockIdx.x - p.key_ctas);
}

// The parts' sums, in their order: a warp a row, its lanes four values each.
// blockIdx.x: the key blocks first (when they have parts), then the row tiles.
constexpr int PARTS_THREADS = 256;
template <Kind KD>
__global__ void __launch_bounds__(PARTS_THREADS) tg_attn_parts_kernel(const __grid_constant__ AttnBackward p) {
    griddep_launch();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int key_blocks = p.key_parts > 1 ? p.blocks * p.h.kv_heads : 0;
    const bool keys = (int)blockIdx.x < key_blocks;
    const int block = keys ? blockIdx.x : blockIdx.x - key_blocks;
    const int head = block % p.h.kv_heads;
    const AttnWork w = keys ? attn_find<true>(p.s, block / p.h.kv_heads, ATTN_KEYS, lane)
                            : attn_find<false>(p.s, block / p.h.kv_heads, p.h.tokens, lane);
    if (w.seq < 0) return;
    int i0, parts;
    if (keys) parts = (attn_key_tiles(p, w, i0) + p.key_tiles - 1) / p.key_tiles;
    else parts = (attn_row_blocks(p, w) + p.row_blocks - 1) / p.row_blocks;
    const int rows = keys ? 2 * ATTN_KEYS : p.h.tokens * p.h.group;
    for (int i = blockIdx.y * (PARTS_THREADS / 32) + warp; i < rows; i += gridDim.y * (PARTS_THREADS / 32)) {
        const float *src;
        uint16_t *dst;
        int64_t step;
        float f = 1.0f;
        if (keys) {
            const int half = i & 1, key = w.first + (i >> 1);
            const AttnOut &out = half ? p.dk : p.dv;
            if (key >= w.lk || !out.ptr) continue;
            step = (int64_t)2 * p.h.kv_heads * p.s.k_rows * p.h.dim;
            src = p.part_keys + (((int64_t)half * p.h.kv_heads + head) * p.s.k_rows + w.k0 + key) * p.h.dim;
            dst = static_cast<uint16_t *>(out.ptr) + (w.k0 + (int64_t)key) * out.ld + head * out.hd;
            if (half) f = p.h.scale;
        } else {
            const int token = w.first + i / p.h.group, qh = head * p.h.group + i % p.h.group;
            if (token >= w.lq) break;
            step = (int64_t)p.h.heads * p.s.q_rows * p.h.dim;
            src = p.part_rows + ((int64_t)qh * p.s.q_rows + w.q0 + token) * p.h.dim;
            dst = static_cast<uint16_t *>(p.dq.ptr) + (w.q0 + (int64_t)token) * p.dq.ld + qh * p.dq.hd;
            f = p.h.scale;
        }
        if (4 * lane >= p.h.dim) continue;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int q = 0; q < parts; ++q) {
            const float4 v = reinterpret_cast<const float4 *>(src + q * step)[lane];
            a.x += v.x;
            a.y += v.y;
            a.z += v.z;
            a.w += v.w;
        }
        *reinterpret_cast<uint2 *>(dst + 4 * lane) =
            make_uint2(pack_half2<KD>(a.x * f, a.y * f), pack_half2<KD>(a.z * f, a.w * f));
    }
}

}  // namespace tg
