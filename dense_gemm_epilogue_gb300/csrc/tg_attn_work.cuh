// Which rows and keys a block of the attention kernels works on.
#pragma once

#include "tg_attn.h"
#include "tg_attn_ptx.cuh"

namespace tg {

// Codes of the attention kernels' bounded waits (beside WaitSite's).
enum AttnSite : uint32_t {
    SITE_SCORES = 12,         // scores in tensor memory
    SITE_PROBABILITIES = 13,  // probabilities (or gradients of scores) back from the warps
};

// wait_phase by a whole warp, with one answer for it.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const WaitCtl &c, uint32_t site) {
    return __all_sync(0xffffffffu, wait_phase(bar, parity, c, site));
}

// A sequence's rows, held inside the tensor and to the bound that the caller
// gave: whatever the arrays hold, nothing outside is touched.
__device__ __forceinline__ void attn_range(const int64_t *starts, const int64_t *lengths, int s,
                                           int rows, int bound, int &at, int &len) {
    const int64_t b = starts[s];
    const int64_t n = lengths ? lengths[s] : starts[s + 1] - b;
    const bool in = b >= 0 && b <= rows && n > 0;
    const int64_t left = in ? rows - b : 0;
    int64_t l = in ? n : 0;
    if (l > left) l = left;
    if (l > bound) l = bound;
    at = in ? (int)b : 0;
    len = (int)l;
}

struct AttnWork {
    int seq;    // -1: nothing
    int first;  // first token (or key) of the tile within the sequence
    int q0, lq, k0, lk;
    int head, split;  // (set by the kernels that need them; head < 0: no more work)
};

// Tile t, counted through the sequences in order, `per` tokens (or keys) each:
// called by a whole warp.  KEYS: tiles of keys instead of tokens.
template <bool KEYS>
__device__ __forceinline__ AttnWork attn_find(const AttnSeqs &s, int t, int per, int lane) {
    AttnWork w;
    w.seq = -1;
    w.first = w.q0 = w.lq = w.k0 = w.lk = 0;
    // One round of loads: every lane holds a sequence's ranges, the one found passes
    // its own to all.
    const bool one = (KEYS ? s.max_k : s.max_q) <= per;  // a sequence is a tile
    // (64 bits: the arrays may say anything, and every range may be the whole tensor)
    int64_t tile = 0, before = 0;
    for (int base = one ? t : 0; base < s.seqs; base += 32) {
        const int q = one ? t : base + lane;
        int q0 = 0, lq = 0, k0 = 0, lk = 0;
        if (q < s.seqs) {
            attn_range(s.q_starts, s.q_lengths, q, s.q_rows, s.max_q, q0, lq);
            attn_range(s.k_starts, s.k_lengths, q, s.k_rows, s.max_k, k0, lk);
        }
        int from = 0;
        if (!one) {
            const int64_t n = ((KEYS ? lk : lq) + (int64_t)per - 1) / per;
            int64_t sum = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            const unsigned who = __ballot_sync(0xffffffffu, t >= before + sum - n && t < before + sum);
            if (!who) {
                before += __shfl_sync(0xffffffffu, sum, 31);
                continue;
            }
            from = __ffs(who) - 1;
            tile = t - (before + __shfl_sync(0xffffffffu, sum - n, from));
        }
        w.seq = __shfl_sync(0xffffffffu, q, from);
        w.q0 = __shfl_sync(0xffffffffu, q0, from);
        w.lq = __shfl_sync(0xffffffffu, lq, from);
        w.k0 = __shfl_sync(0xffffffffu, k0, from);
        w.lk = __shfl_sync(0xffffffffu, lk, from);
        w.first = (int)(tile * per);  // (of a range that holds it: below 2^31)
        if (w.first >= (KEYS ? w.lk : w.lq)) w.seq = -1;
        break;
    }
    return w;
}

// Keys that token i of a sequence sees: 0 to this, less one.
__device__ __forceinline__ int attn_seen(const AttnSeqs &s, const AttnWork &w, int i) {
    if (!s.causal) return w.lk;
    const int n = i + w.lk - w.lq + 1;
    return n < 0 ? 0 : n < w.lk ? n : w.lk;
}

}  // namespace tg
