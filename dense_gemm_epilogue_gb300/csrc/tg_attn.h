// Internal interface between the attention front end (tg_attn.cu) and the
// kernel instantiations (one translation unit per operand type), and what both
// sides of the ABI share about packed sequences.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace tg {

constexpr int ATTN_ROWS = 128;  // rows of a tile: tokens x heads of one group
constexpr int ATTN_KEYS = 128;  // keys of a block
constexpr int ATTN_MAX_DIM = 128;

// Rows of the last of `tiles` row tiles that begin at token i0 of a sequence of lq.  (Held
// to a tile's tokens before the product: the tiles may be one part of the sequence's, and
// what is left of 2^31 rows, times a group of 128, is more than 32 bits hold.)
__host__ __device__ inline int attn_tail_rows(int lq, int i0, int tiles, int tokens, int group) {
    const int left = lq - i0 - (tiles - 1) * tokens;
    return (left < tokens ? left : tokens) * group;
}

// Packed sequences: sequence s owns rows starts[s] to starts[s] + length[s] (or
// starts[s + 1] when no lengths are given) of Q, and of K and V.
struct AttnSeqs {
    const int64_t *q_starts, *q_lengths, *k_starts, *k_lengths;
    int32_t seqs;
    int32_t q_rows, k_rows;  // rows of the tensors
    int32_t max_q, max_k;    // no sequence is longer
    int32_t causal;
};

struct AttnHeads {
    int32_t heads, kv_heads, group;  // group: query heads that share a key head
    int32_t tokens;                  // tokens of a tile: ATTN_ROWS / group
    int32_t dim;
    float scale, scale_log2;         // scale, scale log2 e
};

struct AttnOut {
    void *ptr;
    int64_t ld, hd;  // elements between rows, between heads
};

struct AttnForward {
    CUtensorMap q, k, v;
    AttnSeqs s;
    AttnHeads h;
    AttnOut o;
    float *lse;             // heads x q_rows, or NULL
    float *part_o;          // splits > 1: unnormalised rows, splits x heads x q_rows x dim
    float2 *part_ml;        //   and their (reference exponent, sum)
    int32_t tiles;          // bound on the row tiles (tile pairs) of all sequences
    int32_t splits, chunk;  // key ranges of `chunk` blocks each
    int32_t join_tokens;    // tokens of a CTA's tiles
    int32_t join_rows;      // rows of these that a sequence can have, at most
    uint32_t *status;
    uint64_t wait_limit_ns;
};

constexpr int DELTA_THREADS = 256;
struct AttnDelta {
    const void *o, *dy;
    int64_t ldo, ho, lddy, hdy;
    float *delta;  // heads x rows
    int32_t rows, heads, dim;
};

struct AttnBackward {
    CUtensorMap q, k, v, dy;
    AttnSeqs s;
    AttnHeads h;
    AttnOut dq, dk, dv;     // (NULL pointers: not wanted)
    const float *lse;       // heads x q_rows
    const float *delta;     // heads x q_rows: sum over d of dO O
    int32_t tiles, blocks;  // bounds on the row tiles and on the key blocks of all sequences
    int32_t key_ctas;       // CTAs that work on keys; the rest work on rows
    // A key block's row tiles, and a row tile's key blocks, in so many parts of so many
    // tiles (blocks) each, one a CTA.  With several, FP32 sums go to the workspace:
    // (part, dV or dK, key head, key) and (part, query head, row), dim values each.
    int32_t key_parts, key_tiles, row_parts, row_blocks;
    float *part_keys, *part_rows;
    uint32_t *status;
    uint64_t wait_limit_ns;
};

cudaError_t launch_attn_forward_bf16(const AttnForward &a, int tiles_per_cta, int device, cudaStream_t stream);
cudaError_t launch_attn_forward_fp16(const AttnForward &a, int tiles_per_cta, int device, cudaStream_t stream);
// delta, then the gradients that are wanted.
cudaError_t launch_attn_backward_bf16(const AttnBackward &a, const AttnDelta &d, int device, cudaStream_t stream);
cudaError_t launch_attn_backward_fp16(const AttnBackward &a, const AttnDelta &d, int device, cudaStream_t stream);

}  // namespace tg
