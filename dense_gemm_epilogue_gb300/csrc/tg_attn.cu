// Attention over packed sequences: entry points, argument checks and planner
// (kernels: tg_kernel_attn.cuh).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdio>
#include <mutex>

#include "../../include/tg_gemm.h"
#include "tg_attn.h"
#include "tg_host.h"

namespace {

using namespace tg;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kMaxRows = (int64_t)INT32_MAX - 512;
constexpr double kLog2E = 1.4426950408889634;

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &qr) == cudaSuccess &&
            qr == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// A rows x heads x dim tensor of 16-bit values.
struct Heads {
    const void *ptr;
    int64_t ld, hd;
};

bool heads_ok(const Heads &x, int64_t heads, int64_t dim) {
    if (!x.ptr || (uintptr_t)x.ptr % 16) return false;
    if (x.ld < dim || x.ld % 8 || x.ld >= ((int64_t)1 << 38)) return false;
    return heads == 1 || (x.hd >= dim && x.hd % 8 == 0 && x.hd < ((int64_t)1 << 38) / heads);
}

// An output's rows and heads may not run into each other: heads lie within a row, or
// rows within a head.
bool apart(const Heads &x, int64_t rows, int64_t heads, int64_t dim) {
    return heads == 1 || rows <= 1 || x.ld >= (heads - 1) * x.hd + dim || x.hd >= (rows - 1) * x.ld + dim;
}

// Tensor map (dim, group, heads / group, rows) of the query side, a box of 64 values x
// group x 1 x box_rows; zeros outside.
bool encode_query(CUtensorMap *map, tg_dtype t, const Heads &x, int64_t rows, int64_t heads,
                  int64_t group, int64_t dim, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const int64_t hd = heads == 1 ? x.ld : x.hd;
    cuuint64_t dims[4] = {(cuuint64_t)dim, (cuuint64_t)group, (cuuint64_t)(heads / group), (cuuint64_t)rows};
    cuuint64_t strides[3] = {(cuuint64_t)(2 * hd), (cuuint64_t)(2 * hd * group), (cuuint64_t)(2 * x.ld)};
    cuuint32_t box[4] = {64, (cuuint32_t)group, 1, (cuuint32_t)box_rows};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(map, t == TG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
              const_cast<void *>(x.ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Tensor map (dim, heads, rows) of keys or values, a box of 64 values x 1 x ATTN_KEYS.
bool encode_keys(CUtensorMap *map, tg_dtype t, const Heads &x, int64_t rows, int64_t heads, int64_t dim) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const int64_t hd = heads == 1 ? x.ld : x.hd;
    cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)(2 * hd), (cuuint64_t)(2 * x.ld)};
    cuuint32_t box[3] = {64, 1, ATTN_KEYS};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, t == TG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void *>(x.ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The sizes that every call and workspace query takes.
struct Sizes {
    int64_t seqs, q_rows, k_rows, heads, kv_heads, dim, max_q, max_k;
    tg_dtype dtype;
};

tg_status sizes_ok(const Sizes &z) {
    if (z.seqs < 0 || z.q_rows < 0 || z.k_rows < 0 || z.max_q < 0 || z.max_k < 0) return TG_ERR_INVALID_VALUE;
    if (z.seqs > INT32_MAX / 2 || z.q_rows > kMaxRows || z.k_rows > kMaxRows) return TG_ERR_INVALID_VALUE;
    if (z.heads < 1 || z.kv_heads < 1 || z.heads % z.kv_heads || z.dim < 1) return TG_ERR_INVALID_VALUE;
    if (z.heads > 65536) return TG_ERR_INVALID_VALUE;
    if (z.dtype != TG_BF16 && z.dtype != TG_FP16) return TG_ERR_INVALID_VALUE;
    if (z.dim % 8 || z.dim > ATTN_MAX_DIM || z.heads / z.kv_heads > ATTN_ROWS) return TG_ERR_UNSUPPORTED;
    return TG_OK;
}

int64_t bound_of(int64_t given, int64_t rows) { return given == 0 || given > rows ? rows : given; }

// Tiles of `per` rows that the sequences can have, at most.
int64_t tile_bound(int64_t seqs, int64_t rows, int64_t longest, int64_t per) {
    if (longest <= per) return seqs;
    const int64_t a = seqs * ceil_div(longest, per), b = rows / per + seqs;
    return a < b ? a : b;
}

struct ForwardPlan {
    int nq;           // row tiles a CTA
    int64_t tiles;    // of nq row tiles each
    int64_t splits, chunk;
    int64_t workspace;
};

// The choice with the least estimated time, in cycles: CTAs of one or two row tiles,
// one an SM at a time, over key ranges of `chunk` blocks; a round of a block takes
// 2000 cycles with one tile (its chain: S, softmax, P V), 2700 with two; a CTA's start
// and end 7000; ranges cost a second kernel and their rows' way through memory.
// Several sequences may be of very different lengths, of which max_k says nothing, so
// ranges are of 16 blocks at most there, for an even load (32 single tokens over 355
// to 11800 keys: 91 us; 24 blocks 94, 48 blocks 101; one over 131072: 88.5 in one
// round of CTAs over 54 blocks each, 99 over 16 each).
tg_status plan_forward(const Sizes &z, int sms, ForwardPlan *plan) {
    ForwardPlan &best = *plan = {};
    const int64_t tokens = ATTN_ROWS / (z.heads / z.kv_heads);
    const int64_t max_q = bound_of(z.max_q, z.q_rows), max_k = bound_of(z.max_k, z.k_rows);
    const int64_t blocks = ceil_div(max_k, ATTN_KEYS) > 0 ? ceil_div(max_k, ATTN_KEYS) : 1;
    double least = -1.0;
    for (int nq = 1; nq <= (max_q > tokens ? 2 : 1); ++nq) {
        const int64_t tiles = tile_bound(z.seqs, z.q_rows, max_q, nq * tokens);
        const int64_t ctas = tiles * z.kv_heads;
        int64_t most = ctas < 2 * sms ? ceil_div(2 * sms, ctas > 0 ? ctas : 1) : 1;
        const bool uneven = z.seqs > 1 && max_q <= tokens;
        if (uneven && most < ceil_div(blocks, 16)) most = ceil_div(blocks, 16);
        if (most > ceil_div(blocks, 4)) most = ceil_div(blocks, 4);
        for (int64_t s = 1; s <= most; ++s) {
            const int64_t chunk = ceil_div(blocks, s), splits = ceil_div(blocks, chunk);
            if (splits != s) continue;
            if (ctas > INT32_MAX / splits) break;  // more pieces than a grid
            const double waves = (double)ceil_div(ctas * splits, sms);
            double cycles = waves * (7000.0 + chunk * (nq == 2 ? 2700.0 : 2000.0));
            if (splits > 1) cycles += 6000.0 + 8.0 * splits * z.heads * z.q_rows * z.dim / 2500.0;
            if (uneven && chunk > 16) cycles *= 1.0 + (chunk - 16) / 8.0;
            if (least >= 0.0 && cycles >= least) continue;
            least = cycles;
            best.nq = nq;
            best.tiles = tiles;
            best.splits = splits;
            best.chunk = chunk;
        }
    }
    if (least < 0.0) return TG_ERR_UNSUPPORTED;
    if (best.splits > 1) {
        if ((double)best.splits * z.heads * z.q_rows * (4 * z.dim + 8) > 4e18) return TG_ERR_UNSUPPORTED;
        best.workspace = best.splits * z.heads * z.q_rows * (4 * z.dim + 8);
    }
    return TG_OK;
}

struct BackwardPlan {
    int64_t tiles, blocks;  // row tiles and key blocks of all sequences, at most
    int64_t key_parts, key_tiles, row_parts, row_blocks;
    int64_t delta, part_keys, part_rows;  // workspace bytes, in this order
    int64_t workspace() const { return delta + part_keys + part_rows; }
};

// The longest sequence's key block sees all its row tiles, and a CTA takes them one
// after the other.  Where that is much longer than the whole work shared by all SMs
// (few key heads, one long sequence among short ones) the tiles are cut into parts for
// as many CTAs, and likewise a row tile's key blocks; another kernel adds the parts'
// FP32 sums in order, at about 24000 cycles with what the parts write.  (Cycles a tile:
// 128-wide heads 2700 for keys, 1700 for rows; 64-wide 2000 and 1100.  2048 rows of
// 8 heads over one key head: 198 us whole, 63 in parts; 64 rows over 8192 keys 91 and
// 57; 309 rows of 3 heads, 8 tiles, 22 whole, 25 and 28 in 2 and 8 parts.)
tg_status plan_backward(const Sizes &z, int sms, BackwardPlan *plan) {
    BackwardPlan &p = *plan = {};
    const int64_t group = z.heads / z.kv_heads, tokens = ATTN_ROWS / group;
    const int64_t max_q = bound_of(z.max_q, z.q_rows), max_k = bound_of(z.max_k, z.k_rows);
    p.tiles = z.q_rows ? tile_bound(z.seqs, z.q_rows, max_q, tokens) : 0;
    p.blocks = z.k_rows ? tile_bound(z.seqs, z.k_rows, max_k, ATTN_KEYS) : 0;
    p.delta = ceil_div(4 * z.heads * z.q_rows, 16) * 16;
    const int64_t long_tiles = ceil_div(max_q, tokens), long_blocks = ceil_div(max_k, ATTN_KEYS);
    p.key_parts = p.row_parts = 1;
    p.key_tiles = long_tiles > 0 ? long_tiles : 1;
    p.row_blocks = long_blocks > 0 ? long_blocks : 1;
    const double all_tiles = (double)z.q_rows / tokens;                            // of all sequences
    const double mean_blocks = 0.5 + (double)z.k_rows / ((double)z.seqs * ATTN_KEYS);  // of one
    const double key_cycles = z.dim > 64 ? 2700.0 : 2000.0, row_cycles = z.dim > 64 ? 1700.0 : 1100.0;
    const double share = all_tiles * mean_blocks * z.kv_heads * (key_cycles + row_cycles) / sms;
    auto cut = [&](int64_t most, double cycles, int64_t &parts, int64_t &each) {
        double least = most * cycles > share ? most * cycles : share;
        for (int64_t n = 2; n <= 16 && n <= most; ++n) {
            const int64_t e = ceil_div(most, n);
            const double t = (e * cycles > share ? e * cycles : share) + 24000.0 + 500.0 * n;
            if (t >= least) continue;
            least = t;
            each = e;
            parts = ceil_div(most, e);
        }
    };
    cut(long_tiles, key_cycles, p.key_parts, p.key_tiles);
    cut(long_blocks, row_cycles, p.row_parts, p.row_blocks);
    if (p.key_parts > 1) p.part_keys = 8 * p.key_parts * z.k_rows * z.kv_heads * z.dim;
    if (p.row_parts > 1) p.part_rows = 4 * p.row_parts * z.q_rows * z.heads * z.dim;
    const int64_t ctas = (p.tiles * p.row_parts + p.blocks * p.key_parts) * z.kv_heads;
    return ctas > INT32_MAX || z.q_rows * z.heads / 16 > INT32_MAX - 1 ? TG_ERR_UNSUPPORTED : TG_OK;
}

bool arrays_ok(const int64_t *qs, const int64_t *ql, const int64_t *ks, const int64_t *kl) {
    return qs && ks && !(((uintptr_t)qs | (uintptr_t)ql | (uintptr_t)ks | (uintptr_t)kl) % 8);
}
bool f32_ok(const void *p) { return (uintptr_t)p % 4 == 0; }

AttnHeads make_heads(const Sizes &z, float scale) {
    AttnHeads h = {};
    h.heads = (int32_t)z.heads;
    h.kv_heads = (int32_t)z.kv_heads;
    h.group = (int32_t)(z.heads / z.kv_heads);
    h.tokens = ATTN_ROWS / h.group;
    h.dim = (int32_t)z.dim;
    h.scale = scale;
    h.scale_log2 = (float)((double)scale * kLog2E);
    return h;
}

AttnSeqs make_seqs(const Sizes &z, const int64_t *qs, const int64_t *ql, const int64_t *ks,
                   const int64_t *kl, int32_t causal) {
    AttnSeqs s = {};
    s.q_starts = qs;
    s.q_lengths = ql;
    s.k_starts = ks;
    s.k_lengths = kl;
    s.seqs = (int32_t)z.seqs;
    s.q_rows = (int32_t)z.q_rows;
    s.k_rows = (int32_t)z.k_rows;
    s.max_q = (int32_t)bound_of(z.max_q, z.q_rows);
    s.max_k = (int32_t)bound_of(z.max_k, z.k_rows);
    s.causal = causal;
    return s;
}

bool scale_ok(float s) { return s > 0.0f && std::isfinite(s * (float)kLog2E); }

}  // namespace

extern "C" int64_t tg_attention_workspace_bytes(int64_t seqs, int64_t q_rows, int64_t k_rows,
                                                int64_t heads, int64_t kv_heads, int64_t dim,
                                                int64_t max_q, int64_t max_k, tg_dtype dtype) {
    const Sizes z = {seqs, q_rows, k_rows, heads, kv_heads, dim, max_q, max_k, dtype};
    if (sizes_ok(z) != TG_OK) return -1;
    tg::host::Device dev;
    if (tg::host::device(&dev) != TG_OK) return -1;
    if (seqs == 0 || q_rows == 0) return 0;
    ForwardPlan p;
    return plan_forward(z, dev.sms, &p) == TG_OK ? p.workspace : -1;
}

extern "C" tg_status tg_attention_plan_describe(int64_t seqs, int64_t q_rows, int64_t k_rows, int64_t heads,
                                                int64_t kv_heads, int64_t dim, int64_t max_q,
                                                int64_t max_k, tg_dtype dtype, int32_t num_sms, char *buf,
                                                size_t len) {
    const Sizes z = {seqs, q_rows, k_rows, heads, kv_heads, dim, max_q, max_k, dtype};
    tg_status st = sizes_ok(z);
    if (st != TG_OK) return st;
    if (!buf || len == 0) return TG_ERR_INVALID_VALUE;
    if (num_sms <= 0) {
        tg::host::Device dev;
        st = tg::host::device(&dev);
        if (st != TG_OK) return st;
        num_sms = dev.sms;
    }
    int n;
    if (seqs == 0 || q_rows == 0) {
        n = std::snprintf(buf, len, "empty");
    } else {
        ForwardPlan p;
        st = plan_forward(z, num_sms, &p);
        if (st != TG_OK) return st;
        n = std::snprintf(buf, len, "tiles=%d ctas=%lld ranges=%lld blocks=%lld", p.nq,
                          (long long)(p.tiles * kv_heads * p.splits), (long long)p.splits, (long long)p.chunk);
    }
    return n >= 0 && (size_t)n < len ? TG_OK : TG_ERR_INVALID_VALUE;
}

extern "C" tg_status tg_attention(int64_t seqs, int64_t q_rows, int64_t k_rows, int64_t heads,
                                  int64_t kv_heads, int64_t dim, const void *Q, int64_t ldq, int64_t hq,
                                  const void *K, int64_t ldk, int64_t hk, const void *V, int64_t ldv,
                                  int64_t hv, const int64_t *q_starts, const int64_t *q_lengths,
                                  const int64_t *k_starts, const int64_t *k_lengths, int64_t max_q,
                                  int64_t max_k, int32_t causal, float scale, void *O, int64_t ldo,
                                  int64_t ho, float *LSE, tg_dtype dtype, void *workspace,
                                  int64_t workspace_bytes, void *stream) {
    const Sizes z = {seqs, q_rows, k_rows, heads, kv_heads, dim, max_q, max_k, dtype};
    tg_status st = sizes_ok(z);
    if (st != TG_OK) return st;
    if (!scale_ok(scale) || (causal != 0 && causal != 1) || workspace_bytes < 0 || !f32_ok(LSE))
        return TG_ERR_INVALID_VALUE;
    if (seqs == 0 || q_rows == 0) return TG_OK;
    const Heads q = {Q, ldq, hq}, k = {K, ldk, hk}, v = {V, ldv, hv}, o = {O, ldo, ho};
    if (!heads_ok(q, heads, dim) || !heads_ok(o, heads, dim) || !apart(o, q_rows, heads, dim))
        return TG_ERR_INVALID_VALUE;
    if (k_rows > 0 && (!heads_ok(k, kv_heads, dim) || !heads_ok(v, kv_heads, dim))) return TG_ERR_INVALID_VALUE;
    if (!arrays_ok(q_starts, q_lengths, k_starts, k_lengths)) return TG_ERR_INVALID_VALUE;
    tg::host::Device dev;
    st = tg::host::device(&dev);
    if (st != TG_OK) return st;
    ForwardPlan p;
    st = plan_forward(z, dev.sms, &p);
    if (st != TG_OK) return st;
    if (p.workspace && (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < p.workspace))
        return TG_ERR_INVALID_VALUE;
    AttnForward a = {};
    a.s = make_seqs(z, q_starts, q_lengths, k_starts, k_lengths, causal);
    a.h = make_heads(z, scale);
    // (Without keys nothing is loaded: any map will do.)
    if (!encode_query(&a.q, dtype, q, q_rows, heads, a.h.group, dim, a.h.tokens) ||
        !encode_keys(&a.k, dtype, k_rows ? k : q, k_rows ? k_rows : 1, k_rows ? kv_heads : 1, dim) ||
        !encode_keys(&a.v, dtype, k_rows ? v : q, k_rows ? k_rows : 1, k_rows ? kv_heads : 1, dim))
        return TG_ERR_CUDA;
    a.o = {O, ldo, heads == 1 ? 0 : ho};
    a.lse = LSE;
    a.tiles = (int32_t)p.tiles;
    a.splits = (int32_t)p.splits;
    a.chunk = (int32_t)p.chunk;
    a.join_tokens = p.nq * a.h.tokens;
    a.join_rows = (a.s.max_q < a.join_tokens ? a.s.max_q : a.join_tokens) * a.h.group;
    if (p.workspace) {
        a.part_o = static_cast<float *>(workspace);
        a.part_ml = reinterpret_cast<float2 *>(a.part_o + p.splits * heads * q_rows * dim);
    }
    a.status = dev.status;
    a.wait_limit_ns = dev.wait_limit_ns;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == TG_BF16 ? launch_attn_forward_bf16(a, p.nq, dev.id, cs)
                                           : launch_attn_forward_fp16(a, p.nq, dev.id, cs);
    return e == cudaSuccess ? TG_OK : TG_ERR_CUDA;
}

extern "C" int64_t tg_attention_backward_workspace_bytes(int64_t seqs, int64_t q_rows, int64_t k_rows,
                                                         int64_t heads, int64_t kv_heads, int64_t dim,
                                                         int64_t max_q, int64_t max_k, tg_dtype dtype) {
    const Sizes z = {seqs, q_rows, k_rows, heads, kv_heads, dim, max_q, max_k, dtype};
    if (sizes_ok(z) != TG_OK) return -1;
    if (seqs == 0) return 0;
    tg::host::Device dev;
    if (tg::host::device(&dev) != TG_OK) return -1;
    BackwardPlan p;
    return plan_backward(z, dev.sms, &p) == TG_OK ? p.workspace() : -1;
}

extern "C" tg_status tg_attention_backward(
    int64_t seqs, int64_t q_rows, int64_t k_rows, int64_t heads, int64_t kv_heads, int64_t dim,
    const void *Q, int64_t ldq, int64_t hq, const void *K, int64_t ldk, int64_t hk, const void *V,
    int64_t ldv, int64_t hv, const void *O, int64_t ldo, int64_t ho, const void *dO, int64_t lddo,
    int64_t hdo, const float *LSE, const int64_t *q_starts, const int64_t *q_lengths,
    const int64_t *k_starts, const int64_t *k_lengths, int64_t max_q, int64_t max_k, int32_t causal,
    float scale, void *dQ, int64_t lddq, int64_t hdq, void *dK, int64_t lddk, int64_t hdk, void *dV,
    int64_t lddv, int64_t hdv, tg_dtype dtype, void *workspace, int64_t workspace_bytes, void *stream) {
    const Sizes z = {seqs, q_rows, k_rows, heads, kv_heads, dim, max_q, max_k, dtype};
    tg_status st = sizes_ok(z);
    if (st != TG_OK) return st;
    if (!scale_ok(scale) || (causal != 0 && causal != 1) || workspace_bytes < 0 || !f32_ok(LSE))
        return TG_ERR_INVALID_VALUE;
    if (seqs == 0 || (!dQ && !dK && !dV)) return TG_OK;
    const Heads q = {Q, ldq, hq}, k = {K, ldk, hk}, v = {V, ldv, hv}, o = {O, ldo, ho}, dy = {dO, lddo, hdo};
    const Heads dq = {dQ, lddq, hdq}, dk = {dK, lddk, hdk}, dv = {dV, lddv, hdv};
    if (q_rows > 0 && (!heads_ok(q, heads, dim) || !heads_ok(o, heads, dim) || !heads_ok(dy, heads, dim) || !LSE ||
                       (dQ && (!heads_ok(dq, heads, dim) || !apart(dq, q_rows, heads, dim)))))
        return TG_ERR_INVALID_VALUE;
    if (k_rows > 0 && (!heads_ok(k, kv_heads, dim) || !heads_ok(v, kv_heads, dim) ||
                       (dK && (!heads_ok(dk, kv_heads, dim) || !apart(dk, k_rows, kv_heads, dim))) ||
                       (dV && (!heads_ok(dv, kv_heads, dim) || !apart(dv, k_rows, kv_heads, dim)))))
        return TG_ERR_INVALID_VALUE;
    if (!arrays_ok(q_starts, q_lengths, k_starts, k_lengths)) return TG_ERR_INVALID_VALUE;
    if (q_rows == 0 && k_rows == 0) return TG_OK;
    if (q_rows && (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < 4 * heads * q_rows))
        return TG_ERR_INVALID_VALUE;
    tg::host::Device dev;
    st = tg::host::device(&dev);
    if (st != TG_OK) return st;
    BackwardPlan plan;
    st = plan_backward(z, dev.sms, &plan);
    if (st != TG_OK) return st;
    if (plan.workspace() && (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < plan.workspace()))
        return TG_ERR_INVALID_VALUE;
    AttnBackward a = {};
    a.s = make_seqs(z, q_starts, q_lengths, k_starts, k_lengths, causal);
    a.h = make_heads(z, scale);
    // (A side without rows is not loaded: any map will do.)
    const Heads &any = q_rows ? q : k;
    const int64_t any_rows = 1, any_heads = 1;
    if (!encode_query(&a.q, dtype, q_rows ? q : any, q_rows ? q_rows : any_rows, q_rows ? heads : any_heads,
                      q_rows ? a.h.group : 1, dim, a.h.tokens) ||
        !encode_query(&a.dy, dtype, q_rows ? dy : any, q_rows ? q_rows : any_rows, q_rows ? heads : any_heads,
                      q_rows ? a.h.group : 1, dim, a.h.tokens) ||
        !encode_keys(&a.k, dtype, k_rows ? k : any, k_rows ? k_rows : any_rows, k_rows ? kv_heads : any_heads, dim) ||
        !encode_keys(&a.v, dtype, k_rows ? v : any, k_rows ? k_rows : any_rows, k_rows ? kv_heads : any_heads, dim))
        return TG_ERR_CUDA;
    a.dq = {q_rows ? dQ : nullptr, lddq, heads == 1 ? 0 : hdq};
    a.dk = {k_rows ? dK : nullptr, lddk, kv_heads == 1 ? 0 : hdk};
    a.dv = {k_rows ? dV : nullptr, lddv, kv_heads == 1 ? 0 : hdv};
    a.lse = LSE;
    a.delta = static_cast<const float *>(workspace);
    a.tiles = (int32_t)plan.tiles;
    a.blocks = (int32_t)plan.blocks;
    a.key_parts = a.dk.ptr || a.dv.ptr ? (int32_t)plan.key_parts : 1;
    a.key_tiles = (int32_t)plan.key_tiles;
    a.row_parts = a.dq.ptr ? (int32_t)plan.row_parts : 1;
    a.row_blocks = (int32_t)plan.row_blocks;
    uint8_t *space = static_cast<uint8_t *>(workspace);
    a.part_keys = reinterpret_cast<float *>(space + plan.delta);
    a.part_rows = reinterpret_cast<float *>(space + plan.delta + plan.part_keys);
    a.status = dev.status;
    a.wait_limit_ns = dev.wait_limit_ns;
    AttnDelta d = {};
    d.o = O;
    d.dy = dO;
    d.ldo = ldo;
    d.ho = heads == 1 ? 0 : ho;
    d.lddy = lddo;
    d.hdy = heads == 1 ? 0 : hdo;
    d.delta = static_cast<float *>(workspace);
    d.rows = (int32_t)q_rows;
    d.heads = (int32_t)heads;
    d.dim = (int32_t)dim;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == TG_BF16 ? launch_attn_backward_bf16(a, d, dev.id, cs)
                                           : launch_attn_backward_fp16(a, d, dev.id, cs);
    return e == cudaSuccess ? TG_OK : TG_ERR_CUDA;
}
