// Front end of the feed-forward operators (linear layer and gated unit,
// forward and backward): argument checks, the planner of their products, the
// row-wise kernels of the backward pass, and the entry points.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <cstring>

#include "../../include/tg_gemm.h"
#include "tg_host.h"
#include "tg_mlp.h"
#include "tg_rows.cuh"

namespace tg {

// ------------------------------------------------------------------ row-wise backward kernels

// LINEAR: dz = dy act'(z) (rounded to the operands' type: it is an operand of
// two tensor-core products) and, from the unrounded FP32 values, each block's
// column sums; without z, dz = dy (a repack to aligned rows, or the sums
// alone).  GATED: dg = dh u act'(g), du = dh act(g).
//
// Bound: memory (LINEAR reads 2 and writes 1, GATED reads 3 and writes 2
// values per element).  A warp takes 256 columns of a row, 16 bytes a lane;
// eight warps take rows r, r + 8, ... of the block's band, four rows in flight
// each.  The column sums of a band add up over its rows in registers, then over
// the eight warps in order.
struct ActParams {
    int64_t m, n;
    const void *dy, *z, *u;
    int64_t lddy, ldz, ldu;
    int32_t act;
    int32_t band;       // rows per block
    void *out0, *out1;  // dz, or dg and du (out0 NULL: sums only)
    int64_t ldo0, ldo1;
    float *partial;     // [gridDim.y][n] or NULL
};

// Eight values of a row: consecutive ones from column c (16 bytes), or with
// VEC false the values at c, c + 32, ... (c = the lane's first column).
template <class Ty, bool VEC>
struct ActRow {
    __device__ __forceinline__ static int first(int lane) { return VEC ? lane * 8 : lane; }
    __device__ __forceinline__ static int col(int lane, int i) { return VEC ? lane * 8 + i : lane + 32 * i; }
    // Any columns, bounds checked.
    __device__ __forceinline__ static void load(const typename Ty::T *row, int64_t c, int64_t n,
                                                float (&v)[8]) {
        constexpr int STEP = VEC ? 1 : 32;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + STEP * i < n ? Ty::up(row[c + STEP * i]) : 0.0f;
    }
    __device__ __forceinline__ static void store(typename Ty::T *row, int64_t c, int64_t n,
                                                 const float (&v)[8]) {
        if (VEC && c + 8 <= n) {
            row_store<Ty>(row, c, n, v);
            return;
        }
        constexpr int STEP = VEC ? 1 : 32;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + STEP * i < n) row[c + STEP * i] = Ty::down(v[i]);
    }
};

// One block's band.  INSIDE: 16-byte vectors that all lie inside the rows, so
// that the loads of FLY rows leave together; rows past the band load its last
// row again and are dropped.
template <class Ty, bool VEC, bool GATED, int ACT, bool INSIDE>
__device__ __forceinline__ void act_band(const ActParams &p, int64_t c, int64_t r0, int64_t r1,
                                         float (&s)[8]) {
    using T = typename Ty::T;
    using Row = ActRow<Ty, VEC>;
    const T *dy = static_cast<const T *>(p.dy), *z = static_cast<const T *>(p.z);
    const T *u = static_cast<const T *>(p.u);
    T *o0 = static_cast<T *>(p.out0), *o1 = static_cast<T *>(p.out1);
    constexpr bool READ_Z = GATED || ACT != MLP_NONE;
    constexpr int FLY = INSIDE ? 4 : 1;
    for (int64_t r = r0 + (threadIdx.x >> 5); r < r1; r += 8 * FLY) {
        uint4 vd[FLY], vz[FLY], vu[FLY];
        if constexpr (INSIDE) {
#pragma unroll
            for (int k = 0; k < FLY; ++k) {
                const int64_t rr = r + 8 * k < r1 ? r + 8 * k : r1 - 1;
                vd[k] = __ldcs(reinterpret_cast<const uint4 *>(dy + rr * p.lddy + c));
                if (READ_Z) vz[k] = __ldcs(reinterpret_cast<const uint4 *>(z + rr * p.ldz + c));
                if (GATED) vu[k] = __ldcs(reinterpret_cast<const uint4 *>(u + rr * p.ldu + c));
            }
        }
#pragma unroll
        for (int k = 0; k < FLY; ++k) {
            const int64_t rr = r + 8 * k;
            if (rr < r1) {
                float d[8], a[8], g[8];
                if constexpr (INSIDE) row_unpack<Ty>(vd[k], d);
                else Row::load(dy + rr * p.lddy, c, p.n, d);
                if constexpr (READ_Z) {
                    float y[8];
                    if constexpr (INSIDE) row_unpack<Ty>(vz[k], y);
                    else Row::load(z + rr * p.ldz, c, p.n, y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) mlp_act_grad<ACT>(y[i], a[i], g[i]);
                }
                if constexpr (GATED) {
                    float w[8];
                    if constexpr (INSIDE) row_unpack<Ty>(vu[k], w);
                    else Row::load(u + rr * p.ldu, c, p.n, w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        a[i] *= d[i];
                        d[i] *= w[i] * g[i];
                    }
                    Row::store(o0 + rr * p.ldo0, c, p.n, d);
                    Row::store(o1 + rr * p.ldo1, c, p.n, a);
                } else {
                    if constexpr (READ_Z) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) d[i] *= g[i];
                    }
                    if (o0) Row::store(o0 + rr * p.ldo0, c, p.n, d);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[i] += d[i];
                }
            }
        }
    }
}

template <class Ty, bool VEC, bool GATED>
__global__ void __launch_bounds__(256, 3) tg_act_backward_kernel(const ActParams p) {
    __shared__ float sums[GATED ? 1 : 8][GATED ? 1 : 256];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    griddep_launch();
    griddep_wait();
    const int64_t c0 = (int64_t)blockIdx.x * 256;
    const int64_t r0 = (int64_t)blockIdx.y * p.band;
    const int64_t r1 = r0 + p.band < p.m ? r0 + p.band : p.m;
    using Row = ActRow<Ty, VEC>;
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.0f;
    const int64_t c = c0 + Row::first(lane);
    const bool inside = VEC && c0 + 256 <= p.n;
    mlp_with_act(p.act, [&](auto act) {
        if (inside) act_band<Ty, VEC, GATED, act.value, VEC>(p, c, r0, r1, s);
        else act_band<Ty, VEC, GATED, act.value, false>(p, c, r0, r1, s);
    });
    if constexpr (!GATED) {
        if (!p.partial) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[warp][Row::col(lane, i)] = s[i];
        __syncthreads();
        const int64_t cc = c0 + threadIdx.x;
        if (cc < p.n) {
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < 8; ++w) t += sums[w][threadIdx.x];
            p.partial[(int64_t)blockIdx.y * p.n + cc] = t;
        }
    }
}

}  // namespace tg

namespace {

using namespace tg;
using host::Device;

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }

bool type_ok(tg_dtype t) { return t == TG_BF16 || t == TG_FP16; }
bool act_ok(tg_activation a) { return (int)a >= 0 && (int)a < MLP_ACTS; }
tg_out_dtype out_type(tg_dtype t) { return t == TG_BF16 ? TG_OUT_BF16 : TG_OUT_F16; }

constexpr int64_t kMaxDim = INT32_MAX - 512;  // tile coordinates stay inside 32 bits
bool dims_ok(int64_t m, int64_t n, int64_t k) {
    return m >= 0 && n >= 0 && k >= 0 && m <= kMaxDim && n <= kMaxDim && k <= kMaxDim;
}
// A rows x cols matrix of 2-byte elements: may be NULL only when empty.
bool mat_ok(const void *p, int64_t ld, int64_t rows, int64_t cols, int e = 2) {
    if (ld < cols || ld >= ((int64_t)1 << 36)) return false;
    return (p || rows == 0 || cols == 0) && (uintptr_t)p % e == 0;
}

// A row-major operand or output as the kernels take it.
struct Mat {
    const void *p;
    int64_t ld, rows, cols;
    int e;
};
Mat mat(const void *p, int64_t ld, int64_t rows, int64_t cols, int e = 2) {
    return {p, rows <= 1 && ((uintptr_t)p % 16 == 0) ? round8(cols) : ld, rows, cols, e};
}
// Rows that TMA and 16-byte accesses can address (a single row's stride is free).
bool aligned16(const Mat &a) { return (uintptr_t)a.p % 16 == 0 && (a.ld * a.e) % 16 == 0; }

// The caller's workspace, handed out in 256-byte steps.  With no base it only
// counts (the size queries).
struct Arena {
    uint8_t *base;
    int64_t used = 0;
    explicit Arena(void *b) : base(static_cast<uint8_t *>(b)) {}
    void *take(int64_t bytes) {
        void *p = base ? base + used : nullptr;
        used += (bytes + 255) / 256 * 256;
        return p;
    }
    // Room for a matrix repacked to aligned rows, when `a` needs that.
    Mat repacked(const Mat &a) {
        Mat b = a;
        b.ld = round8(a.cols);
        b.p = take(2 * b.ld * a.rows);
        return b;
    }
};
bool needs_repack(const Mat &a) { return a.rows > 0 && a.cols > 0 && !aligned16(a); }

// ------------------------------------------------------------------ launches

// Bands of the row-wise kernel: about eight blocks per SM in all, at least 32
// rows each (four per warp).
int64_t act_bands(int64_t m, int64_t n, int sms) {
    const int64_t gx = div_up(n, 256);
    int64_t bands = div_up((int64_t)sms * 8, gx);
    if (bands > div_up(m, 32)) bands = div_up(m, 32);
    return bands < 1 ? 1 : (bands > 65535 ? 65535 : bands);
}

template <bool GATED>
cudaError_t launch_act(tg_dtype t, ActParams p, int sms, cudaStream_t stream) {
    const int64_t bands = act_bands(p.m, p.n, sms);
    p.band = (int32_t)div_up(p.m, bands);
    auto al = [](const void *q, int64_t ld) { return (uintptr_t)q % 16 == 0 && ld % 8 == 0; };
    const bool vec = al(p.dy, p.lddy) && (!p.z || al(p.z, p.ldz)) && (!p.u || al(p.u, p.ldu));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)div_up(p.n, 256), (unsigned)div_up(p.m, p.band), 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (t == TG_BF16)
        return vec ? cudaLaunchKernelEx(&cfg, tg_act_backward_kernel<TypeBF16, true, GATED>, p)
                   : cudaLaunchKernelEx(&cfg, tg_act_backward_kernel<TypeBF16, false, GATED>, p);
    return vec ? cudaLaunchKernelEx(&cfg, tg_act_backward_kernel<TypeF16, true, GATED>, p)
               : cudaLaunchKernelEx(&cfg, tg_act_backward_kernel<TypeF16, false, GATED>, p);
}

// `from`, repacked into `to`'s aligned rows.
cudaError_t repack(tg_dtype t, const Mat &from, const Mat &to, int sms, cudaStream_t stream) {
    ActParams p = {};
    p.m = from.rows;
    p.n = from.cols;
    p.dy = from.p;
    p.lddy = from.ld;
    p.out0 = const_cast<void *>(to.p);
    p.ldo0 = to.ld;
    return launch_act<false>(t, p, sms, stream);
}

// One product of the CTA-pair kernel, in role space.
struct Product {
    MlpOp op;
    int64_t m, n;      // rows and columns of one output
    int64_t k[2];      // reduction length of each operand pair (second: 0 if none)
    int entries;
    Mat a[2], b[2];
    Mat out[3];
    bool out_f32;
    int act;
    const float *bias;
    Mat r;             // residual (p NULL: none)
};

struct TilePlan {
    int cg, block_n;
    int64_t tiles, tiles_per_entry;
    int grid, split_max, group;
    bool ticket;
};

// Times of the planner's cost model, in microseconds, measured on long and
// short products of each tile shape: one 64-deep K block of a team's tile; what
// its epilogue adds where nothing overlaps it; and what joining s segments adds
// to a split tile (FP32 partial sums written, then s - 1 of them read back).
// The 128-column tiles move 3/4 of the bytes per K block for half the work, so
// they pay only where they fill SMs that 256-column tiles leave idle.
struct TileCost {
    int cg, bn;
    double block, epilogue, join, join_part;
};
constexpr TileCost kTiles[] = {{2, 256, 0.350, 4.5, 5.0, 3.0},
                               {2, 128, 0.286, 2.0, 3.0, 1.2},
                               {1, 256, 0.395, 4.5, 5.0, 3.0},
                               {1, 128, 0.283, 2.0, 3.0, 1.2}};
constexpr int kSplitMax = SPLIT_PARTS + 1;
constexpr int64_t kMlpTicketWaves = 6;

TilePlan plan_tiles(const Product &q, int sms) {
    const bool dual = q.op == MlpOp::GATED;
    const int64_t nkb = div_up(q.k[0], 64) + div_up(q.k[1], 64);
    TilePlan best = {};
    double best_t = -1;
    for (const TileCost &tc : kTiles) {
        const int64_t teams = sms / tc.cg > 0 ? sms / tc.cg : 1;
        const int64_t mb = div_up(q.m, 128 * tc.cg), nb = div_up(q.n, dual ? tc.bn / 2 : tc.bn);
        const int64_t tiles = q.entries * mb * nb;
        const int64_t rem = tiles % teams;
        const double whole = (double)(tiles / teams) * nkb * tc.block;
        double t = whole + (rem ? nkb * tc.block : 0.0) + tc.epilogue;
        int split = 1;
        for (int s = 2; s <= kSplitMax && rem > 0; ++s) {
            if (s > teams / rem || s > nkb / SPLIT_MIN_KBLOCKS) break;
            const double ts = whole + nkb * tc.block / s + tc.epilogue + tc.join + tc.join_part * (s - 1);
            if (ts < t) {
                t = ts;
                split = s;
            }
        }
        if (best_t >= 0 && t >= best_t) continue;
        best_t = t;
        best.cg = tc.cg;
        best.block_n = tc.bn;
        best.tiles = tiles;
        best.tiles_per_entry = mb * nb;
        best.split_max = split;
        best.ticket = tiles >= kMlpTicketWaves * teams;
        // With a wave or more the grid is every team; below that, one team per
        // tile and K segment.
        best.grid = (int)(tc.cg * (tiles >= teams ? teams : tiles * split));
        const int64_t g = (best.ticket ? 12 : 8) * 2 / tc.cg;
        best.group = (int)(mb < g ? mb : g);
    }
    return best;
}

tg_status run_tiles(const Product &q, tg_dtype t, const Device &dev, cudaStream_t stream) {
    const TilePlan plan = plan_tiles(q, dev.sms);
    MlpLaunch la;
    std::memset(&la, 0, sizeof(la));
    const bool am = q.op == MlpOp::WGRAD, bm = q.op == MlpOp::DGRAD || am;
    const tg_out_dtype ot = out_type(t);
    const int64_t nkb = div_up(q.k[0], 64) + div_up(q.k[1], 64);
    if (nkb > INT32_MAX / 2 || plan.tiles > INT32_MAX) return TG_ERR_INVALID_VALUE;
    for (int i = 0; i < 2 && nkb > 0; ++i) {
        const Mat &a = q.a[i].p ? q.a[i] : q.a[0], &b = q.b[i].p ? q.b[i] : q.b[0];
        if (!host::encode_rows(&la.maps.a[i], ot, a.p, a.rows, a.cols, a.ld, am ? 64 : BLOCK_M) ||
            !host::encode_rows(&la.maps.b[i], ot, b.p, b.rows, b.cols, b.ld,
                               bm ? 64 : q.op == MlpOp::GATED ? plan.block_n / 2 : plan.block_n / plan.cg))
            return TG_ERR_INVALID_VALUE;
    }
    MlpParams &p = la.p;
    for (int i = 0; i < 3; ++i) {
        p.out[i].ptr = const_cast<void *>(q.out[i].p);
        p.out[i].ld = q.out[i].ld;
        p.out[i].vec = q.out[i].p && aligned16(q.out[i]);
    }
    p.r = q.r.p;
    p.ldr = q.r.ld;
    p.r_vec = q.r.p && aligned16(q.r);
    p.bias = q.bias;
    p.act = q.act;
    p.out_f32 = q.out_f32;
    p.k_blocks0 = (int32_t)div_up(q.k[0], 64);
    GemmParams &g = p.g;
    g.m = (int32_t)q.m;
    g.n = (int32_t)q.n;
    g.num_m_blocks = (int32_t)div_up(q.m, 128 * plan.cg);
    g.num_n_blocks = (int32_t)(plan.tiles_per_entry / g.num_m_blocks);
    g.num_k_blocks = (int32_t)nkb;
    g.raster_group = plan.group;
    g.num_tiles = plan.tiles;
    g.tiles_per_batch = plan.tiles_per_entry;
    g.batch = q.entries;
    g.status = dev.status;
    g.wait_limit_ns = dev.wait_limit_ns;
    g.split_max = 1;
    if (plan.split_max > 1 || plan.ticket) {
        host::Scratch w;
        const tg_status st = host::scratch(dev, stream, div_up(dev.sms, 2), &w);
        if (st != TG_OK) return st;
        g.split_max = plan.split_max;
        g.ws_tiles = (int32_t)(w.tiles * 2 / plan.cg);
        g.ws = w.ws;
        g.flags = w.flags;
        g.k_snake = plan.ticket ? 1 : 0;
        if (plan.ticket) g.ticket = w.ticket;
    }
    la.op = q.op;
    la.cg = plan.cg;
    la.block_n = plan.block_n;
    la.grid = plan.grid;
    la.device = dev.id;
    la.stream = stream;
    const cudaError_t e =
        t == TG_BF16 ? (plan.cg == 2 ? launch_mlp_bf16_cg2(la) : launch_mlp_bf16_cg1(la))
                     : (plan.cg == 2 ? launch_mlp_fp16_cg2(la) : launch_mlp_fp16_cg1(la));
    return e == cudaSuccess ? TG_OK : TG_ERR_CUDA;
}

// The weight-streaming kernel takes up to this many tokens: its token operand
// is one MMA's columns, re-read by every weight tile from L2 (16 KB per 16 KB
// of weights at 128 tokens); beyond, 256-row token tiles waste less.
constexpr int64_t kStreamTokens = 128;
// K blocks a CTA's share spans at least: below that the join costs more than
// the loads it spreads.
constexpr int64_t kStreamMinBlocks = 4;

tg_status run_stream(const Product &q, tg_dtype t, const Device &dev, cudaStream_t stream) {
    StreamLaunch la;
    std::memset(&la, 0, sizeof(la));
    la.dual = q.op == MlpOp::GATED;
    la.nt = q.m <= 16 ? 16 : q.m <= 32 ? 32 : q.m <= 64 ? 64 : 128;
    const tg_out_dtype ot = out_type(t);
    bool ok = host::encode_rows(&la.maps.w[0], ot, q.b[0].p, q.n, q.k[0], q.b[0].ld, BLOCK_M) &&
              host::encode_rows(&la.maps.x, ot, q.a[0].p, q.m, q.k[0], q.a[0].ld, la.nt);
    if (ok && la.dual)
        ok = host::encode_rows(&la.maps.w[1], ot, q.b[1].p, q.n, q.k[0], q.b[1].ld, BLOCK_M);
    if (!ok) return TG_ERR_INVALID_VALUE;
    StreamParams &p = la.p;
    p.tokens = (int32_t)q.m;
    p.features = (int32_t)q.n;
    p.tiles = (int32_t)div_up(q.n, BLOCK_M);
    p.num_k_blocks = (int32_t)div_up(q.k[0], 64);
    p.act = q.act;
    p.bias = q.bias;
    p.r = q.r.p;
    p.ldr = q.r.ld;
    for (int i = 0; i < 3; ++i) {
        p.out[i].ptr = const_cast<void *>(q.out[i].p);
        p.out[i].ld = q.out[i].ld;
    }
    const int64_t total = (int64_t)p.tiles * p.num_k_blocks;
    int64_t grid = total / kStreamMinBlocks;
    const int64_t cap = dev.sms < 512 ? dev.sms : 512;
    if (grid > cap) grid = cap;
    if (grid < 1) grid = 1;
    la.grid = (int)grid;
    host::Scratch w;
    const tg_status st = host::scratch(dev, stream, div_up(dev.sms, 2), &w);
    if (st != TG_OK) return st;
    p.ws = w.ws;
    p.flags = w.stream_flags;
    p.status = dev.status;
    p.wait_limit_ns = dev.wait_limit_ns;
    la.device = dev.id;
    la.stream = stream;
    const cudaError_t e = t == TG_BF16 ? launch_stream_bf16(la) : launch_stream_fp16(la);
    return e == cudaSuccess ? TG_OK : TG_ERR_CUDA;
}

bool space_ok(const Arena &need, const void *workspace, int64_t bytes) {
    return need.used == 0 || (workspace && (uintptr_t)workspace % 16 == 0 && bytes >= need.used);
}

#define TG_TRY(expr)                                   \
    do {                                               \
        if ((expr) != cudaSuccess) return TG_ERR_CUDA; \
    } while (0)

// Forward of both operators: `w2` is NULL for the linear layer.
tg_status forward(MlpOp op, int64_t M, int64_t N, int64_t K, Mat x, Mat w, Mat w2, Product &q,
                  tg_dtype dtype, void *workspace, int64_t workspace_bytes, cudaStream_t stream) {
    Arena need(workspace);
    Mat *ops[3] = {&x, &w, &w2};
    Mat from[3] = {x, w, w2};
    bool moved[3] = {false, false, false};
    const int count = op == MlpOp::GATED ? 3 : 2;
    for (int i = 0; i < count; ++i)
        if (K > 0 && needs_repack(*ops[i])) {
            *ops[i] = need.repacked(*ops[i]);
            moved[i] = true;
        }
    if (!space_ok(need, workspace, workspace_bytes)) return TG_ERR_INVALID_VALUE;
    Device dev;
    const tg_status st = host::device(&dev);
    if (st != TG_OK) return st;
    for (int i = 0; i < count; ++i)
        if (moved[i]) TG_TRY(repack(dtype, from[i], *ops[i], dev.sms, stream));
    q.op = op;
    q.m = M;
    q.n = N;
    q.k[0] = K;
    q.entries = 1;
    q.a[0] = x;
    q.b[0] = w;
    q.b[1] = w2;
    if (M <= kStreamTokens && K > 0) return run_stream(q, dtype, dev, stream);
    return run_tiles(q, dtype, dev, stream);
}

}  // namespace

// ------------------------------------------------------------------ C ABI

extern "C" int64_t tg_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, const void *X,
                                             int64_t ldx, const void *W, int64_t ldw,
                                             tg_dtype dtype) {
    if (!dims_ok(M, N, K) || !type_ok(dtype) || ldx < K || ldw < K) return -1;
    Arena need(nullptr);
    for (const Mat &a : {mat(X, ldx, M, K), mat(W, ldw, N, K)})
        if (needs_repack(a)) need.repacked(a);
    return need.used;
}

extern "C" tg_status tg_linear(int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
                               const void *W, int64_t ldw, const float *bias, tg_activation act,
                               const void *R, int64_t ldr, void *Y, int64_t ldy, void *Z,
                               int64_t ldz, tg_dtype dtype, void *workspace,
                               int64_t workspace_bytes, void *stream) {
    if (!dims_ok(M, N, K) || !type_ok(dtype) || !act_ok(act) || workspace_bytes < 0)
        return TG_ERR_INVALID_VALUE;
    if (!mat_ok(X, ldx, M, K) || !mat_ok(W, ldw, N, K) || !mat_ok(Y, ldy, M, N))
        return TG_ERR_INVALID_VALUE;
    if ((R && !mat_ok(R, ldr, M, N)) || (Z && !mat_ok(Z, ldz, M, N)) || (uintptr_t)bias % 4)
        return TG_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return TG_OK;
    Product q = {};
    q.out[0] = mat(Y, ldy, M, N);
    if (Z) q.out[1] = mat(Z, ldz, M, N);
    if (R) q.r = mat(R, ldr, M, N);
    q.bias = bias;
    q.act = (int)act;
    return forward(MlpOp::LINEAR, M, N, K, mat(X, ldx, M, K), mat(W, ldw, N, K), Mat{}, q, dtype,
                   workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

namespace {

// What the linear layer's backward pass keeps in the workspace.
struct LinearSpace {
    Arena arena;
    Mat dz, x, w;
    bool dz_made, x_moved, w_moved;
    float *partial;
    int64_t bands;
};
LinearSpace linear_space(int64_t M, int64_t N, int64_t K, const Mat &dy, const Mat &x, const Mat &w,
                         bool act, bool dx, bool dw, bool db, int sms, void *base) {
    LinearSpace s{Arena(base), dy, x, w, false, false, false, nullptr, 0};
    if (M == 0 || N == 0) return s;
    if (dx || dw) {
        s.dz_made = act || needs_repack(dy);
        if (s.dz_made) s.dz = s.arena.repacked(dy);
        s.x_moved = dw && needs_repack(x);
        if (s.x_moved) s.x = s.arena.repacked(x);
        s.w_moved = dx && needs_repack(w);
        if (s.w_moved) s.w = s.arena.repacked(w);
    }
    if (db) {
        s.bands = act_bands(M, N, sms);
        s.bands = div_up(M, div_up(M, s.bands));
        s.partial = static_cast<float *>(s.arena.take(4 * N * s.bands));
    }
    (void)K;
    return s;
}

}  // namespace

extern "C" int64_t tg_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K,
                                                      const void *dY, int64_t lddy, const void *X,
                                                      int64_t ldx, const void *W, int64_t ldw,
                                                      tg_activation act, tg_dtype dtype) {
    if (!dims_ok(M, N, K) || !type_ok(dtype) || !act_ok(act) || lddy < N || ldx < K || ldw < K)
        return -1;
    Device dev;
    if (host::device(&dev) != TG_OK) return -1;
    return linear_space(M, N, K, mat(dY, lddy, M, N), mat(X, ldx, M, K), mat(W, ldw, N, K),
                        act != TG_ACT_NONE, true, true, true, dev.sms, nullptr)
        .arena.used;
}

extern "C" tg_status tg_linear_backward(int64_t M, int64_t N, int64_t K, const void *dY,
                                        int64_t lddy, const void *X, int64_t ldx, const void *W,
                                        int64_t ldw, const void *Z, int64_t ldz, tg_activation act,
                                        void *dX, int64_t lddx, void *dW, int64_t lddw,
                                        tg_out_dtype dw_dtype, float *db, tg_dtype dtype,
                                        void *workspace, int64_t workspace_bytes,
                                        void *stream_ptr) {
    if (!dims_ok(M, N, K) || !type_ok(dtype) || !act_ok(act) || workspace_bytes < 0)
        return TG_ERR_INVALID_VALUE;
    if (dw_dtype != TG_OUT_F32 && dw_dtype != out_type(dtype)) return TG_ERR_INVALID_VALUE;
    const int ew = dw_dtype == TG_OUT_F32 ? 4 : 2;
    if (!mat_ok(dY, lddy, M, N)) return TG_ERR_INVALID_VALUE;
    if (act != TG_ACT_NONE && !mat_ok(Z, ldz, M, N)) return TG_ERR_INVALID_VALUE;
    if (dX && (!mat_ok(W, ldw, N, K) || !mat_ok(dX, lddx, M, K))) return TG_ERR_INVALID_VALUE;
    if (dW && (!mat_ok(X, ldx, M, K) || !mat_ok(dW, lddw, N, K, ew))) return TG_ERR_INVALID_VALUE;
    if ((uintptr_t)db % 4) return TG_ERR_INVALID_VALUE;
    const bool dx = dX && M > 0 && K > 0, dw = dW && N > 0 && K > 0, sum = db && N > 0;
    if (!dx && !dw && !sum) return TG_OK;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    Device dev;
    tg_status st = host::device(&dev);
    if (st != TG_OK) return st;
    const Mat dy = mat(dY, lddy, M, N), x = mat(X, ldx, M, K), w = mat(W, ldw, N, K);
    LinearSpace s = linear_space(M, N, K, dy, x, w, act != TG_ACT_NONE, dx, dw, sum, dev.sms, workspace);
    if (!space_ok(s.arena, workspace, workspace_bytes)) return TG_ERR_INVALID_VALUE;
    if (s.dz_made || s.partial) {
        ActParams p = {};
        p.m = M;
        p.n = N;
        p.dy = dY;
        p.lddy = lddy;
        if (act != TG_ACT_NONE) {
            p.z = Z;
            p.ldz = ldz;
        }
        p.act = (int32_t)act;
        if (s.dz_made) {
            p.out0 = const_cast<void *>(s.dz.p);
            p.ldo0 = s.dz.ld;
        }
        p.partial = s.partial;
        TG_TRY(launch_act<false>(dtype, p, dev.sms, stream));
    }
    if (sum) TG_TRY(host::colsum_finish(s.partial, nullptr, (int32_t)s.bands, N, db, nullptr, stream));
    if (s.w_moved) TG_TRY(repack(dtype, w, s.w, dev.sms, stream));
    if (s.x_moved) TG_TRY(repack(dtype, x, s.x, dev.sms, stream));
    if (dx) {
        Product q = {};
        q.op = MlpOp::DGRAD;
        q.m = M;
        q.n = K;
        q.k[0] = N;
        q.entries = 1;
        q.a[0] = s.dz;
        q.b[0] = s.w;
        q.out[0] = mat(dX, lddx, M, K);
        st = run_tiles(q, dtype, dev, stream);
        if (st != TG_OK) return st;
    }
    if (dw) {
        Product q = {};
        q.op = MlpOp::WGRAD;
        q.m = N;
        q.n = K;
        q.k[0] = M;
        q.entries = 1;
        q.a[0] = s.dz;
        q.b[0] = s.x;
        q.out[0] = mat(dW, lddw, N, K, ew);
        q.out_f32 = dw_dtype == TG_OUT_F32;
        st = run_tiles(q, dtype, dev, stream);
        if (st != TG_OK) return st;
    }
    return TG_OK;
}

extern "C" int64_t tg_gated_workspace_bytes(int64_t M, int64_t N, int64_t K, const void *X,
                                            int64_t ldx, const void *Wg, int64_t ldwg,
                                            const void *Wu, int64_t ldwu, tg_dtype dtype) {
    if (!dims_ok(M, N, K) || !type_ok(dtype) || ldx < K || ldwg < K || ldwu < K) return -1;
    Arena need(nullptr);
    for (const Mat &a : {mat(X, ldx, M, K), mat(Wg, ldwg, N, K), mat(Wu, ldwu, N, K)})
        if (needs_repack(a)) need.repacked(a);
    return need.used;
}

extern "C" tg_status tg_gated(int64_t M, int64_t N, int64_t K, const void *X, int64_t ldx,
                              const void *Wg, int64_t ldwg, const void *Wu, int64_t ldwu,
                              tg_activation act, void *H, int64_t ldh, void *G, int64_t ldg, void *U,
                              int64_t ldu, tg_dtype dtype, void *workspace,
                              int64_t workspace_bytes, void *stream) {
    if (!dims_ok(M, N, K) || !type_ok(dtype) || !act_ok(act) || workspace_bytes < 0)
        return TG_ERR_INVALID_VALUE;
    if (!mat_ok(X, ldx, M, K) || !mat_ok(Wg, ldwg, N, K) || !mat_ok(Wu, ldwu, N, K) ||
        !mat_ok(H, ldh, M, N))
        return TG_ERR_INVALID_VALUE;
    if ((G && !mat_ok(G, ldg, M, N)) || (U && !mat_ok(U, ldu, M, N))) return TG_ERR_INVALID_VALUE;
    if (M == 0 || N == 0) return TG_OK;
    Product q = {};
    q.out[0] = mat(H, ldh, M, N);
    if (G) q.out[1] = mat(G, ldg, M, N);
    if (U) q.out[2] = mat(U, ldu, M, N);
    q.act = (int)act;
    return forward(MlpOp::GATED, M, N, K, mat(X, ldx, M, K), mat(Wg, ldwg, N, K),
                   mat(Wu, ldwu, N, K), q, dtype, workspace, workspace_bytes,
                   static_cast<cudaStream_t>(stream));
}

namespace {

struct GatedSpace {
    Arena arena;
    Mat dg, du, x, wg, wu;
    bool x_moved, wg_moved, wu_moved;
};
GatedSpace gated_space(int64_t M, int64_t N, const Mat &x, const Mat &wg, const Mat &wu, bool dx,
                       bool dw, void *base) {
    GatedSpace s{Arena(base), {}, {}, x, wg, wu, false, false, false};
    if (M == 0 || N == 0) return s;
    const Mat dh = {nullptr, N, M, N, 2};
    s.dg = s.arena.repacked(dh);
    s.du = s.arena.repacked(dh);
    if ((s.x_moved = dw && needs_repack(x))) s.x = s.arena.repacked(x);
    if ((s.wg_moved = dx && needs_repack(wg))) s.wg = s.arena.repacked(wg);
    if ((s.wu_moved = dx && needs_repack(wu))) s.wu = s.arena.repacked(wu);
    return s;
}

}  // namespace

extern "C" int64_t tg_gated_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, const void *X,
                                                     int64_t ldx, const void *Wg, int64_t ldwg,
                                                     const void *Wu, int64_t ldwu, tg_dtype dtype) {
    if (!dims_ok(M, N, K) || !type_ok(dtype) || ldx < K || ldwg < K || ldwu < K) return -1;
    return gated_space(M, N, mat(X, ldx, M, K), mat(Wg, ldwg, N, K), mat(Wu, ldwu, N, K), true, true,
                       nullptr)
        .arena.used;
}

extern "C" tg_status tg_gated_backward(int64_t M, int64_t N, int64_t K, const void *dH, int64_t lddh,
                                       const void *X, int64_t ldx, const void *Wg, int64_t ldwg,
                                       const void *Wu, int64_t ldwu, const void *G, int64_t ldg,
                                       const void *U, int64_t ldu, tg_activation act, void *dX,
                                       int64_t lddx, void *dWg, int64_t lddwg, void *dWu,
                                       int64_t lddwu, tg_out_dtype dw_dtype, tg_dtype dtype,
                                       void *workspace, int64_t workspace_bytes, void *stream_ptr) {
    if (!dims_ok(M, N, K) || !type_ok(dtype) || !act_ok(act) || workspace_bytes < 0)
        return TG_ERR_INVALID_VALUE;
    if (dw_dtype != TG_OUT_F32 && dw_dtype != out_type(dtype)) return TG_ERR_INVALID_VALUE;
    const int ew = dw_dtype == TG_OUT_F32 ? 4 : 2;
    if (!mat_ok(dH, lddh, M, N) || !mat_ok(G, ldg, M, N) || !mat_ok(U, ldu, M, N))
        return TG_ERR_INVALID_VALUE;
    if (dX && (!mat_ok(Wg, ldwg, N, K) || !mat_ok(Wu, ldwu, N, K) || !mat_ok(dX, lddx, M, K)))
        return TG_ERR_INVALID_VALUE;
    if ((dWg || dWu) && !mat_ok(X, ldx, M, K)) return TG_ERR_INVALID_VALUE;
    if ((dWg && !mat_ok(dWg, lddwg, N, K, ew)) || (dWu && !mat_ok(dWu, lddwu, N, K, ew)))
        return TG_ERR_INVALID_VALUE;
    const bool dx = dX && M > 0 && K > 0, dw = (dWg || dWu) && N > 0 && K > 0;
    if (!dx && !dw) return TG_OK;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    Device dev;
    tg_status st = host::device(&dev);
    if (st != TG_OK) return st;
    const Mat x = mat(X, ldx, M, K), wg = mat(Wg, ldwg, N, K), wu = mat(Wu, ldwu, N, K);
    GatedSpace s = gated_space(M, N, x, wg, wu, dx, dw, workspace);
    if (!space_ok(s.arena, workspace, workspace_bytes)) return TG_ERR_INVALID_VALUE;
    if (M > 0 && N > 0) {
        ActParams p = {};
        p.m = M;
        p.n = N;
        p.dy = dH;
        p.lddy = lddh;
        p.z = G;
        p.ldz = ldg;
        p.u = U;
        p.ldu = ldu;
        p.act = (int32_t)act;
        p.out0 = const_cast<void *>(s.dg.p);
        p.ldo0 = s.dg.ld;
        p.out1 = const_cast<void *>(s.du.p);
        p.ldo1 = s.du.ld;
        TG_TRY(launch_act<true>(dtype, p, dev.sms, stream));
    }
    if (s.wg_moved) TG_TRY(repack(dtype, wg, s.wg, dev.sms, stream));
    if (s.wu_moved) TG_TRY(repack(dtype, wu, s.wu, dev.sms, stream));
    if (s.x_moved) TG_TRY(repack(dtype, x, s.x, dev.sms, stream));
    if (dx) {
        Product q = {};
        q.op = MlpOp::DGRAD;
        q.m = M;
        q.n = K;
        q.k[0] = q.k[1] = N;
        q.entries = 1;
        q.a[0] = s.dg;
        q.a[1] = s.du;
        q.b[0] = s.wg;
        q.b[1] = s.wu;
        q.out[0] = mat(dX, lddx, M, K);
        st = run_tiles(q, dtype, dev, stream);
        if (st != TG_OK) return st;
    }
    if (dw) {
        Product q = {};
        q.op = MlpOp::WGRAD;
        q.m = N;
        q.n = K;
        q.k[0] = M;
        q.entries = dWg && dWu ? 2 : 1;
        q.a[0] = dWg ? s.dg : s.du;
        q.a[1] = s.du;
        q.b[0] = s.x;
        q.out[0] = dWg ? mat(dWg, lddwg, N, K, ew) : mat(dWu, lddwu, N, K, ew);
        if (q.entries == 2) q.out[1] = mat(dWu, lddwu, N, K, ew);
        q.out_f32 = dw_dtype == TG_OUT_F32;
        st = run_tiles(q, dtype, dev, stream);
        if (st != TG_OK) return st;
    }
    return TG_OK;
}

// ------------------------------------------------------------------ shared launch

namespace tg {
namespace host {

cudaError_t colsum_finish(const float *partial0, const float *partial1, int32_t parts, int64_t n,
                          float *out0, float *out1, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)div_up(n, FINISH_COLS), out1 ? 2 : 1, 1);
    cfg.blockDim = dim3(FINISH_COLS, FINISH_ROWS, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tg_colsum_finish_kernel, partial0, partial1, parts, n, out0, out1);
}

}  // namespace host
}  // namespace tg
