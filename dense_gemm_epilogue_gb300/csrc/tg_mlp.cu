// Front end of the feed-forward operators (linear layer and gated unit,
// forward and backward): argument checks, the planner of their products, the
// row-wise kernels of the backward pass, and the entry points.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../include/tg_gemm.h"
#include "tg_host.h"
#include "tg_mlp.h"
#include "tg_rows.cuh"

namespace tg {

// ------------------------------------------------------------------ row-wise jobs

// What the products need done to whole matrices first, as up to four jobs of
// one launch (each with its own blocks):
//   LINEAR  dz = dy act'(z), rounded to the operands' type (it is an operand of
//           two tensor-core products), and from the unrounded FP32 values the
//           column sums db; without z, dz = dy: a repack to aligned rows, or
//           the sums alone;
//   GATED   dg = dh u act'(g), du = dh act(g).
//
// Bound: memory (LINEAR reads 2 and writes 1, GATED reads 3 and writes 2 values
// per element), with an activation close to issue: 4096 x 16384 BF16 with GELU and
// column sums 71 us from cold caches, 5.7 TB/s with 68 % of the issue slots taken;
// the column sums alone (268 MB read, nothing written) 55 us.  A warp takes 256
// columns of a row, 8 values a lane; eight warps take rows r, r + 8, ... of the
// block's band, two (GATED: one; without z: four) rows in flight each.  Rows that are not
// 16-byte aligned are read as the two aligned 16-byte words that hold a lane's
// values and shifted into place (the shift is the same for a whole row); a
// row's first and last values, whose words reach past it, come one by one.
//
// Column sums: a band's add up over its rows in registers, then over the eight
// warps in order, into the workspace; tg_colsum_finish_kernel adds the bands in
// order, after the products, which do not wait for it (the last block of each
// strip finishing its own sums held them up by 4 us at 777 x 1001).
constexpr int ROW_JOBS = 4;
constexpr int ROW_COLS = 256;

struct RowJob {
    int64_t m, n;
    const void *dy, *z, *u;
    int64_t lddy, ldz, ldu;
    void *out0, *out1;  // dz, or dg and du (out0 NULL: sums only); 16-byte aligned rows
    int64_t ldo0, ldo1;
    float *partial;     // [bands][n] or NULL
    int32_t act;
    int32_t gated;
    int32_t aligned;    // every input's rows are 16-byte aligned
    int32_t band;       // rows per block
    int32_t bands, strips;
};
struct RowJobs {
    RowJob job[ROW_JOBS];
    int32_t first[ROW_JOBS + 1];  // first block of each job
    int32_t count;
};

// Eight 16-bit values at any 2-byte aligned address, from the two aligned
// 16-byte words around them.
__device__ __forceinline__ uint4 load_shifted(const unsigned short *q) {
    const uintptr_t at = (uintptr_t)q;
    const uint4 *w = reinterpret_cast<const uint4 *>(at & ~(uintptr_t)15);
    const uint32_t s = (uint32_t)at & 15u;
    const uint4 a = w[0];
    if (s == 0) return a;
    const uint4 b = w[1];
    const uint32_t bits = (s & 2u) * 8;
    uint32_t x0, x1, x2, x3, x4;
    switch (s >> 2) {
    case 0: x0 = a.x; x1 = a.y; x2 = a.z; x3 = a.w; x4 = b.x; break;
    case 1: x0 = a.y; x1 = a.z; x2 = a.w; x3 = b.x; x4 = b.y; break;
    case 2: x0 = a.z; x1 = a.w; x2 = b.x; x3 = b.y; x4 = b.z; break;
    default: x0 = a.w; x1 = b.x; x2 = b.y; x3 = b.z; x4 = b.w; break;
    }
    return make_uint4(__funnelshift_r(x0, x1, bits), __funnelshift_r(x1, x2, bits),
                      __funnelshift_r(x2, x3, bits), __funnelshift_r(x3, x4, bits));
}

// Values c .. c + 7 of a row, one by one, zero past its end.
__device__ __forceinline__ uint4 load_edge(const unsigned short *row, int64_t c, int64_t n) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < n) w[i / 2] |= (uint32_t)row[c + i] << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One block's band; c: this lane's first column.
template <class Ty, bool GATED, int ACT, bool ALIGNED>
__device__ __forceinline__ void row_band(const RowJob &p, int64_t c, int64_t r0, int64_t r1,
                                         float (&s)[8]) {
    using T = unsigned short;
    const T *dy = static_cast<const T *>(p.dy), *z = static_cast<const T *>(p.z);
    const T *u = static_cast<const T *>(p.u);
    T *o0 = static_cast<T *>(p.out0), *o1 = static_cast<T *>(p.out1);
    constexpr bool READ_Z = GATED || ACT != MLP_NONE;
    constexpr int FLY = GATED ? 1 : READ_Z ? 2 : 4;  // rows in flight per warp
    if (c >= p.n) return;
    // Whole vectors: aligned ones that end inside the row; shifted ones whose
    // two words lie inside it.
    const bool mid = ALIGNED ? c + 8 <= p.n : c >= 8 && c + 16 <= p.n;
    for (int64_t r = r0 + (threadIdx.x >> 5); r < r1; r += 8 * FLY) {
        uint4 vd[FLY], vz[FLY], vu[FLY];
        auto load = [&](auto get) {
#pragma unroll
            for (int k = 0; k < FLY; ++k) {
                // (rows past the band load its last row again and are dropped)
                const int64_t rr = r + 8 * k < r1 ? r + 8 * k : r1 - 1;
                vd[k] = get(dy + rr * p.lddy);
                if (READ_Z) vz[k] = get(z + rr * p.ldz);
                if (GATED) vu[k] = get(u + rr * p.ldu);
            }
        };
        if (mid) {
            if (ALIGNED) load([&](const T *row) { return __ldcs(reinterpret_cast<const uint4 *>(row + c)); });
            else load([&](const T *row) { return load_shifted(row + c); });
        } else {
            load([&](const T *row) { return load_edge(row, c, p.n); });
        }
#pragma unroll
        for (int k = 0; k < FLY; ++k) {
            const int64_t rr = r + 8 * k;
            if (rr < r1) {
                float d[8], a[8], g[8];
                row_unpack<Ty>(vd[k], d);
                if constexpr (READ_Z) {
                    float y[8];
                    row_unpack<Ty>(vz[k], y);
#pragma unroll
                    for (int i = 0; i < 8; ++i) mlp_act_grad<ACT>(y[i], a[i], g[i]);
                }
                if constexpr (GATED) {
                    float w[8];
                    row_unpack<Ty>(vu[k], w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        a[i] *= d[i];
                        d[i] *= w[i] * g[i];
                    }
                    row_store<Ty>(o0 + rr * p.ldo0, c, p.n, d);
                    row_store<Ty>(o1 + rr * p.ldo1, c, p.n, a);
                } else if constexpr (READ_Z) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[i] *= g[i];
                    if (o0) row_store<Ty>(o0 + rr * p.ldo0, c, p.n, d);
                } else if (o0) {  // a plain copy keeps every bit (NaN payloads too)
                    T *q = o0 + rr * p.ldo0 + c;
                    if (c + 8 <= p.n) {
                        *reinterpret_cast<uint4 *>(q) = vd[k];
                    } else {
                        const T *e = reinterpret_cast<const T *>(&vd[k]);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (c + i < p.n) q[i] = e[i];
                    }
                }
                if constexpr (!GATED) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[i] += d[i];
                }
            }
        }
    }
}

template <class Ty>
__global__ void __launch_bounds__(256, 4) tg_row_jobs_kernel(const __grid_constant__ RowJobs jobs) {
    __shared__ float sums[8][ROW_COLS];
    griddep_launch();
    griddep_wait();
    int j = 0;
    while (j + 1 < jobs.count && (int)blockIdx.x >= jobs.first[j + 1]) ++j;
    const RowJob &p = jobs.job[j];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int local = (int)blockIdx.x - jobs.first[j];
    const int band = local / p.strips, strip = local - band * p.strips;
    const int64_t c0 = (int64_t)strip * ROW_COLS, c = c0 + lane * 8;
    const int64_t r0 = (int64_t)band * p.band;
    const int64_t r1 = r0 + p.band < p.m ? r0 + p.band : p.m;
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.0f;
    mlp_with_act(p.act, [&](auto act) {
        if (p.gated) {
            if (p.aligned) row_band<Ty, true, act.value, true>(p, c, r0, r1, s);
            else row_band<Ty, true, act.value, false>(p, c, r0, r1, s);
        } else {
            if (p.aligned) row_band<Ty, false, act.value, true>(p, c, r0, r1, s);
            else row_band<Ty, false, act.value, false>(p, c, r0, r1, s);
        }
    });
    if (!p.partial) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[warp][lane * 8 + i] = s[i];
    __syncthreads();
    const int64_t cc = c0 + threadIdx.x;
    if (cc < p.n) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += sums[w][threadIdx.x];
        p.partial[(int64_t)band * p.n + cc] = t;
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

// Bands of a row-wise job: about eight blocks per SM in all, at least 32 rows
// each (four per warp).
int64_t row_bands(int64_t m, int64_t n, int sms) {
    const int64_t strips = div_up(n, ROW_COLS);
    int64_t bands = div_up((int64_t)sms * 8, strips);
    if (bands > div_up(m, 32)) bands = div_up(m, 32);
    if (bands < 1) bands = 1;
    return m > 0 ? div_up(m, div_up(m, bands)) : 1;
}

// The jobs of one launch.
struct RowWork {
    RowJobs jobs;
    int64_t blocks = 0;
    int sms;
    explicit RowWork(int sms_) : sms(sms_) { jobs.count = 0; }
    RowJob &add(int64_t m, int64_t n) {
        RowJob &p = jobs.job[jobs.count];
        std::memset(&p, 0, sizeof(p));
        p.m = m;
        p.n = n;
        p.bands = (int32_t)row_bands(m, n, sms);
        p.band = (int32_t)div_up(m, p.bands);
        p.strips = (int32_t)div_up(n, ROW_COLS);
        jobs.first[jobs.count++] = (int32_t)blocks;
        blocks += (int64_t)p.bands * p.strips;
        return p;
    }
    // `from`, repacked into `to`'s aligned rows.
    void repack(const Mat &from, const Mat &to) {
        RowJob &p = add(from.rows, from.cols);
        p.dy = from.p;
        p.lddy = from.ld;
        p.out0 = const_cast<void *>(to.p);
        p.ldo0 = to.ld;
    }
    cudaError_t launch(tg_dtype t, cudaStream_t stream) {
        if (jobs.count == 0) return cudaSuccess;
        if (blocks > INT32_MAX) return cudaErrorInvalidValue;
        for (int i = 0; i < jobs.count; ++i) {
            RowJob &p = jobs.job[i];
            auto al = [](const void *q, int64_t ld) { return (uintptr_t)q % 16 == 0 && ld % 8 == 0; };
            p.aligned = al(p.dy, p.lddy) && (!p.z || al(p.z, p.ldz)) && (!p.u || al(p.u, p.ldu));
        }
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3((unsigned)blocks, 1, 1);
        cfg.blockDim = dim3(256, 1, 1);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return t == TG_BF16 ? cudaLaunchKernelEx(&cfg, tg_row_jobs_kernel<TypeBF16>, jobs)
                            : cudaLaunchKernelEx(&cfg, tg_row_jobs_kernel<TypeF16>, jobs);
    }
};

// One product, in role space.
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
    uint32_t *gate;    // MlpParams::gate (input gradient: raised; weight gradient: runs beside it)
};

struct TilePlan {
    int cg, block_n;
    int64_t tiles, tiles_per_entry;
    int grid, split_max, group;
    bool ticket;
    double time;  // the model's, in microseconds
};

// Times of the planner's cost model, in microseconds, measured on long and
// short products of each tile shape: one 64-deep K block of a team's tile; what
// its epilogue adds where nothing overlaps it; and what joining s segments adds
// to a split tile (FP32 partial sums written, then s - 1 of them read back).
// (One wave of tiles, 2048 and 8192 deep, inputs past L2: 0.29, 0.28, 0.38 and 0.28 a
// K block on the present build; the first takes 0.36 in long products, at the power
// limit.)  The 128-column tiles move 3/4 of the bytes per K block for half the work, so
// they pay only where they fill SMs that 256-column tiles leave idle.  A 256 x 128
// pair tile takes what two 128 x 128 CTAs on the same two SMs take for the same
// work, so it is never the cheapest alone; but it leaves whole twos of SMs to a
// second product in pairs beside it (both gradients of 777 x 1001 x 1365: 32.5 us
// with it, 33.3 with single CTAs for both), so the gradients have it.
struct TileCost {
    int cg, bn;
    double block, epilogue, join, join_part;
};
constexpr TileCost kTiles[] = {{2, 256, 0.350, 4.5, 5.0, 3.0},
                               {2, 128, 0.286, 2.0, 3.0, 1.2},
                               {1, 256, 0.395, 4.5, 5.0, 3.0},
                               {1, 128, 0.283, 2.0, 3.0, 1.2}};
constexpr int kSplitMax = SPLIT_PARTS + 1;
// Tickets (units claimed in order from a counter) from six waves of tiles up,
// as in the CTA-pair GEMM, and only for tiles that take longer than a claim
// (about 2 us: at one K block, 1 x 1168 x 7568, tickets cost 18 of 22 us).
constexpr int64_t kMlpTicketWaves = 6, kMlpTicketBlocks = 16;

// The cheapest plan; or (shape >= 0) kTiles[shape] without split tiles.
TilePlan plan_tiles(const Product &q, int sms, int shape = -1) {
    const bool dual = q.op == MlpOp::GATED;
    const int64_t nkb = div_up(q.k[0], 64) + div_up(q.k[1], 64);
    TilePlan best = {};
    double best_t = -1;
    for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
        if (shape >= 0 && i != shape) continue;
        const TileCost &tc = kTiles[i];
        if (tc.cg == 2 && tc.bn == 128 && q.op != MlpOp::DGRAD && q.op != MlpOp::WGRAD) continue;
        const int64_t teams = sms / tc.cg > 0 ? sms / tc.cg : 1;
        const int64_t mb = div_up(q.m, 128 * tc.cg), nb = div_up(q.n, dual ? tc.bn / 2 : tc.bn);
        const int64_t tiles = q.entries * mb * nb;
        const int64_t rem = tiles % teams;
        const double whole = (double)(tiles / teams) * nkb * tc.block;
        double t = whole + (rem ? nkb * tc.block : 0.0) + tc.epilogue;
        int split = 1;
        for (int s = 2; s <= kSplitMax && rem > 0 && shape < 0; ++s) {
            if (s > teams / rem || s > nkb / SPLIT_MIN_KBLOCKS) break;
            const double ts = whole + nkb * tc.block / s + tc.epilogue + tc.join + tc.join_part * (s - 1);
            if (ts < t) {
                t = ts;
                split = s;
            }
        }
        if (best_t >= 0 && t >= best_t) continue;
        best_t = best.time = t;
        best.cg = tc.cg;
        best.block_n = tc.bn;
        best.tiles = tiles;
        best.tiles_per_entry = mb * nb;
        best.split_max = split;
        best.ticket = tiles >= kMlpTicketWaves * teams && nkb >= kMlpTicketBlocks;
        // With a wave or more the grid is every team; below that, one team per
        // tile and K segment.
        best.grid = (int)(tc.cg * (tiles >= teams ? teams : tiles * split));
        const int64_t g = (best.ticket ? 12 : 8) * 2 / tc.cg;
        best.group = (int)(mb < g ? mb : g);
    }
    return best;
}

// Plans for an input gradient `x` and the weight gradient `w` after it, when
// both fit the SMs together and running side by side is cheaper than in turn
// (777 x 1000 x 1368: 44 pairs of 256 x 128 tiles and 24 of 256 x 256 at once 21.5
// us, one after the other 25.1; 3 x 1628 x 256, streaming, 12.2 and 15.6).
struct Beside {
    bool on = false;
    TilePlan x, w;
};

tg_status run_stream(const Product &q, tg_dtype t, const Device &dev, cudaStream_t stream);

// The weight-streaming kernel takes up to 64 tokens, gated 32.  Every weight tile
// reads them again from L2, and the join's traffic grows with them (twice as much
// for the gated unit's two products), while a 128-row token tile costs the same for
// any count.  Streaming and tiles in us, a captured chain of calls, inputs past L2:
//               N x K             32 tokens     64 tokens     96 tokens
//   linear      4096 x 4096       12.2  16.8    14.9  16.9    17.5  17.3
//               4096 x 14336      26.9  30.6    29.7  30.8    32.8  31.4
//   dX          4096 x 4096       13.8  15.2    14.5  15.3    16.9  15.5
//               14336 x 4096      25.4  27.6    29.1  27.7    31.8  28.2
//   gated       4096 x 4096       18.1  20.1    22.4  20.4    26.2  20.4
//               1024 x 4096       14.1  14.4    18.0  14.4    22.0  14.7
//               14336 x 4096      45.4  43.0    48.2  43.0    52.2  43.0
//   gated dX    4096 x 4096       25.0  24.6    26.5  25.4    28.5  25.9
//               1024 x 4096       14.5  16.8    15.6  16.9    17.7  17.2
bool streams(const Product &q) {
    return q.m <= (q.op == MlpOp::GATED ? 32 : 64) && q.op != MlpOp::WGRAD && q.k[0] > 0;
}

// Whether `w`'s CTAs find room while all of `x`'s run.  A CTA pair needs both SMs
// of a neighbouring two, and single CTAs before it are spread over as many such
// twos as there are.
bool fit_beside(const TilePlan &x, const TilePlan &w, int sms) {
    if (w.cg == 1) return x.grid + w.grid <= sms;
    const int twos = sms / 2, taken = x.cg == 2 ? x.grid / 2 : x.grid < twos ? x.grid : twos;
    return taken + w.grid / 2 <= twos;
}

Beside plan_beside(const Product &x, const Product &w, int sms) {
    Beside best;
    if (streams(x) || x.k[0] == 0 || w.k[0] == 0) return best;
    double t = plan_tiles(x, sms).time + plan_tiles(w, sms).time;
    constexpr int SHAPES = sizeof(kTiles) / sizeof(kTiles[0]);
    for (int i = 0; i < SHAPES; ++i)
        for (int j = 0; j < SHAPES; ++j) {
            const TilePlan a = plan_tiles(x, sms, i), b = plan_tiles(w, sms, j);
            const double both = a.time > b.time ? a.time : b.time;
            if (!fit_beside(a, b, sms) || a.ticket || b.ticket || both >= t) continue;
            t = both;
            best.on = true;
            best.x = a;
            best.w = b;
        }
    return best;
}

tg_status run_product(const Product &q, tg_dtype t, const Device &dev, cudaStream_t stream,
                      const TilePlan *chosen = nullptr) {
    if (streams(q)) return run_stream(q, t, dev, stream);
    const TilePlan plan = chosen ? *chosen : plan_tiles(q, dev.sms);
    MlpLaunch la;
    std::memset(&la, 0, sizeof(la));
    const bool am = q.op == MlpOp::WGRAD, bm = q.op == MlpOp::DGRAD || am;
    const tg_out_dtype ot = out_type(t);
    const int64_t nkb = div_up(q.k[0], 64) + div_up(q.k[1], 64);
    if (nkb > INT32_MAX / 2 || plan.tiles > INT32_MAX) return TG_ERR_INVALID_VALUE;
    const int b_box = bm ? 64 : q.op == MlpOp::GATED ? plan.block_n / 2 : plan.block_n / plan.cg;
    for (int i = 0; i < 2 && nkb > 0; ++i) {
        const Mat &a = q.a[i], &b = q.b[i];
        if (a.p && !host::encode_rows(&la.maps.a[i], ot, a.p, a.rows, a.cols, a.ld, am ? 64 : BLOCK_M))
            return TG_ERR_INVALID_VALUE;
        if (b.p && !host::encode_rows(&la.maps.b[i], ot, b.p, b.rows, b.cols, b.ld, b_box))
            return TG_ERR_INVALID_VALUE;
    }
    MlpParams &p = la.p;
    for (int i = 0; i < 3; ++i) {
        p.out[i].ptr = const_cast<void *>(q.out[i].p);
        p.out[i].ld = q.out[i].ld;
        p.out[i].tma = q.out[i].p && aligned16(q.out[i]) &&
                       host::encode_rows(&la.maps.out[i], q.out_f32 ? TG_OUT_F32 : ot, q.out[i].p,
                                         q.out[i].rows, q.out[i].cols, q.out[i].ld, 32, 64);
    }
    p.clip = (q.n * (q.out_f32 ? 4 : 2)) % 16 == 0;
    p.r = q.r.p;
    p.ldr = q.r.ld;
    p.r_tma = q.r.p && aligned16(q.r) &&
              host::encode_rows(&la.maps.r, ot, q.r.p, q.r.rows, q.r.cols, q.r.ld, 32, 64);
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
    p.gate = q.gate;
    p.late_wait = q.gate && q.op == MlpOp::WGRAD;
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

// K blocks a CTA's share spans at least: below that the join, whose reads grow
// with the tokens, costs more than the loads it spreads (60 x 1216 x 2560: 11.0
// us, 12.4 at 4 blocks; 30 tokens 9.8, 10.0).
int64_t stream_min_blocks(int nt) { return nt <= 16 ? 4 : nt <= 32 ? 6 : 8; }

struct StreamPlan {
    int nt;  // token columns of the MMA
    int64_t tiles, k_blocks;
    int grid;
};
StreamPlan plan_stream(const Product &q, int sms) {
    StreamPlan s;
    s.nt = q.m <= 16 ? 16 : q.m <= 32 ? 32 : 64;
    s.tiles = div_up(q.n, BLOCK_M);
    s.k_blocks = div_up(q.k[0], 64) + div_up(q.k[1], 64);
    int64_t grid = s.tiles * s.k_blocks / stream_min_blocks(s.nt);
    const int64_t cap = sms < 512 ? sms : 512;
    if (grid > cap) grid = cap;
    s.grid = (int)(grid < 1 ? 1 : grid);
    return s;
}

tg_status run_stream(const Product &q, tg_dtype t, const Device &dev, cudaStream_t stream) {
    const StreamPlan plan = plan_stream(q, dev.sms);
    StreamLaunch la;
    std::memset(&la, 0, sizeof(la));
    la.op = q.op == MlpOp::GATED   ? StreamOp::GATED
            : q.op == MlpOp::DGRAD ? StreamOp::DGRAD
                                   : StreamOp::LINEAR;
    la.nt = plan.nt;
    la.grid = plan.grid;
    const tg_out_dtype ot = out_type(t);
    // Weights: 128-row boxes, or 64 x 64 ones where they are read transposed.
    const int box = q.op == MlpOp::DGRAD ? 64 : BLOCK_M;
    for (int i = 0; i < 2; ++i) {
        if (i > 0 && !q.b[i].p) break;
        const Mat &a = q.a[i].p ? q.a[i] : q.a[0];
        if (!host::encode_rows(&la.maps.w[i], ot, q.b[i].p, q.b[i].rows, q.b[i].cols, q.b[i].ld, box) ||
            !host::encode_rows(&la.maps.x[i], ot, a.p, a.rows, a.cols, a.ld, la.nt))
            return TG_ERR_INVALID_VALUE;
    }
    StreamParams &p = la.p;
    p.tokens = (int32_t)q.m;
    p.features = (int32_t)q.n;
    p.tiles = (int32_t)plan.tiles;
    p.k_blocks0 = (int32_t)div_up(q.k[0], 64);
    p.num_k_blocks = (int32_t)plan.k_blocks;
    p.act = q.act;
    p.bias = q.bias;
    p.r = q.r.p;
    p.ldr = q.r.ld;
    for (int i = 0; i < 3; ++i) {
        p.out[i].ptr = const_cast<void *>(q.out[i].p);
        p.out[i].ld = q.out[i].ld;
    }
    host::Scratch w;
    const tg_status st = host::scratch(dev, stream, div_up(dev.sms, 2), &w);
    if (st != TG_OK) return st;
    p.ws = w.ws;
    p.flags = w.stream_flags;
    p.gate = q.gate;
    p.status = dev.status;
    p.wait_limit_ns = dev.wait_limit_ns;
    la.device = dev.id;
    la.stream = stream;
    const cudaError_t e = t == TG_BF16 ? launch_stream_bf16(la) : launch_stream_fp16(la);
    return e == cudaSuccess ? TG_OK : TG_ERR_CUDA;
}

// A weight gradient that needs no workspace (no split tiles, no tickets) may
// run beside the input gradient, which may be using it.
bool runs_beside(const TilePlan &w) { return w.split_max == 1 && !w.ticket; }

// The input gradient, then the weight gradient (either may be missing).
tg_status run_gradients(Product *x, Product *w, tg_dtype t, const Device &dev, cudaStream_t stream) {
    Beside both;
    TilePlan wp = {};
    if (w) {
        if (x) both = plan_beside(*x, *w, dev.sms);
        wp = both.on ? both.w : plan_tiles(*w, dev.sms);
        // (a captured stream that has no workspace yet goes without the gate: the
        // weight gradient then waits its turn)
        const int64_t room = div_up(dev.sms, 2);
        if (x && runs_beside(wp) && !host::scratch_blocked(dev, stream, room)) {
            host::Scratch s;
            const tg_status st = host::scratch(dev, stream, room, &s);
            if (st != TG_OK) return st;
            x->gate = w->gate = s.gate;
        }
    }
    tg_status st = x ? run_product(*x, t, dev, stream, both.on ? &both.x : nullptr) : TG_OK;
    if (st == TG_OK && w) st = run_product(*w, t, dev, stream, &wp);
    return st;
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
    RowWork work(dev.sms);
    for (int i = 0; i < count; ++i)
        if (moved[i]) work.repack(from[i], *ops[i]);
    TG_TRY(work.launch(dtype, stream));
    q.op = op;
    q.m = M;
    q.n = N;
    q.k[0] = K;
    q.entries = 1;
    q.a[0] = x;
    q.b[0] = w;
    q.b[1] = w2;
    return run_product(q, dtype, dev, stream);
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
LinearSpace linear_space(int64_t M, int64_t N, const Mat &dy, const Mat &x, const Mat &w,
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
        s.bands = row_bands(M, N, sms);
        s.partial = static_cast<float *>(s.arena.take(4 * N * s.bands));
    }
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
    return linear_space(M, N, mat(dY, lddy, M, N), mat(X, ldx, M, K), mat(W, ldw, N, K),
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
    LinearSpace s = linear_space(M, N, dy, x, w, act != TG_ACT_NONE, dx, dw, sum, dev.sms, workspace);
    if (!space_ok(s.arena, workspace, workspace_bytes)) return TG_ERR_INVALID_VALUE;
    RowWork work(dev.sms);
    if (s.dz_made || s.partial) {
        RowJob &p = work.add(M, N);
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
    }
    if (s.w_moved) work.repack(w, s.w);
    if (s.x_moved) work.repack(x, s.x);
    TG_TRY(work.launch(dtype, stream));
    Product qx = {}, qw = {};
    qx.op = MlpOp::DGRAD;
    qx.m = M;
    qx.n = K;
    qx.k[0] = N;
    qx.entries = 1;
    qx.a[0] = s.dz;
    qx.b[0] = s.w;
    qx.out[0] = mat(dX, lddx, M, K);
    qw.op = MlpOp::WGRAD;
    qw.m = N;
    qw.n = K;
    qw.k[0] = M;
    qw.entries = 1;
    qw.a[0] = s.dz;
    qw.b[0] = s.x;
    qw.out[0] = mat(dW, lddw, N, K, ew);
    qw.out_f32 = dw_dtype == TG_OUT_F32;
    st = run_gradients(dx ? &qx : nullptr, dw ? &qw : nullptr, dtype, dev, stream);
    if (st != TG_OK) return st;
    if (sum)
        TG_TRY(host::colsum_finish(s.partial, nullptr, (int32_t)s.bands, N, db, nullptr, stream));
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
    RowWork work(dev.sms);
    if (M > 0 && N > 0) {
        RowJob &p = work.add(M, N);
        p.gated = 1;
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
    }
    if (s.wg_moved) work.repack(wg, s.wg);
    if (s.wu_moved) work.repack(wu, s.wu);
    if (s.x_moved) work.repack(x, s.x);
    TG_TRY(work.launch(dtype, stream));
    Product qx = {}, qw = {};
    qx.op = MlpOp::DGRAD;
    qx.m = M;
    qx.n = K;
    qx.k[0] = qx.k[1] = N;
    qx.entries = 1;
    qx.a[0] = s.dg;
    qx.a[1] = s.du;
    qx.b[0] = s.wg;
    qx.b[1] = s.wu;
    qx.out[0] = mat(dX, lddx, M, K);
    qw.op = MlpOp::WGRAD;
    qw.m = N;
    qw.n = K;
    qw.k[0] = M;
    qw.entries = dWg && dWu ? 2 : 1;
    qw.a[0] = dWg ? s.dg : s.du;
    qw.a[1] = s.du;
    qw.b[0] = s.x;
    qw.out[0] = dWg ? mat(dWg, lddwg, N, K, ew) : mat(dWu, lddwu, N, K, ew);
    if (qw.entries == 2) qw.out[1] = mat(dWu, lddwu, N, K, ew);
    qw.out_f32 = dw_dtype == TG_OUT_F32;
    return run_gradients(dx ? &qx : nullptr, dw ? &qw : nullptr, dtype, dev, stream);
}

// ------------------------------------------------------------------ the planner's choice as text

namespace {

Product shape_of(MlpOp op, int64_t m, int64_t n, int64_t k0, int64_t k1, int entries) {
    Product q = {};
    q.op = op;
    q.m = m;
    q.n = n;
    q.k[0] = k0;
    q.k[1] = k1;
    q.entries = entries;
    return q;
}

}  // namespace

extern "C" tg_status tg_product_plan_describe(tg_product product, int64_t M, int64_t N, int64_t K,
                                              int32_t num_sms, char *buf, size_t len) {
    if (!buf || len == 0) return TG_ERR_INVALID_VALUE;
    buf[0] = '\0';
    if (!dims_ok(M, N, K) || (int)product < 0 || (int)product > (int)TG_PRODUCT_GATED_DW)
        return TG_ERR_INVALID_VALUE;
    int sms = num_sms;
    if (sms <= 0) {
        Device dev;
        const tg_status st = host::device(&dev);
        if (st != TG_OK) return st;
        sms = dev.sms;
    }
    const bool gated = product == TG_PRODUCT_GATED || product == TG_PRODUCT_GATED_DX || product == TG_PRODUCT_GATED_DW;
    const bool dw = product == TG_PRODUCT_LINEAR_DW || product == TG_PRODUCT_GATED_DW;
    const bool dx = product == TG_PRODUCT_LINEAR_DX || product == TG_PRODUCT_GATED_DX;
    const Product x = shape_of(MlpOp::DGRAD, M, K, N, gated ? N : 0, 1);
    const Product w = shape_of(MlpOp::WGRAD, N, K, M, 0, gated ? 2 : 1);
    const Product y = shape_of(gated ? MlpOp::GATED : MlpOp::LINEAR, M, N, K, 0, 1);
    const Product &q = dw ? w : dx ? x : y;
    int n;
    if (q.m == 0 || q.n == 0) {
        n = std::snprintf(buf, len, "empty");
    } else if (streams(q)) {
        const StreamPlan s = plan_stream(q, sms);
        n = std::snprintf(buf, len, "stream 128x%d tiles=%lld k_blocks=%lld grid=%d", s.nt,
                          (long long)s.tiles, (long long)s.k_blocks, s.grid);
    } else {
        const bool both = (dw || dx) && M > 0 && N > 0 && K > 0;
        Beside b;
        if (both) b = plan_beside(x, w, sms);
        const TilePlan p = b.on ? (dw ? b.w : b.x) : plan_tiles(q, sms);
        const TilePlan wp = b.on ? b.w : plan_tiles(w, sms);
        const int64_t teams = sms / p.cg > 0 ? sms / p.cg : 1;
        n = std::snprintf(buf, len,
                          "%s %dx%d tiles=%lld k_blocks=%lld grid=%d raster=%d split=%lldx%d schedule=%s "
                          "beside=%d",
                          p.cg == 2 ? "pair" : "single", 128 * p.cg, p.block_n, (long long)p.tiles,
                          (long long)(div_up(q.k[0], 64) + div_up(q.k[1], 64)), p.grid, p.group,
                          (long long)(p.split_max > 1 ? p.tiles % teams : 0), p.split_max,
                          p.ticket ? "ticket" : "static", both && runs_beside(wp) ? 1 : 0);
    }
    return (n >= 0 && (size_t)n < len) ? TG_OK : TG_ERR_INVALID_VALUE;
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
