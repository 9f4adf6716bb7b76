// The experts' products and their gradients: one matrix product per
// contiguous run of rows (moe_recv.h's grouped buffer), all runs in one launch.
//
//   forward   z = x W_e^T + b_e,  y = act(z) + residual
//   dx        g = dy W_e,         dx = act'(z_prev) g
//   dw        dW_e = dy_e^T x_e,  db_e = column sums of dy_e
//
// Large calls are bound by the matrix cores at the clock that the card's power
// leaves (one run of 8192 rows, 8192 x 7168: 735 us, 1.31 PFLOP/s), small ones by
// reading the weights, and small dw by writing them.  Eight uneven runs of 16384
// rows: K = 7168, N = 2048 gated, z kept, 810 us, 1.19 PFLOP/s; dx of N = 7168, K =
// 2048 through SwiGLU 485, its dw 445, 1.0 and 1.1 PFLOP/s.  64 uneven runs of 4099
// rows, K = 1024, N = 4096, bias and residual: 138 us, 4.4 TB/s.  dw in bf16 takes
// 0.8 to 0.9 of its fp32 time, accumulated 0.9 to 1.1 of it.  Where
// all tiles fit the card at once a call takes one tile's time: 8 uneven runs of
// 8192 rows, K = 768, N = 2048: dx 44 us, dw 46.
//
// Each is a tile of outputs, C[row, col] = sum_r Q[row, r] P[col, r], with
// `col` the output's contiguous dimension.  The MFMA's first operand is P, so
// a lane ends with four consecutive columns of one row and stores them at
// once.  An operand lies in memory with r contiguous (x, dy, and W in the
// forward pass) or with its own index contiguous (W in dx, both in dw).
#include "expert_finish.hpp"
#include "expert_list.hpp"
#include "expert_tile.hpp"
#include "launch.hpp"

namespace moe {
namespace {

constexpr int kPartExperts = 256;   // (PartList)

struct Args {
    const uint16_t *p, *q;  // operands as above
    const int32_t *offsets;
    int E, max_rows;
    int R, C;               // reduced length (forward K, dx N), columns of one half of the output
    int act;
    const float *bias;
    const uint16_t *residual, *z;
    void *out;
    uint16_t *preact;
    float *db;
    int flags;
    int rows;               // dw: rows of the output (N)
    int height;             // forward, dx: rows of a tile
    // in parts: how many, their sums in the MFMA's layout, those of db
    int parts, tiles;       // (tiles: the most that the workspace is for)
    f32x4 *part;
    float *part_db;
};

// Forward: bias, pre-activations, activation, residual.  GATED: blocks 0, 1, 4,
// 5 of v are the gate's, 2, 3, 6, 7 the up half's.
template <int FR, bool GATED>
struct FinishForward {
    static constexpr int kBlocks = GATED ? FR / 2 : FR, P = 2 * kBlocks;
    const Args &a;
    MOE_LDS char *lds;
    Pieces<P> out, res, pre, pre_up;
    f32x4 bias[FR];
    u32x4 ahead[P / 4];  // the residual's next 16 rows

    __device__ __forceinline__ FinishForward(const Args &a_, MOE_LDS char *lds_, int e, int first, int n, int c, int inside, int row)
        : a(a_), lds(lds_), out(a.out, first, n, a.C, 2, c, inside), res(a.residual ? a.residual : a.q, first, n, a.C, 2, c, inside),
          pre(a.preact ? a.preact : a.q, first, n, GATED ? 2 * a.C : a.C, 2, c, inside),
          pre_up(a.preact ? a.preact : a.q, first, n, GATED ? 2 * a.C : a.C, 2, GATED ? c + a.C : c, inside)
    {
        if (a.bias) {
            const float *b = a.bias + static_cast<int64_t>(e) * (GATED ? 2 : 1) * a.C + c + lane_id() / 16 * 4;
#pragma unroll
            for (int i = 0; i < FR; ++i) {
                const int o = GATED ? i / 4 * 32 + i % 2 * 16 : i * 16;
                bias[i] = f32x4{};
                if (o < inside)
                    bias[i] = *reinterpret_cast<const f32x4 *>(b + o + (GATED && i / 2 % 2 ? a.C : 0));
            }
        }
        if (a.residual)
            load(row);
    }
    __device__ __forceinline__ void load(int row)
    {
#pragma unroll
        for (int j = 0; j < P / 4; ++j)
            ahead[j] = res.load(row, j);
    }
    __device__ __forceinline__ void operator()(int row, int next, f32x4 (&v)[FR])
    {
        f32x4 y[kBlocks], add[kBlocks];
        if (a.residual) {
            to_blocks<P>(lds, ahead, add);
            load(next);  // in front of this block's stores: waiting for it is then not waiting for them
        }
        if (a.bias)
#pragma unroll
            for (int i = 0; i < FR; ++i)
                v[i] += bias[i];
        if constexpr (GATED) {
            f32x4 g[kBlocks], u[kBlocks];
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                g[i] = v[i / 2 * 4 + i % 2];
                u[i] = v[i / 2 * 4 + i % 2 + 2];
            }
            if (a.preact) {
                store_blocks<P>(lds, g, pre, row);
                store_blocks<P>(lds, u, pre_up, row);
            }
#pragma unroll
            for (int i = 0; i < 4 * kBlocks; ++i) {
                const float x = g[i / 4][i % 4];
                y[i / 4][i % 4] = x * sigmoid(x) * u[i / 4][i % 4];
            }
        } else {
            if (a.preact)
                store_blocks<P>(lds, v, pre, row);
            apply_act(v, a.act);
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
                y[i] = v[i];
        }
        if (a.residual)
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
                y[i] += add[i];
        store_blocks<P>(lds, y, out, row);
    }
};

// dx: through the activation that made the product's input.
template <int FR>
struct FinishDx {
    static constexpr int P = 2 * FR;
    const Args &a;
    MOE_LDS char *lds;
    const bool gated;
    Pieces<P> out, out_up, pre, pre_up;
    u32x4 ahead[P / 4], ahead_up[P / 4];

    __device__ __forceinline__ FinishDx(const Args &a_, MOE_LDS char *lds_, int first, int n, int c, int inside, int row)
        : a(a_), lds(lds_), gated(a_.act == MOE_ACT_SWIGLU), out(a.out, first, n, gated ? 2 * a.C : a.C, 2, c, inside),
          out_up(a.out, first, n, gated ? 2 * a.C : a.C, 2, gated ? c + a.C : c, inside),
          pre(a.z ? a.z : a.q, first, n, gated ? 2 * a.C : a.C, 2, c, inside),
          pre_up(a.z ? a.z : a.q, first, n, gated ? 2 * a.C : a.C, 2, gated ? c + a.C : c, inside)
    {
        load(row);
    }
    __device__ __forceinline__ void load(int row)
    {
        if (a.act == MOE_ACT_NONE)
            return;
#pragma unroll
        for (int j = 0; j < P / 4; ++j)
            ahead[j] = pre.load(row, j);
        if (gated)
#pragma unroll
            for (int j = 0; j < P / 4; ++j)
                ahead_up[j] = pre_up.load(row, j);
    }
    __device__ __forceinline__ void operator()(int row, int next, f32x4 (&v)[FR])
    {
        if (a.act != MOE_ACT_NONE) {
            f32x4 z[FR];
            to_blocks<P>(lds, ahead, z);
            if (gated) {
                f32x4 u[FR];
                to_blocks<P>(lds, ahead_up, u);
                load(next);
#pragma unroll
                for (int i = 0; i < 4 * FR; ++i) {
                    const float g = z[i / 4][i % 4], up = u[i / 4][i % 4], x = v[i / 4][i % 4], s = sigmoid(g);
                    v[i / 4][i % 4] = x * up * (s * (1.0f + g * (1.0f - s)));
                    u[i / 4][i % 4] = x * (g * s);
                }
                store_blocks<P>(lds, u, out_up, row);
            } else {
                load(next);
                apply_slope(v, z, a.act);
            }
        }
        store_blocks<P>(lds, v, out, row);
    }
};

template <int FR>
struct FinishDw {
    const Args &a;
    MOE_LDS char *lds;
    const bool half;
    Pieces<2 * FR> out;      // bf16: all columns
    Pieces<16> lower, upper;  // fp32: 64 columns each

    __device__ __forceinline__ FinishDw(const Args &a_, MOE_LDS char *lds_, int64_t first, int n, int c, int inside)
        : a(a_), lds(lds_), half((a_.flags & MOE_GRAD_BF16) != 0), out(a.out, first, n, a.C, 2, c, inside),
          lower(a.out, first, n, a.C, 4, c, inside), upper(a.out, first, n, a.C, 4, c + 64, inside - 64)
    {
    }
    __device__ __forceinline__ void operator()(int row, int, f32x4 (&v)[FR])
    {
        if (half) {
            store_blocks<2 * FR>(lds, v, out, row);
            return;
        }
        fp32_half(lds, lower, row, v[0], v[1], v[2], v[3]);
        if constexpr (FR == 8)
            fp32_half(lds, upper, row, v[4], v[5], v[6], v[7]);
    }
    __device__ __forceinline__ void fp32_half(MOE_LDS char *__restrict__ place, const Pieces<16> &to, int row,
                                              f32x4 v0, f32x4 v1, f32x4 v2, f32x4 v3) const
    {
        const f32x4 v[4] = {v0, v1, v2, v3};
        u32x4 old[4];
        if (a.flags & MOE_GRAD_ACCUMULATE)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                old[j] = to.load(row, j);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<MOE_LDS f32x4 *>(place + Place::whole(c)) = v[c];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f32x4 x = *reinterpret_cast<const MOE_LDS f32x4 *>(place + Place::piece<16>(j));
            if (a.flags & MOE_GRAD_ACCUMULATE)
                x += __builtin_bit_cast(f32x4, old[j]);
            to.store(row, j, __builtin_bit_cast(u32x4, x));
        }
    }
};

template <Op OP, bool GATED, int TILE_COLS>
__global__ __launch_bounds__(64 * kTileWaves) void expert_kernel(Args a)
{
    typedef Tile<TILE_COLS, OP == kForward, OP != kDw, GATED> T;
    constexpr int kCols = GATED ? T::kCols / 2 : T::kCols;  // output columns of a tile
    // one array: for two the compiler would wait for all loads before a read
    typedef TileList<OP, kCols, Args> List;
    __shared__ __align__(1024) char shared[T::kLdsBytes + List::kBytes];
    MOE_LDS char *lds = (MOE_LDS char *)shared;
    List list;
    list.build(a, reinterpret_cast<int32_t *>(shared + T::kLdsBytes));

    T t;
    auto start = [&](const Work &k) {  // the loads of a tile's first stages
        t.R = k.R;
        if (OP == kForward) {
            const int64_t rows = static_cast<int64_t>(k.e) * (GATED ? 2 : 1) * a.C + k.c0;
            t.p.init(a.p + rows * a.R, a.p + (rows + a.C) * a.R, a.R, min(kCols, a.C - k.c0));
        } else if (OP == kDx) {
            t.p.init(a.p + static_cast<int64_t>(k.e) * a.C * a.R + k.c0, nullptr, a.C, min(kCols, a.C - k.c0));
        } else {
            t.p.init(a.p + static_cast<int64_t>(k.r_first) * a.C + k.c0, nullptr, a.C, min(kCols, a.C - k.c0));
        }
        if (OP == kDw)
            t.q.init(a.q + static_cast<int64_t>(k.r_first) * a.rows + k.first, nullptr, a.rows, k.n);
        else
            t.q.init(a.q + static_cast<int64_t>(k.first) * a.R, nullptr, a.R, k.n);
        t.start_rows(k.n, lds);
    };

    int i = 0;
    Work k;
    if (!list.next(a, i, k))
        return;
    start(k);
    for (;;) {
        t.clear();
        const bool sums = OP == kDw && a.db && k.c0 == 0;
        if (sums)
            t.template run_rows<OP == kDw>(k.n, lds);
        else
            t.template run_rows<false>(k.n, lds);
        Work after = k;
        ++i;
        const bool more = list.next(a, i, after);
        if (more)
            start(after);  // runs beside the rest of this tile
        if (sums) {
            // lanes l, l + 16, l + 32 and l + 48 hold parts of row l's and row l + 16's sums
            const int lane = lane_id();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float sum[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    sum[h] = t.sum[b][h] + __shfl_xor(t.sum[b][h], 16);
                    sum[h] += __shfl_xor(sum[h], 32);
                }
                const int row = t.row0(t.wave() % 2 * 2 + b) + lane % 32;
                if (lane < 32 && row < k.n) {
                    float *db = a.db + static_cast<int64_t>(k.e) * a.rows + k.first + row;
                    *db = ((a.flags & MOE_GRAD_ACCUMULATE) ? *db : 0.0f) + sum[lane / 16];
                }
            }
        }
        const int c = k.c0 + t.col0() / (GATED ? 2 : 1), inside = a.C - c;
        MOE_LDS char *place = t.out_place(lds);
        if constexpr (OP == kForward) {
            FinishForward<T::kFrags, GATED> f(a, place, k.e, k.first, k.n, c, inside, t.row0(0));
            t.finish(k.n, f);
        } else if constexpr (OP == kDx) {
            FinishDx<T::kFrags> f(a, place, k.first, k.n, c, inside, t.row0(0));
            t.finish(k.n, f);
        } else {
            FinishDw<T::kFrags> f(a, place, static_cast<int64_t>(k.e) * a.rows + k.first, k.n, c, inside);
            t.finish(k.n, f);
        }
        if (!more)
            return;
        k = after;
    }
}

// Few outputs of a long reduced length: every tile, of 64 x 128, is
// shared by up to `parts` workgroups, each of which takes a piece of the
// length and leaves its sums, as its accumulators hold them, in the workspace; a
// second kernel adds them in order and finishes the tile.  Two workgroups
// share a CU (THIN).  dw of 16384 rows, 512 x 512: 23 us, 100 in whole tiles;
// 8192 rows, 128 x 2048: 19 and 54; dx of 512 rows, 8192 -> 256: 21 and 54.
template <Op OP, bool GATED>
struct PartList {
    static constexpr int kCols = GATED ? 64 : 128;  // output columns of a tile
    static constexpr int kBytes = 4 * (2 * kPartExperts + 1);
    int32_t *starts, *upto;  // as in TileList; upto: not for dw
    int E, tiles, col_tiles, row_tiles;

    __device__ __forceinline__ void build(const Args &a, int32_t *lds)
    {
        E = a.E;
        starts = lds;
        upto = lds + E + 1;
        col_tiles = (a.C + kCols - 1) / kCols;
        row_tiles = (a.rows + 63) / 64;  // dw
        for (int e = threadIdx.x; e <= E; e += blockDim.x)
            starts[e] = run_start(a.offsets, e, a.max_rows);
        __syncthreads();
        tiles = E * row_tiles * col_tiles;
        if (OP != kDw) {
            if (uniform(threadIdx.x / kWave) == 0) {
                int before = 0;
                for (int e0 = 0; e0 < E; e0 += kWave) {
                    const int e = e0 + lane_id();
                    const int sum = before + wave_inclusive_scan(e < E ? (run(e).n + 63) / 64 : 0);
                    if (e < E)
                        upto[e] = sum;
                    before = lane_value(sum, kWave - 1);
                }
            }
            __syncthreads();
            tiles = min(static_cast<int>(uniform(upto[E - 1])) * col_tiles, a.tiles);
        }
    }
    __device__ __forceinline__ ExpertRun run(int e) const
    {
        const int first = starts[e];
        return {first, max(starts[e + 1] - first, 0)};
    }
    __device__ __forceinline__ ExpertRun uniform_run(int e) const
    {
        const ExpertRun r = run(e);
        return {static_cast<int>(uniform(r.first)), static_cast<int>(uniform(r.n))};
    }
    __device__ __forceinline__ Work at(const Args &a, int tile) const
    {
        Work t;
        t.c0 = tile % col_tiles * kCols;
        const int row = tile / col_tiles;
        if (OP != kDw) {
            t.e = 0;
            for (int e0 = 0; e0 < E; e0 += kWave) {
                const int e = e0 + lane_id();
                t.e += __builtin_popcountll(__ballot(e < E && upto[e] <= row));
            }
            t.e = static_cast<int>(uniform(t.e));
            const ExpertRun r = uniform_run(t.e);
            const int in_run = (row - (t.e ? static_cast<int>(uniform(upto[t.e - 1])) : 0)) * 64;
            t.first = r.first + in_run;
            t.n = min(64, r.n - in_run);
            t.R = a.R;
        } else {
            t.e = row / row_tiles;
            const ExpertRun r = uniform_run(t.e);
            t.first = row % row_tiles * 64;
            t.n = min(64, a.rows - t.first);
            t.r_first = r.first;
            t.R = r.n;
        }
        return t;
    }
    // r of a tile's part
    static __device__ __forceinline__ int share(const Args &a, int R)
    {
        return ((R + kStep - 1) / kStep + a.parts - 1) / a.parts * kStep;
    }
};

template <Op OP, bool GATED>
__global__ __launch_bounds__(64 * kTileWaves, 2) void expert_part_kernel(Args a)
{
    typedef Tile<128, OP == kForward, OP != kDw, GATED, true> T;
    typedef PartList<OP, GATED> List;
    __shared__ __align__(1024) char shared[T::kLdsBytes + List::kBytes];
    MOE_LDS char *lds = (MOE_LDS char *)shared;
    List list;
    list.build(a, reinterpret_cast<int32_t *>(shared + T::kLdsBytes));
    T t;
    for (int j = blockIdx.x; j < list.tiles * a.parts; j += gridDim.x) {
        const int tile = j / a.parts, part = j % a.parts;
        const Work k = list.at(a, tile);
        const int share = List::share(a, k.R), r0 = part * share;
        if (r0 >= k.R)
            continue;
        t.R = min(share, k.R - r0);
        if (OP != kDw) {
            if (OP == kForward) {
                const int64_t rows = static_cast<int64_t>(k.e) * (GATED ? 2 : 1) * a.C + k.c0;
                t.p.init(a.p + rows * a.R + r0, a.p + (rows + a.C) * a.R + r0, a.R, min(List::kCols, a.C - k.c0));
            } else {
                t.p.init(a.p + (static_cast<int64_t>(k.e) * a.R + r0) * a.C + k.c0, nullptr, a.C, min(128, a.C - k.c0));
            }
            t.q.init(a.q + static_cast<int64_t>(k.first) * a.R + r0, nullptr, a.R, k.n);
        } else {
            t.p.init(a.p + (static_cast<int64_t>(k.r_first) + r0) * a.C + k.c0, nullptr, a.C, min(128, a.C - k.c0));
            t.q.init(a.q + (static_cast<int64_t>(k.r_first) + r0) * a.rows + k.first, nullptr, a.rows, k.n);
        }
        t.start_rows(k.n, lds);
        t.clear();
        const bool sums = OP == kDw && a.db && k.c0 == 0;
        if (sums)
            t.template run_rows<OP == kDw>(k.n, lds);
        else
            t.template run_rows<false>(k.n, lds);
        f32x4 *to = a.part + ((static_cast<int64_t>(tile) * a.parts + part) * kTileWaves + t.wave()) * (2 * T::kFrags * kWave) +
                    lane_id();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < T::kFrags; ++c)
                to[(i * T::kFrags + c) * kWave] = T::read_acc(t.acc[c][0][i]);
        if (sums && t.wave() % 2 == 0) {  // (as in expert_kernel)
            const int lane = lane_id();
            float sum[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                sum[h] = t.sum[0][h] + __shfl_xor(t.sum[0][h], 16);
                sum[h] += __shfl_xor(sum[h], 32);
            }
            if (lane < 32)
                a.part_db[(static_cast<int64_t>(tile / list.col_tiles) * a.parts + part) * 64 + t.row0(0) + lane] =
                    sum[lane / 16];
        }
    }
}

// One wave for each 16 rows that a wave of the parts' kernel held: most of it
// is waiting for the parts.
template <Op OP, bool GATED>
__global__ __launch_bounds__(kWave) void expert_join_kernel(Args a)
{
    constexpr int kFrags = 4, kUnits = 2 * kTileWaves, kUnit = kFrags * kWave;  // of a tile's part, in f32x4
    typedef PartList<OP, GATED> List;
    __shared__ __align__(1024) char shared[4096 + List::kBytes];
    List list;
    list.build(a, reinterpret_cast<int32_t *>(shared + 4096));
    const int tile = blockIdx.x / kUnits, unit = blockIdx.x % kUnits, wave = unit / 2, lane = lane_id();
    if (tile >= list.tiles)
        return;
    const Work k = list.at(a, tile);
    const int share = List::share(a, k.R), live = k.R > 0 ? (k.R + share - 1) / share : 0;
    if (OP == kDw && a.db && k.c0 == 0 && unit == 0 && lane < k.n) {
        float sum = 0.0f;
        for (int p = 0; p < live; ++p)
            sum += a.part_db[(static_cast<int64_t>(tile / list.col_tiles) * a.parts + p) * 64 + lane];
        float *db = a.db + static_cast<int64_t>(k.e) * a.rows + k.first + lane;
        *db = ((a.flags & MOE_GRAD_ACCUMULATE) ? *db : 0.0f) + sum;
    }
    const int row = wave / 2 * 32 + unit % 2 * 16, c = k.c0 + wave % 2 * (64 / (GATED ? 2 : 1)), inside = a.C - c;
    if (row >= k.n)
        return;
    const f32x4 *from = a.part + (static_cast<int64_t>(tile) * a.parts * kUnits + unit) * kUnit + lane;
    f32x4 v[kFrags] = {};
#pragma unroll 4
    for (int p = 0; p < live; ++p)
#pragma unroll
        for (int b = 0; b < kFrags; ++b)
            v[b] += from[p * (kUnits * kUnit) + b * kWave];
    MOE_LDS char *place = (MOE_LDS char *)shared;
    if constexpr (OP == kForward) {
        FinishForward<kFrags, GATED> f(a, place, k.e, k.first, k.n, c, inside, row);
        f(row, row, v);
    } else if constexpr (OP == kDx) {
        FinishDx<kFrags> f(a, place, k.first, k.n, c, inside, row);
        f(row, row, v);
    } else {
        FinishDw<kFrags> f(a, place, static_cast<int64_t>(k.e) * a.rows + k.first, k.n, c, inside);
        f(row, row, v);
    }
}

// In how many parts a tile's reduced length R is best taken (1: not at all): as
// many as fill the card, of at least four steps of 64 each, where they save 16
// steps or more, of about 0.45 us, against the 5 us of the second kernel.
int parts_of(int64_t tiles, int E, int64_t R)
{
    const int64_t steps = R / kStep;
    if (tiles < 1 || tiles > kCus / 2 || E > kPartExperts)
        return 1;
    const int64_t n = steps / 4 < 2 * kCus / tiles ? steps / 4 : 2 * kCus / tiles;
    return n >= 2 && steps - steps / n >= 16 ? static_cast<int>(n) : 1;
}
constexpr int64_t kPartBytes = 64 * 128 * 4, kPartDbBytes = 64 * 4;  // of a part of a tile, and of a row of tiles

// Workgroups of a call of at most n tiles: one for each of the card's 256
// CUs, whose LDS it fills, each with a list of tiles.  (Each of the two lists
// is a whole number for each XCD: spare entries.)
dim3 grid_for(int64_t n) { return dim3(static_cast<unsigned>(n + 14 < kCus ? (n + 14) / 8 * 8 : kCus)); }

#define MOE_EXPERT(OP, GATED, COLS, TILES)                                                     \
    if ((COLS) == 128)                                                                         \
        expert_kernel<OP, GATED, 128><<<grid_for(TILES), 64 * kTileWaves, 0, stream>>>(a);     \
    else                                                                                       \
        expert_kernel<OP, GATED, 256><<<grid_for(TILES), 64 * kTileWaves, 0, stream>>>(a)

}  // namespace

Parts row_parts(int E, int64_t max_rows, int R, int C, int unit)
{
    Parts g{};
    g.tiles = max_row_tiles(max_rows, E, 64) * ((C + unit - 1) / unit);
    g.parts = parts_of(g.tiles, E, R);
    g.bytes = g.parts > 1 ? g.tiles * g.parts * kPartBytes : 0;
    return g;
}

Parts forward_parts(int act, int E, int64_t max_rows, int K, int N)
{
    const Parts g = row_parts(E, max_rows, K, N, act == MOE_ACT_SWIGLU ? 64 : 128);
    return g.parts > 1 && !few_rows_pay(act, E, max_rows, K, N, g.parts) ? g : Parts{1, g.tiles, 0};
}

Parts dw_parts(int E, int64_t max_rows, int K, int N)
{
    Parts g{};
    const int64_t rows = static_cast<int64_t>(E) * ((N + 63) / 64);
    g.tiles = rows * ((K + 127) / 128);
    g.parts = parts_of(g.tiles, E, max_rows / E);
    g.bytes = g.parts > 1 ? g.parts * (g.tiles * kPartBytes + rows * kPartDbBytes) : 0;
    return g;
}

template <Op OP, bool GATED>
static hipError_t launch_parts(Args &a, const Parts &g, void *workspace, hipStream_t stream)
{
    a.parts = g.parts, a.tiles = static_cast<int>(g.tiles);
    a.part = static_cast<f32x4 *>(workspace);
    a.part_db = reinterpret_cast<float *>(static_cast<char *>(workspace) + g.tiles * g.parts * kPartBytes);
    const int64_t n = g.tiles * g.parts;
    expert_part_kernel<OP, GATED><<<dim3(static_cast<unsigned>(n < 2 * kCus ? n : 2 * kCus)), 64 * kTileWaves, 0, stream>>>(a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return err;
    expert_join_kernel<OP, GATED><<<dim3(static_cast<unsigned>(g.tiles * 2 * kTileWaves)), kWave, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_expert_matmul(const void *x, const int32_t *offsets, const void *w,
                                const float *bias, int act, const void *residual, int E,
                                int64_t max_rows, int K, int N, void *out, void *preact,
                                void *workspace, hipStream_t stream)
{
    Args a{};
    a.p = static_cast<const uint16_t *>(w);
    a.q = static_cast<const uint16_t *>(x);
    a.offsets = offsets, a.E = E, a.max_rows = static_cast<int>(max_rows), a.R = K, a.C = N;
    a.act = act, a.bias = bias, a.residual = static_cast<const uint16_t *>(residual);
    a.out = out, a.preact = static_cast<uint16_t *>(preact);
    const bool gated = act == MOE_ACT_SWIGLU;
    const Parts parts = forward_parts(act, E, max_rows, K, N);
    const bool shared = workspace && parts.parts > 1;
    if (!shared && few_rows_pay(act, E, max_rows, K, N, 1))
        return launch_expert_few(x, offsets, w, bias, act, residual, E, max_rows, K, N, out, preact, stream);
    if (shared)
        return gated ? launch_parts<kForward, true>(a, parts, workspace, stream)
                     : launch_parts<kForward, false>(a, parts, workspace, stream);
    const TileShape shape = tile_shape(E, max_rows, N, gated ? 64 : 128);
    a.height = shape.rows;
    if (gated) {
        MOE_EXPERT(kForward, true, shape.cols, shape.tiles);
    } else {
        MOE_EXPERT(kForward, false, shape.cols, shape.tiles);
    }
    return hipGetLastError();
}

hipError_t launch_expert_matmul_dx(const void *dy, const int32_t *offsets, const void *w, int act,
                                   const void *z, int E, int64_t max_rows, int K, int N, void *dx,
                                   void *workspace, hipStream_t stream)
{
    Args a{};
    a.p = static_cast<const uint16_t *>(w);
    a.q = static_cast<const uint16_t *>(dy);
    a.offsets = offsets, a.E = E, a.max_rows = static_cast<int>(max_rows), a.R = N, a.C = K;
    a.act = act, a.z = static_cast<const uint16_t *>(z), a.out = dx;
    const Parts parts = row_parts(E, max_rows, N, K, 128);
    if (workspace && parts.parts > 1)
        return launch_parts<kDx, false>(a, parts, workspace, stream);
    const TileShape shape = tile_shape(E, max_rows, K, 128);
    a.height = shape.rows;
    MOE_EXPERT(kDx, false, shape.cols, shape.tiles);
    return hipGetLastError();
}

hipError_t launch_expert_matmul_dw(const void *dy, const void *x, const int32_t *offsets, int E,
                                   int64_t max_rows, int K, int N, int flags, void *dw, float *db,
                                   void *workspace, hipStream_t stream)
{
    Args a{};
    a.p = static_cast<const uint16_t *>(x);
    a.q = static_cast<const uint16_t *>(dy);
    a.offsets = offsets, a.E = E, a.max_rows = static_cast<int>(max_rows), a.C = K, a.rows = N;
    a.out = dw, a.db = db, a.flags = flags;
    const Parts parts = dw_parts(E, max_rows, K, N);
    if (workspace && parts.parts > 1)
        return launch_parts<kDw, false>(a, parts, workspace, stream);
    const int64_t n = static_cast<int64_t>(E) * ((N + 255) / 256) * ((K + 255) / 256);  // cut into up to 4 each
    MOE_EXPERT(kDw, false, 2 * n <= kCus ? 128 : 256, 8 * n);
    return hipGetLastError();
}

}  // namespace moe
