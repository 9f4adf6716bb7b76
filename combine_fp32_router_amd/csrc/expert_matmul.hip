// The experts' products and their gradients: one matrix product per
// contiguous run of rows (moe_recv.h's grouped buffer), all runs in one launch.
//
//   forward   z = x W_e^T + b_e,  y = act(z) + residual
//   dx        g = dy W_e,         dx = act'(z_prev) g
//   dw        dW_e = dy_e^T x_e,  db_e = column sums of dy_e
//
// Each is a tile of outputs, C[row, col] = sum_r Q[row, r] P[col, r], with
// `col` the output's contiguous dimension.  The MFMA's first operand is P, so
// a lane ends with four consecutive columns of one row and stores them at
// once.  An operand lies in memory with r contiguous (x, dy, and W in the
// forward pass) or with its own index contiguous (W in dx, both in dw).
#include "expert_tile.hpp"
#include "launch.hpp"

namespace moe {
namespace {

enum Op { kForward, kDx, kDw };

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
};

constexpr int kFrags = 8;  // column blocks of 16 that a wave finishes of a row, four columns a lane

__device__ __forceinline__ f32x4 load4(const uint16_t *p)
{
    const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
    return f32x4{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
}
__device__ __forceinline__ void store4(uint16_t *p, f32x4 f)
{
    *reinterpret_cast<u32x2 *>(p) = u32x2{pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w)};
}

// One row of the forward product: v[i] has columns c + 16 i .. + 3 (i < n
// inside), GATED: v[4 i + j] of the gate and v[4 i + 2 + j] of the up half
// columns c + 32 i + 16 j.
template <bool GATED>
__device__ __forceinline__ void finish_forward(const Args &a, int e, int64_t row, int c, int n,
                                               f32x4 (&v)[kFrags])
{
    constexpr int wide = GATED ? 2 : 1;
    if (a.bias) {
        const float *b = a.bias + static_cast<int64_t>(e) * wide * a.C + c;
#pragma unroll
        for (int i = 0; i < kFrags; ++i) {
            const int o = GATED ? i / 4 * 32 + i % 2 * 16 : i * 16;
            if (o < n)
                v[i] += *reinterpret_cast<const f32x4 *>(b + o + (GATED ? i / 2 % 2 * a.C : 0));
        }
    }
    if (a.preact) {
        uint16_t *z = a.preact + row * wide * a.C + c;
#pragma unroll
        for (int i = 0; i < kFrags; ++i) {
            const int o = GATED ? i / 4 * 32 + i % 2 * 16 : i * 16;
            if (o < n)
                store4(z + o + (GATED ? i / 2 % 2 * a.C : 0), v[i]);
        }
    }
    if (GATED) {
#pragma unroll
        for (int i = 0; i < kFrags; ++i)
            if (i / 2 % 2 == 0)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[i][j] = v[i][j] * sigmoid(v[i][j]) * v[i + 2][j];
    } else {
        apply_act(v, a.act);
    }
    uint16_t *out = static_cast<uint16_t *>(a.out) + row * a.C + c;
    if (a.residual) {
        const uint16_t *res = a.residual + row * a.C + c;
#pragma unroll
        for (int i = 0; i < kFrags; ++i) {
            const int o = GATED ? i / 4 * 32 + i % 2 * 16 : i * 16;
            if ((!GATED || i / 2 % 2 == 0) && o < n)
                v[i] += load4(res + o);
        }
    }
#pragma unroll
    for (int i = 0; i < kFrags; ++i) {
        const int o = GATED ? i / 4 * 32 + i % 2 * 16 : i * 16;
        if ((!GATED || i / 2 % 2 == 0) && o < n)
            store4(out + o, v[i]);
    }
}

__device__ __forceinline__ void finish_dx(const Args &a, int64_t row, int c, int n, f32x4 (&v)[kFrags])
{
    uint16_t *out = static_cast<uint16_t *>(a.out);
    if (a.act == MOE_ACT_SWIGLU) {
        const int64_t at = row * 2 * a.C + c;
#pragma unroll
        for (int i = 0; i < kFrags; ++i)
            if (i * 16 < n) {
                const f32x4 g = load4(a.z + at + i * 16), u = load4(a.z + at + a.C + i * 16);
                f32x4 dg, du;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float s = sigmoid(g[j]);
                    dg[j] = v[i][j] * u[j] * (s * (1.0f + g[j] * (1.0f - s)));
                    du[j] = v[i][j] * (g[j] * s);
                }
                store4(out + at + i * 16, dg);
                store4(out + at + a.C + i * 16, du);
            }
        return;
    }
    const int64_t at = row * a.C + c;
    if (a.act != MOE_ACT_NONE) {
        f32x4 z[kFrags];
#pragma unroll
        for (int i = 0; i < kFrags; ++i)
            z[i] = i * 16 < n ? load4(a.z + at + i * 16) : f32x4{};
        apply_slope(v, z, a.act);
    }
#pragma unroll
    for (int i = 0; i < kFrags; ++i)
        if (i * 16 < n)
            store4(out + at + i * 16, v[i]);
}

__device__ __forceinline__ void finish_dw(const Args &a, int e, int64_t row, int c, int n, f32x4 (&v)[kFrags])
{
    const int64_t at = (static_cast<int64_t>(e) * a.rows + row) * a.C + c;
    if (a.flags & MOE_GRAD_BF16) {
#pragma unroll
        for (int i = 0; i < kFrags; ++i)
            if (i * 16 < n)
                store4(static_cast<uint16_t *>(a.out) + at + i * 16, v[i]);
        return;
    }
    f32x4 *o = reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + at);
    if (a.flags & MOE_GRAD_ACCUMULATE)
#pragma unroll
        for (int i = 0; i < kFrags; ++i)
            if (i * 16 < n)
                v[i] += o[i * 4];
#pragma unroll
    for (int i = 0; i < kFrags; ++i)
        if (i * 16 < n)
            o[i * 4] = v[i];
}

// One tile of a workgroup's list.
struct Work {
    int e;           // expert
    int first, n;    // its rows of the output
    int c0;          // its first output column
    int r_first, R;  // dw: the expert's run
};

// The tiles of a call, in the order in which they are handed out: workgroup b
// takes entries b, b + gridDim.x, ...  Entry j runs on XCD j % 8, so every
// list is dealt out in eight contiguous parts (xcd_order).  forward, dx: the
// whole tiles of all runs, then the runs' short ends, which fill up the last
// round.  dw: expert after expert, the longest runs first.
template <Op OP, int ROWS, int COLS>
struct TileList {
    int32_t *table;  // LDS: [E] upto of the whole tiles, [E] of the ends (dw: [E] experts in order)
    int whole, ends, col_tiles, row_tiles;

    __device__ __forceinline__ void build(const Args &a, int32_t *lds)
    {
        table = lds;
        col_tiles = (a.C + COLS - 1) / COLS;
        row_tiles = (a.rows + ROWS - 1) / ROWS;  // dw
        const int w = threadIdx.x / kWave, lane = lane_id();
        if (OP == kDw) {
            if (a.E <= kWave && w == 0) {
                const int n = lane < a.E ? expert_run(a.offsets, lane, a.max_rows).n : -1;
                int rank = 0;
                for (int j = 0; j < a.E; ++j) {
                    const int m = lane_value(n, j);
                    rank += m > n || (m == n && j < lane);
                }
                if (lane < a.E)
                    table[rank] = lane;
            } else if (a.E > kWave) {
                for (int e = threadIdx.x; e < a.E; e += blockDim.x)
                    table[e] = e;
            }
        } else if (w < 2) {
            int32_t *upto = table + w * a.E;
            int before = 0;
            for (int e0 = 0; e0 < a.E; e0 += kWave) {
                const int e = e0 + lane;
                const int n = e < a.E ? expert_run(a.offsets, e, a.max_rows).n : 0;
                const int sum = before + wave_inclusive_scan(w == 0 ? n / ROWS : (n % ROWS != 0));
                if (e < a.E)
                    upto[e] = sum;
                before = lane_value(sum, kWave - 1);
            }
        }
        __syncthreads();
        if (OP == kDw) {
            whole = ends = 0;
        } else {
            whole = static_cast<int>(uniform(table[a.E - 1]));
            ends = static_cast<int>(uniform(table[2 * a.E - 1]));
        }
    }

    // Expert of entry k of a list whose counts add up to upto[].
    __device__ __forceinline__ int expert_of(const int32_t *upto, int E, int k) const
    {
        int e = 0;
        for (int e0 = 0; e0 < E; e0 += kWave) {
            const int at = e0 + lane_id();
            e += __builtin_popcountll(__ballot(at < E && upto[at] <= k));
        }
        return static_cast<int>(uniform(e));
    }

    // Moves j to the next entry with work; false at the end of the list.
    __device__ __forceinline__ bool next(const Args &a, int64_t &j, Work &t) const
    {
        const int64_t per = static_cast<int64_t>(row_tiles) * col_tiles, per8 = (per + 7) / 8 * 8;
        const int64_t nw = static_cast<int64_t>(whole) * col_tiles, ne = static_cast<int64_t>(ends) * col_tiles;
        const int64_t nw8 = (nw + 7) / 8 * 8, end = OP == kDw ? per8 * a.E : nw8 + (ne + 7) / 8 * 8;
        for (; j < end; j += gridDim.x) {
            if (OP == kDw) {
                const int64_t id = xcd_order(j % per8, per);
                if (id < 0)
                    continue;
                t.e = static_cast<int>(uniform(table[j / per8]));
                const TileAt at = grouped_order(id, row_tiles, col_tiles);
                const ExpertRun run = expert_run(a.offsets, t.e, a.max_rows);
                t.first = at.row * ROWS;
                t.n = min(ROWS, a.rows - t.first);
                t.c0 = at.col * COLS;
                t.r_first = run.first;
                t.R = run.n;
            } else {
                const bool end_tile = j >= nw8;
                const int64_t id = end_tile ? xcd_order(j - nw8, ne) : xcd_order(j, nw);
                if (id < 0)
                    continue;
                const TileAt at = grouped_order(id, end_tile ? ends : whole, col_tiles);
                const int32_t *upto = table + (end_tile ? a.E : 0);
                t.e = expert_of(upto, a.E, at.row);
                const ExpertRun run = expert_run(a.offsets, t.e, a.max_rows);
                const int before = t.e ? static_cast<int>(uniform(upto[t.e - 1])) : 0;
                const int in_run = end_tile ? run.n / ROWS * ROWS : (at.row - before) * ROWS;
                t.first = run.first + in_run;
                t.n = min(ROWS, run.n - in_run);
                t.c0 = at.col * COLS;
                t.R = a.R;
            }
            return true;
        }
        return false;
    }
};

template <Op OP, bool GATED>
__global__ __launch_bounds__(64 * kTileWaves) void expert_kernel(Args a)
{
    typedef Tile<OP == kForward, OP != kDw, GATED> T;
    constexpr int kCols = GATED ? T::kCols / 2 : T::kCols;  // output columns of a tile
    // one array: for two the compiler would wait for all loads before a read
    __shared__ __align__(1024) char shared[T::kLdsBytes + 8 * MOE_MAX_EXPERTS];
    MOE_LDS char *lds = (MOE_LDS char *)shared;
    TileList<OP, T::kRows, kCols> list;
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

    int64_t j = blockIdx.x;
    Work k;
    if (!list.next(a, j, k))
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
        j += gridDim.x;
        const bool more = list.next(a, j, after);
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
        t.finish(k.n, [&](int row, int col, f32x4 (&v)[kFrags]) {
            const int c = GATED ? k.c0 + (col - col % 16) / 2 + col % 16 : k.c0 + col;
            const int n = a.C - (c - col % 16);  // columns inside, from the wave's first
            if (OP == kForward)
                finish_forward<GATED>(a, k.e, k.first + row, c, n, v);
            else if (OP == kDx)
                finish_dx(a, k.first + row, c, n, v);
            else
                finish_dw(a, k.e, k.first + row, c, n, v);
        });
        if (!more)
            return;
        k = after;
    }
}

int64_t tiles(int64_t n, int t) { return (n + t - 1) / t; }

// Workgroups of a call of at most n tiles: one for each of the card's 256
// CUs, whose LDS it fills, each with a list of tiles.
unsigned grid_for(int64_t n) { return static_cast<unsigned>(n < 256 ? n : 256); }

}  // namespace

hipError_t launch_expert_matmul(const void *x, const int32_t *offsets, const void *w,
                                const float *bias, int act, const void *residual, int E,
                                int64_t max_rows, int K, int N, void *out, void *preact,
                                hipStream_t stream)
{
    Args a{};
    a.p = static_cast<const uint16_t *>(w);
    a.q = static_cast<const uint16_t *>(x);
    a.offsets = offsets, a.E = E, a.max_rows = static_cast<int>(max_rows), a.R = K, a.C = N;
    a.act = act, a.bias = bias, a.residual = static_cast<const uint16_t *>(residual);
    a.out = out, a.preact = static_cast<uint16_t *>(preact);
    // spare entries: each of the two lists is a whole number for each XCD
    const int64_t rt = max_row_tiles(max_rows, E, 256);
    if (act == MOE_ACT_SWIGLU)
        expert_kernel<kForward, true><<<grid_for(rt * tiles(N, 128) + 14), 64 * kTileWaves, 0, stream>>>(a);
    else
        expert_kernel<kForward, false><<<grid_for(rt * tiles(N, 256) + 14), 64 * kTileWaves, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_expert_matmul_dx(const void *dy, const int32_t *offsets, const void *w, int act,
                                   const void *z, int E, int64_t max_rows, int K, int N, void *dx,
                                   hipStream_t stream)
{
    Args a{};
    a.p = static_cast<const uint16_t *>(w);
    a.q = static_cast<const uint16_t *>(dy);
    a.offsets = offsets, a.E = E, a.max_rows = static_cast<int>(max_rows), a.R = N, a.C = K;
    a.act = act, a.z = static_cast<const uint16_t *>(z), a.out = dx;
    const int64_t rt = max_row_tiles(max_rows, E, 256);
    expert_kernel<kDx, false><<<grid_for(rt * tiles(K, 256) + 14), 64 * kTileWaves, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_expert_matmul_dw(const void *dy, const void *x, const int32_t *offsets, int E,
                                   int64_t max_rows, int K, int N, int flags, void *dw, float *db,
                                   hipStream_t stream)
{
    Args a{};
    a.p = static_cast<const uint16_t *>(x);
    a.q = static_cast<const uint16_t *>(dy);
    a.offsets = offsets, a.E = E, a.max_rows = static_cast<int>(max_rows), a.C = K, a.rows = N;
    a.out = dw, a.db = db, a.flags = flags;
    const int64_t n = E * ((tiles(K, 256) * tiles(N, 256) + 7) / 8 * 8);
    expert_kernel<kDw, false><<<grid_for(n), 64 * kTileWaves, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace moe
