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

constexpr int kOut = 8;  // columns of one row that a lane finishes at a time: 16 bytes of bf16

__device__ __forceinline__ void load_row8(const uint16_t *p, float f[kOut])
{
    unpack8(*reinterpret_cast<const u32x4 *>(p), f);
}
__device__ __forceinline__ void store_row8(uint16_t *p, const float f[kOut])
{
    *reinterpret_cast<u32x4 *>(p) = pack8(f);
}
__device__ __forceinline__ void add_bias(const float *b, float f[kOut])
{
    const float4 x = *reinterpret_cast<const float4 *>(b), y = *reinterpret_cast<const float4 *>(b + 4);
    f[0] += x.x, f[1] += x.y, f[2] += x.z, f[3] += x.w;
    f[4] += y.x, f[5] += y.y, f[6] += y.z, f[7] += y.w;
}

// Columns c.. of one row of the forward product; u: the up half (GATED).
template <bool GATED>
__device__ __forceinline__ void finish_forward(const Args &a, int e, int64_t row, int c, float v[kOut],
                                               float u[kOut])
{
    constexpr int wide = GATED ? 2 : 1;
    if (a.bias) {
        const float *b = a.bias + static_cast<int64_t>(e) * wide * a.C + c;
        add_bias(b, v);
        if (GATED)
            add_bias(b + a.C, u);
    }
    if (a.preact) {
        uint16_t *z = a.preact + row * wide * a.C + c;
        store_row8(z, v);
        if (GATED)
            store_row8(z + a.C, u);
    }
    float res[kOut] = {};
    if (a.residual)
        load_row8(a.residual + row * a.C + c, res);
#pragma unroll
    for (int i = 0; i < kOut; ++i)
        v[i] = (GATED ? v[i] * sigmoid(v[i]) * u[i] : act_value(v[i], a.act)) + res[i];
    store_row8(static_cast<uint16_t *>(a.out) + row * a.C + c, v);
}

__device__ __forceinline__ void finish_dx(const Args &a, int64_t row, int c, float v[kOut])
{
    uint16_t *out = static_cast<uint16_t *>(a.out);
    if (a.act == MOE_ACT_SWIGLU) {
        float g[kOut], u[kOut];
        load_row8(a.z + row * 2 * a.C + c, g);
        load_row8(a.z + row * 2 * a.C + a.C + c, u);
#pragma unroll
        for (int i = 0; i < kOut; ++i) {
            const float s = sigmoid(g[i]), dg = v[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
            u[i] = v[i] * g[i] * s;
            g[i] = dg;
        }
        store_row8(out + row * 2 * a.C + c, g);
        store_row8(out + row * 2 * a.C + a.C + c, u);
        return;
    }
    if (a.act != MOE_ACT_NONE) {
        float z[kOut];
        load_row8(a.z + row * a.C + c, z);
#pragma unroll
        for (int i = 0; i < kOut; ++i)
            v[i] *= act_slope(z[i], a.act);
    }
    store_row8(out + row * a.C + c, v);
}

__device__ __forceinline__ void finish_dw(const Args &a, int e, int64_t row, int c, float v[kOut])
{
    const int64_t at = (static_cast<int64_t>(e) * a.rows + row) * a.C + c;
    if (a.flags & MOE_GRAD_BF16) {
        store_row8(static_cast<uint16_t *>(a.out) + at, v);
        return;
    }
    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at);
    if (a.flags & MOE_GRAD_ACCUMULATE)
        add_bias(reinterpret_cast<const float *>(o), v);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
}

template <Op OP, bool GATED, int BR, int WR, int WC>
__global__ __launch_bounds__(64 * WR * WC) void expert_kernel(Args a)
{
    typedef Tile<BR, 256, WR, WC, OP == kForward, OP != kDw, GATED> T;
    __shared__ __align__(1024) char lds[2][T::kStageBytes];
    constexpr int kCols = GATED ? 128 : 256;  // output columns of a tile
    const int col_tiles = (a.C + kCols - 1) / kCols;

    RowTile tile;
    int c0, R = a.R;
    const uint16_t *p, *p2 = nullptr, *q;
    if (OP == kDw) {
        const int row_tiles = (a.rows + BR - 1) / BR, per = row_tiles * col_tiles;
        const int id = xcd_order(blockIdx.x, per * a.E);
        if (id < 0)
            return;
        tile.e = id / per;
        const TileAt at = grouped_order(id % per, row_tiles, col_tiles);
        tile.first = at.row * BR;
        tile.n = min(BR, a.rows - tile.first);
        c0 = at.col * kCols;
        const ExpertRun run = expert_run(a.offsets, tile.e, a.max_rows);
        R = run.n;
        p = a.p + static_cast<int64_t>(run.first) * a.C + c0;
        q = a.q + static_cast<int64_t>(run.first) * a.rows + tile.first;
    } else {
        const int row_tiles = count_row_tiles(a.offsets, a.E, a.max_rows, BR);
        const int id = xcd_order(blockIdx.x, row_tiles * col_tiles);
        if (id < 0)
            return;
        const TileAt at = grouped_order(id, row_tiles, col_tiles);
        tile = find_row_tile(a.offsets, a.E, a.max_rows, BR, at.row);
        c0 = at.col * kCols;
        q = a.q + static_cast<int64_t>(tile.first) * R;
        if (OP == kForward) {
            p = a.p + (static_cast<int64_t>(tile.e) * (GATED ? 2 : 1) * a.C + c0) * R;
            p2 = p + static_cast<int64_t>(a.C) * R;
        } else {
            p = a.p + static_cast<int64_t>(tile.e) * a.C * R + c0;
        }
    }
    const int ncols = min(kCols, a.C - c0);
    T t;
    t.init(p, p2, OP == kForward ? R : a.C, ncols, q, OP == kDw ? a.rows : R, tile.n, R);
    if (OP == kDw && a.db && c0 == 0) {
        t.template run<true>(lds);
        // every column of a block of sums holds the same value
        const int lane = lane_id(), block = t.wave() % WC;
        const int row = t.row0() + block * 32 + lane;
        if (block < T::kRowFrags && lane < 32 && row < tile.n) {
            float *db = a.db + static_cast<int64_t>(tile.e) * a.rows + tile.first + row;
            *db = ((a.flags & MOE_GRAD_ACCUMULATE) ? *db : 0.0f) + t.sums[0];
        }
    } else {
        t.run(lds);
    }
    t.finish(lds, [&](int row_in, int col, float v[kOut], float u[kOut]) {
        const int c = c0 + col;
        if (row_in >= tile.n || c >= a.C)
            return;
        if (OP == kForward)
            finish_forward<GATED>(a, tile.e, tile.first + row_in, c, v, u);
        else if (OP == kDx)
            finish_dx(a, tile.first + row_in, c, v);
        else
            finish_dw(a, tile.e, tile.first + row_in, c, v);
    });
}

int64_t tiles(int64_t n, int t) { return (n + t - 1) / t; }

// Blocks of a grid of `n` tiles, a whole number for each XCD.
unsigned grid_for(int64_t n) { return static_cast<unsigned>((n + 7) / 8 * 8); }

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
    const int64_t rt = max_row_tiles(max_rows, E, 256);
    if (act == MOE_ACT_SWIGLU)
        expert_kernel<kForward, true, 256, 2, 4><<<grid_for(rt * tiles(N, 128)), 512, 0, stream>>>(a);
    else
        expert_kernel<kForward, false, 256, 2, 4><<<grid_for(rt * tiles(N, 256)), 512, 0, stream>>>(a);
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
    expert_kernel<kDx, false, 256, 2, 4><<<grid_for(rt * tiles(K, 256)), 512, 0, stream>>>(a);
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
    const int64_t n = E * tiles(K, 256) * tiles(N, 256);
    expert_kernel<kDw, false, 256, 2, 4><<<grid_for(n), 512, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace moe
