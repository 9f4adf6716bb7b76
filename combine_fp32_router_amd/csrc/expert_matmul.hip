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
#include "expert_rows.hpp"
#include "launch.hpp"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kTile = 128, kStep = 32, kPitch = kStep + 8;

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

// Stages a [128 index][32 r] operand tile in LDS, zeros outside.
// CONTIG: memory is [index][r] with row pitch `pitch`, else [r][index].
template <bool CONTIG>
__device__ __forceinline__ void stage(uint16_t *lds, const uint16_t *src, int64_t pitch, int r0,
                                      int R, int i0, int n, int half, int wide)
{
    for (int v = threadIdx.x; v < kTile * kStep / 8; v += 256) {
        if (CONTIG) {
            const int i = v / 4, r = (v % 4) * 8;
            int row = i0 + i;
            bool in = i < n;
            if (wide == 2) {  // blocks of 32: gate, up, gate, up
                row = i0 + (i / 64) * 32 + i % 32;
                in = row < half;
                row += (i / 32 % 2) * half;
            }
            u32x4 x{0, 0, 0, 0};
            if (in && r0 + r < R)
                x = *reinterpret_cast<const u32x4 *>(src + row * pitch + r0 + r);
            *reinterpret_cast<u32x4 *>(lds + i * kPitch + r) = x;
        } else {
            const int r = v / 16, i = (v % 16) * 8;
            u32x4 x{0, 0, 0, 0};
            if (i < n && r0 + r < R)
                x = *reinterpret_cast<const u32x4 *>(src + (r0 + r) * pitch + i0 + i);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                lds[(i + j) * kPitch + r] = static_cast<uint16_t>(w[j / 2] >> (16 * (j % 2)));
        }
    }
}

__device__ __forceinline__ void load4(const uint16_t *p, float f[4])
{
    const u32x2 v = *reinterpret_cast<const u32x2 *>(p);
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
}
__device__ __forceinline__ void store4(uint16_t *p, const float f[4])
{
    *reinterpret_cast<u32x2 *>(p) = u32x2{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
}

template <Op OP>
__global__ __launch_bounds__(256) void expert_kernel(Args a)
{
    __shared__ uint16_t lp[kTile * kPitch], lq[kTile * kPitch];
    const int wide = a.act == MOE_ACT_SWIGLU ? 2 : 1;
    const int tile_cols = OP == kForward && wide == 2 ? kTile / 2 : kTile;
    RowTile tile;
    int R = a.R, c0 = (OP == kDw ? blockIdx.x : blockIdx.y) * tile_cols;
    int64_t run0 = 0;
    if (OP == kDw) {
        tile.e = blockIdx.z;
        tile.first = blockIdx.y * kTile;
        tile.n = min(kTile, a.rows - tile.first);
        const ExpertRun run = expert_run(a.offsets, tile.e, a.max_rows);
        R = run.n;
        run0 = run.first;
    } else {
        tile = find_row_tile(a.offsets, a.E, a.max_rows, kTile, blockIdx.x);
        if (tile.n <= 0)
            return;
    }
    const int ncols = min(tile_cols, a.C - c0);
    const int lane = lane_id(), w = threadIdx.x / kWave, wc = w % 2, wr = w / 2;
    f32x16 acc[2][2] = {};
    float colsum = 0.0f;
    for (int r0 = 0; r0 < R; r0 += kStep) {
        __syncthreads();
        if (OP == kForward) {
            stage<true>(lp, a.p + static_cast<int64_t>(tile.e) * wide * a.C * R, R, r0, R, c0, ncols, a.C, wide);
            stage<true>(lq, a.q, R, r0, R, tile.first, tile.n, 0, 1);
        } else if (OP == kDx) {
            stage<false>(lp, a.p + static_cast<int64_t>(tile.e) * a.C * R, a.C, r0, R, c0, ncols, 0, 1);
            stage<true>(lq, a.q, R, r0, R, tile.first, tile.n, 0, 1);
        } else {
            stage<false>(lp, a.p + run0 * a.C, a.C, r0, R, c0, ncols, 0, 1);
            stage<false>(lq, a.q + run0 * a.rows, a.rows, r0, R, tile.first, tile.n, 0, 1);
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kStep; s += 16) {
            bf16x8 fp[2], fq[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                fp[b] = *reinterpret_cast<bf16x8 *>(lp + (wc * 64 + b * 32 + lane % 32) * kPitch + s + lane / 32 * 8);
                fq[b] = *reinterpret_cast<bf16x8 *>(lq + (wr * 64 + b * 32 + lane % 32) * kPitch + s + lane / 32 * 8);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    acc[c][r] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fp[c], fq[r], acc[c][r], 0, 0, 0);
        }
        if (OP == kDw && a.db && blockIdx.x == 0 && threadIdx.x < kTile)
            for (int s = 0; s < kStep; ++s)
                colsum += __uint_as_float(static_cast<uint32_t>(lq[threadIdx.x * kPitch + s]) << 16);
    }
    if (OP == kDw && a.db && blockIdx.x == 0 && static_cast<int>(threadIdx.x) < tile.n) {
        float *db = a.db + static_cast<int64_t>(tile.e) * a.rows + tile.first + threadIdx.x;
        *db = (a.flags & MOE_GRAD_ACCUMULATE) ? *db + colsum : colsum;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row_in = wr * 64 + r * 32 + lane % 32;
        if (row_in >= tile.n)
            continue;
        const int64_t row = tile.first + row_in;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int sub = g * 8 + lane / 32 * 4;
            if (OP == kForward && wide == 2) {
                const int c = c0 + wc * 32 + sub;
                if (c >= a.C)
                    continue;
                float zg[4], zu[4], y[4], res[4] = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    zg[i] = acc[0][r][4 * g + i];
                    zu[i] = acc[1][r][4 * g + i];
                    if (a.bias) {
                        zg[i] += a.bias[static_cast<int64_t>(tile.e) * 2 * a.C + c + i];
                        zu[i] += a.bias[static_cast<int64_t>(tile.e) * 2 * a.C + a.C + c + i];
                    }
                }
                if (a.residual)
                    load4(a.residual + row * a.C + c, res);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[i] = zg[i] * sigmoid(zg[i]) * zu[i] + res[i];
                store4(static_cast<uint16_t *>(a.out) + row * a.C + c, y);
                if (a.preact) {
                    store4(a.preact + row * 2 * a.C + c, zg);
                    store4(a.preact + row * 2 * a.C + a.C + c, zu);
                }
                continue;
            }
#pragma unroll
            for (int cb = 0; cb < 2; ++cb) {
                const int c = c0 + wc * 64 + cb * 32 + sub;
                if (c >= a.C)
                    continue;
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[i] = acc[cb][r][4 * g + i];
                if (OP == kForward) {
                    float res[4] = {0, 0, 0, 0};
                    if (a.bias)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[i] += a.bias[static_cast<int64_t>(tile.e) * a.C + c + i];
                    if (a.preact)
                        store4(a.preact + row * a.C + c, v);
                    if (a.residual)
                        load4(a.residual + row * a.C + c, res);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = act_value(v[i], a.act) + res[i];
                    store4(static_cast<uint16_t *>(a.out) + row * a.C + c, v);
                } else if (OP == kDx) {
                    if (wide == 2) {
                        float zg[4], zu[4], dg[4], du[4];
                        load4(a.z + row * 2 * a.C + c, zg);
                        load4(a.z + row * 2 * a.C + a.C + c, zu);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float s = sigmoid(zg[i]);
                            dg[i] = v[i] * zu[i] * s * (1.0f + zg[i] * (1.0f - s));
                            du[i] = v[i] * zg[i] * s;
                        }
                        store4(static_cast<uint16_t *>(a.out) + row * 2 * a.C + c, dg);
                        store4(static_cast<uint16_t *>(a.out) + row * 2 * a.C + a.C + c, du);
                    } else {
                        if (a.act != MOE_ACT_NONE) {
                            float z[4];
                            load4(a.z + row * a.C + c, z);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                v[i] *= act_slope(z[i], a.act);
                        }
                        store4(static_cast<uint16_t *>(a.out) + row * a.C + c, v);
                    }
                } else {
                    const int64_t at = (static_cast<int64_t>(tile.e) * a.rows + row) * a.C + c;
                    if (a.flags & MOE_GRAD_BF16) {
                        store4(static_cast<uint16_t *>(a.out) + at, v);
                    } else {
                        float *o = static_cast<float *>(a.out) + at;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[i] = (a.flags & MOE_GRAD_ACCUMULATE) ? o[i] + v[i] : v[i];
                    }
                }
            }
        }
    }
}

int tiles(int64_t n, int t) { return static_cast<int>((n + t - 1) / t); }

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
    const dim3 grid(static_cast<unsigned>(max_row_tiles(max_rows, E, kTile)),
                    tiles(N, act == MOE_ACT_SWIGLU ? kTile / 2 : kTile));
    expert_kernel<kForward><<<grid, 256, 0, stream>>>(a);
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
    const dim3 grid(static_cast<unsigned>(max_row_tiles(max_rows, E, kTile)), tiles(K, kTile));
    expert_kernel<kDx><<<grid, 256, 0, stream>>>(a);
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
    const dim3 grid(tiles(K, kTile), tiles(N, kTile), E);
    expert_kernel<kDw><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace moe
