// The experts' products of E4M3 rows and weights, and the gradient of their rows:
//
//   forward   z = sum over blocks b of 128 of  xs[p, b] ws[n / 128, b] (xc wc)_b + bias,  y = act(z) + residual
//   dx        g = the same of dy's codes and the transposed weights',  dx = act'(z_prev) g
//
// A block's codes are multiplied in one matrix instruction (16 x 16 x 128) and
// its sums scaled into fp32 accumulators.  The results leave in bf16, in codes, or
// both.
#include "expert_rows.hpp"
#include "fp8_codes.hpp"
#include "launch.hpp"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kOutside = static_cast<int>(0x80000000u);

struct Fp8 {
    const uint8_t *w, *x;   // [E][wide][C][steps' length], [max_rows][...]
    const float *ws, *xs;
    int xs_cols;            // scales of a row: 1, or one a step
    const int32_t *offsets;
    int E, max_rows;
    int R, segments;        // reduced length: `segments` of R
    int C, act;             // output columns (of one half)
    const float *bias;
    const uint16_t *residual, *z;
    uint16_t *out, *preact;
    uint8_t *codes;
    float *scales;
};

// Largest size of this lane's values of a row's block and of the three lanes' that
// hold the rest of it.
__device__ __forceinline__ uint32_t block_top(const f32x4 (&v)[8], int inside)
{
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (c * 16 < inside)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                top = umax(top, size_bits(v[c][j]));
    top = umax(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));
    return umax(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
}

__device__ __forceinline__ void store4(uint16_t *p, f32x4 f)
{
    *reinterpret_cast<u32x2 *>(p) = u32x2{pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w)};
}
__device__ __forceinline__ f32x4 load4(const uint16_t *p)
{
    const u32x2 s = *reinterpret_cast<const u32x2 *>(p);
    return f32x4{bf16_lo(s.x), bf16_hi(s.x), bf16_lo(s.y), bf16_hi(s.y)};
}

// Stores 128 columns of one row a lane (block `half` of `halves`): v[c] has columns
// c0 + 16 c + 4 (lane / 16) .. + 3.
__device__ __forceinline__ void store_block(const Fp8 &a, const f32x4 (&v)[8], int64_t row, bool live, int c0,
                                            int halves, int half)
{
    const int inside = a.C - c0, at = lane_id() / 16 * 4;
    const int64_t line = (row * halves + half) * a.C + c0 + at;
    const uint32_t top = block_top(v, inside);
    if (!live)
        return;
    const float scale = scale_of(top);
#pragma unroll
    for (int c = 0; c < 8; ++c)
        if (c * 16 < inside) {
            if (a.out)
                store4(a.out + line + c * 16, v[c]);
            if (a.codes)
                *reinterpret_cast<uint32_t *>(a.codes + line + c * 16) = codes4(v[c][0], v[c][1], v[c][2], v[c][3], scale);
        }
    if (a.codes && at == 0)
        a.scales[(row * halves + half) * code_blocks(a.C) + c0 / kCodeBlock] = scale;
}

// One wave for 16 rows of a tile by 128 columns; GATED: of both halves.
template <bool DX, bool GATED>
__global__ __launch_bounds__(256) void expert_fp8_kernel(Fp8 a)
{
    constexpr int wide = GATED ? 2 : 1;
    const int lane = lane_id(), w = static_cast<int>(uniform(threadIdx.x / kWave));
    const int col_tiles = code_blocks(a.C);
    const RowTile t = find_row_tile(a.offsets, a.E, a.max_rows, 64, blockIdx.x / col_tiles);
    const int n = t.n - 16 * w;
    if (n <= 0)
        return;
    const int cb = blockIdx.x % col_tiles, c0 = cb * kCodeBlock, inside = a.C - c0;
    const int nb = code_blocks(a.R), steps = nb * a.segments, pitch = a.R * a.segments;
    const int64_t first = t.first + 16 * w;
    const __amdgpu_buffer_rsrc_t xr = row_rsrc(const_cast<uint8_t *>(a.x) + first * pitch, min(n, 16) * pitch);
    const float *xs = a.xs + (first + min(lane % 16, n - 1)) * a.xs_cols;
    f32x4 acc[wide][8] = {};
    for (int k = 0; k < steps; ++k) {
        const int r0 = k / nb * a.R + k % nb * kCodeBlock, end = (k / nb + 1) * a.R, r = r0 + lane / 16 * 32;
        auto fragment = [&](const __amdgpu_buffer_rsrc_t &rsrc, int row) {
            const u32x4 lo = load_cached(rsrc, r < end ? row * pitch + r : kOutside);
            const u32x4 hi = load_cached(rsrc, r + 16 < end ? row * pitch + r + 16 : kOutside);
            return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
        };
        const i32x8 q = fragment(xr, lane % 16);
        const float s = xs[a.xs_cols == 1 ? 0 : k];
#pragma unroll
        for (int g = 0; g < wide; ++g) {
            const int64_t block = (static_cast<int64_t>(t.e) * wide + g) * col_tiles + cb;
            const __amdgpu_buffer_rsrc_t wr = row_rsrc(
                const_cast<uint8_t *>(a.w) + ((static_cast<int64_t>(t.e) * wide + g) * a.C + c0) * pitch, min(inside, 128) * pitch);
            const float scale = s * a.ws[block * steps + k];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const i32x8 p = fragment(wr, c * 16 + lane % 16);
                const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q, f32x4{}, 0, 0, 0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[g][c][j] = fmaf(d[j], scale, acc[g][c][j]);
            }
        }
    }
    const int64_t row = first + lane % 16;
    const bool live = lane % 16 < n;
    const int at = lane / 16 * 4;
    if constexpr (DX) {
        const bool gated = a.act == MOE_ACT_SWIGLU;
        f32x4 up[8] = {};
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            if (!live || c * 16 >= inside)
                continue;
            const int col = c0 + c * 16 + at;
            if (gated) {
                const f32x4 g = load4(a.z + row * 2 * a.C + col), u = load4(a.z + (row * 2 + 1) * a.C + col);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x = acc[0][c][j], s = sigmoid(g[j]);
                    acc[0][c][j] = x * u[j] * (s * (1.0f + g[j] * (1.0f - s)));
                    up[c][j] = x * (g[j] * s);
                }
            } else if (a.act != MOE_ACT_NONE) {
                const f32x4 z[1] = {load4(a.z + row * a.C + col)};
                f32x4 v[1] = {acc[0][c]};
                apply_slope(v, z, a.act);
                acc[0][c] = v[0];
            }
        }
        store_block(a, acc[0], row, live, c0, gated ? 2 : 1, 0);
        if (gated)
            store_block(a, up, row, live, c0, 2, 1);
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            if (!live || c * 16 >= inside)
                continue;
            const int col = c0 + c * 16 + at;
#pragma unroll
            for (int g = 0; g < wide; ++g) {
                if (a.bias)
                    acc[g][c] += *reinterpret_cast<const f32x4 *>(a.bias + (static_cast<int64_t>(t.e) * wide + g) * a.C + col);
                if (a.preact)
                    store4(a.preact + (row * wide + g) * a.C + col, acc[g][c]);
            }
            f32x4 y[1] = {acc[0][c]};
            if (GATED) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    y[0][j] = y[0][j] * sigmoid(y[0][j]) * acc[wide - 1][c][j];
            } else {
                apply_act(y, a.act);
            }
            if (a.residual)
                y[0] += load4(a.residual + row * a.C + col);
            acc[0][c] = y[0];
        }
        store_block(a, acc[0], row, live, c0, 1, 0);
    }
}

}  // namespace

hipError_t launch_expert_fp8(const void *x, const float *xs, int xs_cols, const int32_t *offsets, const void *w,
                             const float *ws, const float *bias, int act, const void *residual, int E, int64_t max_rows,
                             int K, int N, void *out, void *codes, float *scales, void *preact, hipStream_t stream)
{
    Fp8 a{};
    a.x = static_cast<const uint8_t *>(x), a.xs = xs, a.xs_cols = xs_cols, a.offsets = offsets;
    a.w = static_cast<const uint8_t *>(w), a.ws = ws, a.bias = bias, a.act = act;
    a.residual = static_cast<const uint16_t *>(residual), a.E = E, a.max_rows = static_cast<int>(max_rows);
    a.R = K, a.segments = 1, a.C = N, a.out = static_cast<uint16_t *>(out), a.codes = static_cast<uint8_t *>(codes);
    a.scales = scales, a.preact = static_cast<uint16_t *>(preact);
    const dim3 grid(static_cast<unsigned>(max_row_tiles(max_rows, E, 64) * code_blocks(N)));
    if (act == MOE_ACT_SWIGLU)
        expert_fp8_kernel<false, true><<<grid, 256, 0, stream>>>(a);
    else
        expert_fp8_kernel<false, false><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_expert_fp8_dx(const void *dy, const float *dys, const int32_t *offsets, const void *wt,
                                const float *wts, int halves, int act, const void *z, int E, int64_t max_rows, int K,
                                int N, void *dx, void *codes, float *scales, hipStream_t stream)
{
    Fp8 a{};
    a.x = static_cast<const uint8_t *>(dy), a.xs = dys, a.xs_cols = halves * code_blocks(N), a.offsets = offsets;
    a.w = static_cast<const uint8_t *>(wt), a.ws = wts, a.act = act, a.z = static_cast<const uint16_t *>(z);
    a.E = E, a.max_rows = static_cast<int>(max_rows), a.R = N, a.segments = halves, a.C = K;
    a.out = static_cast<uint16_t *>(dx), a.codes = static_cast<uint8_t *>(codes), a.scales = scales;
    const dim3 grid(static_cast<unsigned>(max_row_tiles(max_rows, E, 64) * code_blocks(K)));
    expert_fp8_kernel<true, false><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace moe
