// Device helpers of the experts' products: where each expert's run of rows
// lies, and the activations with their derivatives.
#pragma once

#include "../../include/moe_recv.h"
#include "common.hpp"

namespace moe {

// An expert's run: rows [first, first + n) of the buffers.
struct ExpertRun {
    int first, n;
};

// First row of expert e's run (e = E: the end of the last).  Row 0 of the
// buffers is row offsets[0] of the flat numbering; runs are cut at max_rows,
// so no offset reaches past the buffers.
__device__ __forceinline__ int run_start(const int32_t *__restrict__ offsets, int e, int max_rows)
{
    return min(max(offsets[e] - offsets[0], 0), max_rows);
}

// The index-th tile of `height` rows over all runs in expert order (a run's
// last tile is short); n == 0 past the last.
struct RowTile {
    int e, first, n;
};
__device__ __forceinline__ RowTile find_row_tile(const int32_t *__restrict__ offsets, int E, int max_rows,
                                                 int height, int index)
{
    int before = 0;  // tiles of the experts below e0
    for (int e0 = 0; e0 < E; e0 += kWave) {
        const int e = min(e0 + lane_id(), E);
        const int first = run_start(offsets, e, max_rows);
        const int n = max(run_start(offsets, min(e + 1, E), max_rows) - first, 0);
        const int tiles = (n + height - 1) / height;
        const int upto = before + wave_inclusive_scan(tiles);
        const uint64_t hit = __ballot(upto > index);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const int in_run = (index - (lane_value(upto, l) - lane_value(tiles, l))) * height;
            return {e0 + l, lane_value(first, l) + in_run, min(height, lane_value(n, l) - in_run)};
        }
        before = lane_value(upto, kWave - 1);
    }
    return {0, 0, 0};
}

// Workgroup j of a round runs on XCD j % 8, each with an L2 of its own: give
// every XCD a contiguous range of the n entries.  -1 for spare workgroups.
__device__ __forceinline__ int xcd_order(int j, int n)
{
    const int x = j % 8, i = j / 8, each = n / 8, more = n % 8;
    if (i >= each + (x < more))
        return -1;
    return x * each + min(x, more) + i;
}

struct TileAt {
    int row, col;
};

// Groups of eight row tiles, all columns of a group before the next: tiles
// that run side by side share both operands' pieces in L2.
__device__ __forceinline__ TileAt grouped_order(int id, int row_tiles, int col_tiles)
{
    const int group = id / (8 * col_tiles), in = id % (8 * col_tiles);
    const int height = min(8, row_tiles - 8 * group);
    return {8 * group + in % height, in / height};
}

// exp and the reciprocal in single instructions, good to 1 ulp each, behind a
// rounded product: off by at most (1.25 |z| + 5) 2^-24 of the result, against
// the 2^-8 of the bf16 that is stored.  Past +-88 they give 0 and 1.
__device__ __forceinline__ float sigmoid(float z)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}

// The normal distribution function, branchless, from its tail Q(z) = erfc(z /
// sqrt 2) / 2 for z >= 0: with x = z / sqrt 2 and t = 1 / (1 + x/2), erfc(x) = t
// exp(-x^2 + r(t)) (the form of Press et al., Numerical Recipes, 6.2), r a
// polynomial of our own, fitted to log(erfc(x) exp(x^2) / t) on [0, 9.6] (off by
// 5e-8); p has it in base 2, with the half.  In fp32, with instructions off by 1
// ulp, Q is good to 2e-6 of itself for z < 5.6 and the result to 3.5e-7.
__device__ __forceinline__ float normal_below(float z)
{
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.35355339f, 1.0f));
    float p = 0.20405643f;
    p = fmaf(p, t, -0.95468861f);
    p = fmaf(p, t, 1.6036917f);
    p = fmaf(p, t, -0.91733694f);
    p = fmaf(p, t, -0.18831943f);
    p = fmaf(p, t, 0.040594943f);
    p = fmaf(p, t, 0.036643088f);
    p = fmaf(p, t, 0.56060416f);
    p = fmaf(p, t, 1.4403937f);
    p = fmaf(p, t, -2.8256390f);
    const float q = t * __builtin_amdgcn_exp2f(fmaf(z * z, -0.72134752f, p));
    return z < 0.0f ? q : 1.0f - q;
}

// Its density.
__device__ __forceinline__ float normal_density(float z)
{
    return __builtin_amdgcn_exp2f(fmaf(z * z, -0.72134752f, -1.3257480f));
}

// v[i][j] = act(v[i][j]) for the activations of one value.  A NaN stays one
// (a maximum with 0 would make it 0).
template <int N, typename V>
__device__ __forceinline__ void apply_act(V (&v)[N], int act)
{
    if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 4 * N; ++i)
            v[i / 4][i % 4] = v[i / 4][i % 4] <= 0.0f ? 0.0f : v[i / 4][i % 4];
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 4 * N; ++i)
            v[i / 4][i % 4] *= sigmoid(v[i / 4][i % 4]);
    } else if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 4 * N; ++i)
            v[i / 4][i % 4] *= normal_below(v[i / 4][i % 4]);
    }
}

// v[i][j] *= act'(z[i][j]).  ReLU stops a gradient where z <= 0, so not at a
// NaN.
template <int N, typename V>
__device__ __forceinline__ void apply_slope(V (&v)[N], const V (&z)[N], int act)
{
    if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 4 * N; ++i)
            v[i / 4][i % 4] = z[i / 4][i % 4] <= 0.0f ? 0.0f : v[i / 4][i % 4];
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 4 * N; ++i) {
            const float x = z[i / 4][i % 4], s = sigmoid(x);
            v[i / 4][i % 4] *= s * (1.0f + x * (1.0f - s));
        }
    } else if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 4 * N; ++i) {
            const float x = z[i / 4][i % 4];
            v[i / 4][i % 4] *= fmaf(x, normal_density(x), normal_below(x));
        }
    }
}

}  // namespace moe
