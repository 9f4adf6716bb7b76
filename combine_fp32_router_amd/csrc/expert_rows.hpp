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

// Row 0 of the buffers is row offsets[0] of the flat numbering; runs are cut
// at max_rows, so no offset reaches past the buffers.
__device__ __forceinline__ ExpertRun expert_run(const int32_t *__restrict__ offsets, int e,
                                                int max_rows)
{
    const int base = offsets[0];
    const int a = min(max(offsets[e] - base, 0), max_rows);
    const int b = min(max(offsets[e + 1] - base, a), max_rows);
    return {a, b - a};
}

// Workgroup j of a round runs on XCD j % 8, each with an L2 of its own: give
// every XCD a contiguous range of the n entries.  -1 for spare workgroups.
__device__ __forceinline__ int64_t xcd_order(int64_t j, int64_t n)
{
    const int64_t x = j % 8, i = j / 8, each = n / 8, more = n % 8;
    if (i >= each + (x < more))
        return -1;
    return x * each + min(x, more) + i;
}

struct TileAt {
    int row, col;
};

// Groups of eight row tiles, all columns of a group before the next: tiles
// that run side by side share both operands' pieces in L2.
__device__ __forceinline__ TileAt grouped_order(int64_t id, int row_tiles, int col_tiles)
{
    const int group = static_cast<int>(id / (8 * col_tiles)), in = static_cast<int>(id % (8 * col_tiles));
    const int height = min(8, row_tiles - 8 * group);
    return {8 * group + in % height, in / height};
}

// Most tiles that E runs of together max_rows rows can have.
inline int64_t max_row_tiles(int64_t max_rows, int E, int height)
{
    const int64_t live = max_rows < E ? max_rows : E;
    return (max_rows - live) / height + live;
}

// exp and the reciprocal in single instructions, good to 1 ulp each, behind a
// rounded product: off by about (|z| + 2) 2^-24 of the result, against the
// 2^-9 of the bf16 that is stored.  Past +-88 they give 0 and 1.
__device__ __forceinline__ float sigmoid(float z)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}

// v[i][j] = act(v[i][j]) for the activations of one value.
template <int N, typename V>
__device__ __forceinline__ void apply_act(V (&v)[N], int act)
{
    if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 4 * N; ++i)
            v[i / 4][i % 4] = fmaxf(v[i / 4][i % 4], 0.0f);
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 4 * N; ++i)
            v[i / 4][i % 4] *= sigmoid(v[i / 4][i % 4]);
    } else if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 4 * N; ++i) {
            const float z = v[i / 4][i % 4];
            v[i / 4][i % 4] = 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
        }
    }
}

// v[i][j] *= act'(z[i][j]).
template <int N, typename V>
__device__ __forceinline__ void apply_slope(V (&v)[N], const V (&z)[N], int act)
{
    if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 4 * N; ++i)
            v[i / 4][i % 4] = z[i / 4][i % 4] > 0.0f ? v[i / 4][i % 4] : 0.0f;
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
            v[i / 4][i % 4] *= 0.5f * (1.0f + erff(x * 0.70710678118654752f)) +
                               x * __expf(-0.5f * x * x) * 0.39894228040143268f;
        }
    }
}

}  // namespace moe
