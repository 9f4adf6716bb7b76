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

// A tile of rows of one expert: rows [first, first + n), n <= the tile's
// height; n == 0 past the last tile.
struct RowTile {
    int e, first, n;
};

// The index-th tile of `height` rows over all experts' runs in expert order
// (a run's last tile is short).  Every lane of the wave calls it; index is
// uniform.  64 experts' tile counts are scanned at a time.
__device__ __forceinline__ RowTile find_row_tile(const int32_t *__restrict__ offsets, int E,
                                                 int max_rows, int height, int index)
{
    int before = 0;  // tiles of the experts below `e0`
    for (int e0 = 0; e0 < E; e0 += kWave) {
        const int e = e0 + lane_id();
        const ExpertRun run = e < E ? expert_run(offsets, e, max_rows) : ExpertRun{0, 0};
        const int tiles = (run.n + height - 1) / height;
        const int upto = before + wave_inclusive_scan(tiles);
        const uint64_t hit = __ballot(upto > index);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            const int in_run = (index - (lane_value(upto, l) - lane_value(tiles, l))) * height;
            return {e0 + l, lane_value(run.first, l) + in_run,
                    min(height, lane_value(run.n, l) - in_run)};
        }
        before = lane_value(upto, kWave - 1);
    }
    return {0, 0, 0};
}

// Most tiles that E runs of together max_rows rows can have.
inline int64_t max_row_tiles(int64_t max_rows, int E, int height)
{
    const int64_t live = max_rows < E ? max_rows : E;
    return (max_rows - live) / height + live;
}

__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

// act(z) for the activations of one value (SwiGLU: act_pair).
__device__ __forceinline__ float act_value(float z, int act)
{
    if (act == MOE_ACT_RELU)
        return fmaxf(z, 0.0f);
    if (act == MOE_ACT_SILU)
        return z * sigmoid(z);
    if (act == MOE_ACT_GELU)
        return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    return z;
}

// d act / d z.
__device__ __forceinline__ float act_slope(float z, int act)
{
    if (act == MOE_ACT_RELU)
        return z > 0.0f ? 1.0f : 0.0f;
    if (act == MOE_ACT_SILU) {
        const float s = sigmoid(z);
        return s * (1.0f + z * (1.0f - s));
    }
    if (act == MOE_ACT_GELU)
        return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) +
               z * expf(-0.5f * z * z) * 0.39894228040143268f;
    return 1.0f;
}

}  // namespace moe
