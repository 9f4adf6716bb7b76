// Arguments of the 8-bit products' kernels, and what both of them need for codes.
#pragma once

#include "expert_finish.hpp"
#include "fp8_codes.hpp"

namespace moe {

struct Fp8 {
    const uint8_t *w, *q;   // weights and rows, of `segments` times R bytes
    const float *ws, *xs;
    int xs_cols;            // scales of a row: 1, or one a block
    const int32_t *offsets;
    int E, max_rows;
    int R, segments;
    int C, act;             // output columns (of one half)
    const float *bias;
    const uint16_t *residual, *z;
    void *out;
    uint16_t *preact;
    uint8_t *codes;
    float *scales;
    int height;             // rows of a tile
    float *wide_out;        // few rows: results in fp32, to be coded
};

// The products for few rows an expert; workspace: few_fp8_bytes, or null.
hipError_t launch_fp8_few(Fp8 &a, int64_t max_rows, void *workspace, hipStream_t stream);

// Largest size of a lane's values of a row and of the three lanes' that hold the
// rest of them.
template <int BLOCKS>
__device__ __forceinline__ uint32_t row_top(const f32x4 (&v)[BLOCKS])
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4 * BLOCKS; ++i)
        top = umax(top, size_bits(v[i / 4][i % 4]));
    top = umax(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16)));
    return umax(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32)));
}

}  // namespace moe
