// Arguments of the 8-bit products' kernels, and what both of them need for codes.
#pragma once

#include "expert_finish.hpp"
#include "fp8_codes.hpp"

namespace moe {

// Forward, of a gated product, dx, dx through SwiGLU.
enum Kind { kPlain, kGated, kBack, kBackGated };

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
    float *wide_out;        // few rows: results in fp32, of both halves, to be coded
};

// The products for few rows an expert, and whether they pay: `wide` halves of
// weights, C columns, sums over R in all; whole_blocks: codes are wanted, and no
// workspace is for them.  workspace: few_fp8_bytes (of `halves` of results; 0: none is
// worth it), or null.
bool few_fp8_pay(int wide, int E, int64_t max_rows, int R, int C, bool whole_blocks);
int64_t few_fp8_bytes(int wide, int halves, int E, int64_t max_rows, int R, int C);
hipError_t launch_fp8_few(Kind kind, Fp8 &a, int64_t max_rows, void *workspace, hipStream_t stream);

// Largest size of a lane's values of a row and of the three lanes' that hold the
// rest of them.
template <int BLOCKS>
__device__ __forceinline__ uint32_t row_top(const f32x4 (&v)[BLOCKS])
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4 * BLOCKS; ++i)
        top = umax(top, size_bits(v[i / 4][i % 4]));
    // (of a row's four lanes, 16 apart: rows of 16 lanes 1, 3 change places with 0, 2, then halves)
    const auto x = __builtin_amdgcn_permlane16_swap(top, top, false, false);
    top = umax(x[0], x[1]);
    const auto y = __builtin_amdgcn_permlane32_swap(top, top, false, false);
    return umax(y[0], y[1]);
}

// Gradients of silu(gate) * up: of the gate's inputs into d, of the up half's into du.
__device__ __forceinline__ void swiglu_slopes(f32x4 &d, f32x4 &du, const f32x4 &gate, const f32x4 &up)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float g = gate[j], x = d[j], s = sigmoid(g);
        d[j] = x * up[j] * (s * (1.0f + g * (1.0f - s)));
        du[j] = x * (g * s);
    }
}

}  // namespace moe
