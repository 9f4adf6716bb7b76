// The 8-bit products for few rows an expert, as serving single tokens has them.
//
// Every live expert's weights are read once and multiplied with up to 16 rows, so the
// reading bounds it.  A wave has 16 output columns (GATED: 16 of both halves): two
// loads of 16 bytes a lane are a matrix instruction's operand, 16 rows of one whole
// line each, so they go straight to registers, four blocks of 128 ahead, or eight where
// one to four waves a CU are all there is: 1 row, 4096 -> 4096 (one a CU), 9.3 us against
// 12.5; -> 8192 (two) 13.7 against 17.3; -> 16320 (four) 21.9 against 24.4.  Of a short sum
// half of them would be loads of nothing: 515 rows, 272 <- 512, 5.9 against 5.4, so sums up to
// 1024 take four.  (With four waves a CU the two meet at 2048; 1040 -> 16320 is 7.4 against 6.7.)
//
// A CU takes some 30 GB/s, so all of them have to read: 32 columns a workgroup
// where 64 would make one for every CU, else 16.  (One token at 8 of 32 experts, 7168 ->
// 2048 gated, 235 MB of weights: 44 us, 5.3 TB/s, in 512 workgroups or 256, 66 in 128;
// 2048 -> 7168, 117 MB: 26 us in 1792 workgroups, 28 in 896 of twice the columns.)  But
// the scale of a coded block goes by 128 columns: their workgroups have all of them, or,
// with a workspace, leave the results there in fp32 for a second kernel to code.
#include "fp8_args.hpp"
#include "launch.hpp"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

template <Kind KIND, int CW, int kDepth>
__global__ __launch_bounds__(64 * CW) void fp8_few_kernel(Fp8 a)
{
    constexpr bool GATED = KIND == kGated, BOTH = KIND == kBackGated;
    constexpr int wide = GATED ? 2 : 1, out = BOTH ? 2 : 1;  // halves of the weights, of the results
    __shared__ uint32_t tops[out][CW][16];
    const int lane = lane_id(), w = static_cast<int>(uniform(threadIdx.x / kWave));
    const int groups = (a.C + 16 * CW - 1) / (16 * CW), nbc = code_blocks(a.C);
    const RowTile t = find_row_tile(a.offsets, a.E, a.max_rows, 16, blockIdx.x / groups);
    if (t.n <= 0)
        return;
    const int c0 = blockIdx.x % groups * (16 * CW) + w * 16;
    const int pitch = a.R * a.segments, blocks = code_blocks(a.R), steps = blocks * a.segments;
    const bool inside = c0 < a.C;  // of the array; a.C is a multiple of 16
    __amdgpu_buffer_rsrc_t wr[wide], wsr[wide];
#pragma unroll
    for (int g = 0; g < wide; ++g) {
        const int64_t half = static_cast<int64_t>(t.e) * wide + g;
        wr[g] = row_rsrc(const_cast<uint8_t *>(a.w) + (half * a.C + c0) * pitch, inside ? 16 * pitch : 0);
        wsr[g] = row_rsrc(const_cast<float *>(a.ws) + (half * nbc + c0 / kCodeBlock) * steps, inside ? steps * 4 : 0);
    }
    const __amdgpu_buffer_rsrc_t xr = row_rsrc(const_cast<uint8_t *>(a.q) + static_cast<int64_t>(t.first) * pitch, t.n * pitch);
    const __amdgpu_buffer_rsrc_t xsr =
        row_rsrc(const_cast<float *>(a.xs) + static_cast<int64_t>(t.first) * a.xs_cols, t.n * a.xs_cols * 4);
    const int row = lane % 16, at = lane / 16 * 16, xs_step = a.xs_cols == 1 ? 0 : 4;

    struct Block {
        u32x4 w[wide][2], x[2];
        float ws[wide], xs;
    };
    Block ring[kDepth];
    auto load = [&](Block &b, int k) {
        const int segment = k < blocks ? 0 : a.R;  // of at most two
        const int r = (k < blocks ? k : k - blocks) * kCodeBlock + at;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int o = k < steps && r + 64 * h < a.R ? row * pitch + segment + r + 64 * h : kOutside;
#pragma unroll
            for (int g = 0; g < wide; ++g)
                b.w[g][h] = load_cached(wr[g], o);  // (past the caches, the line's second half comes from memory again: 85 us)
            b.x[h] = load_cached(xr, o);
        }
#pragma unroll
        for (int g = 0; g < wide; ++g)
            b.ws[g] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(wsr[g], k * 4, 0, 0));
        b.xs = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
            xsr, k < steps ? row * a.xs_cols * 4 + k * xs_step : kOutside, 0, 0));
    };
    auto operand = [](const u32x4 (&v)[2]) {
        return i32x8{(int)v[0].x, (int)v[0].y, (int)v[0].z, (int)v[0].w, (int)v[1].x, (int)v[1].y, (int)v[1].z, (int)v[1].w};
    };
    f32x4 acc[wide] = {};
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
        load(ring[d], d);
    for (int k = 0; k < steps; k += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
#pragma unroll
            for (int g = 0; g < wide; ++g) {
                const f32x4 v = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(ring[d].w[g]), operand(ring[d].x),
                                                                                 f32x4{}, 0, 0, 0, 0, 0, 0);
                const float s = ring[d].ws[g] * ring[d].xs;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[g][j] = fmaf(v[j], s, acc[g][j]);
            }
            load(ring[d], k + d + kDepth);
        }
    }
    // four columns of one row a lane
    const int c = c0 + lane / 16 * 4;
    const bool live = inside && row < t.n;
    const int64_t r = t.first + row;
    auto load4 = [](const uint16_t *p) { return widen4(*reinterpret_cast<const u32x2 *>(p)); };
    auto store4 = [](uint16_t *p, f32x4 f) { *reinterpret_cast<u32x2 *>(p) = round4(f); };
    f32x4 y[out][1] = {};
    y[0][0] = acc[0];
    if constexpr (KIND == kBack) {
        if (a.act != MOE_ACT_NONE && live) {
            const f32x4 z[1] = {load4(a.z + r * a.C + c)};
            apply_slope(y[0], z, a.act);
        }
    } else if constexpr (BOTH) {
        if (live) {
            const f32x4 g = load4(a.z + r * 2 * a.C + c), u = load4(a.z + (r * 2 + 1) * a.C + c);
            swiglu_slopes(y[0][0], y[1][0], g, u);
        }
    } else {
#pragma unroll
        for (int g = 0; g < wide; ++g) {
            if (a.bias && live)
                acc[g] += *reinterpret_cast<const f32x4 *>(a.bias + (static_cast<int64_t>(t.e) * wide + g) * a.C + c);
            if (a.preact && live)
                store4(a.preact + (r * wide + g) * a.C + c, acc[g]);
        }
        y[0][0] = acc[0];
        if (GATED) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[0][0][j] *= sigmoid(y[0][0][j]) * acc[wide - 1][j];
        } else {
            apply_act(y[0], a.act);
        }
        if (a.residual && live)
            y[0][0] += load4(a.residual + r * a.C + c);
    }
#pragma unroll
    for (int o = 0; o < out; ++o) {
        if (a.wide_out && live)
            *reinterpret_cast<f32x4 *>(a.wide_out + (r * out + o) * a.C + c) = y[o][0];
        if (a.out && live)
            store4(static_cast<uint16_t *>(a.out) + (r * out + o) * a.C + c, y[o][0]);
    }
    if constexpr (CW == 8) {
#pragma unroll
        for (int o = 0; o < out; ++o) {
            const uint32_t mine = row_top(y[o]);
            tops[o][w][row] = live ? mine : 0u;  // (four lanes of a row, the same value)
        }
        __syncthreads();
#pragma unroll
        for (int o = 0; o < out; ++o) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < CW; ++i)
                top = umax(top, tops[o][i][row]);
            const float scale = scale_of(top);
            const uint32_t q = Coder(scale).codes4(y[o][0][0], y[o][0][1], y[o][0][2], y[o][0][3]);
            if (!live)
                continue;
            *reinterpret_cast<uint32_t *>(a.codes + (r * out + o) * a.C + c) = q;
            if (w == 0 && lane < 16)
                a.scales[(r * out + o) * nbc + c0 / kCodeBlock] = scale;
        }
    }
}

template <Kind KIND, int CW, int DEPTH = 4>
void launch(const Fp8 &a, int64_t tiles, hipStream_t stream)
{
    fp8_few_kernel<KIND, CW, DEPTH>
        <<<dim3(static_cast<unsigned>(tiles * ((a.C + 16 * CW - 1) / (16 * CW)))), 64 * CW, 0, stream>>>(a);
}
template <Kind KIND>
hipError_t launch(Fp8 &a, int64_t max_rows, void *workspace, hipStream_t stream)
{
    constexpr int halves_in = KIND == kGated ? 2 : 1, out = KIND == kBackGated ? 2 : 1;
    const int64_t tiles = max_row_tiles(max_rows, a.E, 16);
    uint8_t *codes = a.codes;
    a.max_rows = static_cast<int>(max_rows);
    if (codes && !(workspace && few_fp8_bytes(halves_in, out, a.E, max_rows, a.R * a.segments, a.C))) {
        launch<KIND, 8>(a, tiles, stream);
        return hipGetLastError();
    }
    a.codes = nullptr;
    a.wide_out = codes ? static_cast<float *>(workspace) : nullptr;
    if (tiles * ((a.C + 63) / 64) >= kCus)
        launch<KIND, 2>(a, tiles, stream);
    else if (KIND != kGated && a.R * a.segments > 8 * kCodeBlock)
        launch<KIND, 1, KIND == kGated ? 4 : 8>(a, tiles, stream);
    else
        launch<KIND, 1>(a, tiles, stream);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess || !codes)
        return err;
    return launch_quant_wide_rows(a.wide_out, a.offsets, a.E, max_rows, a.C, out, codes, a.scales, stream);
}

}  // namespace

// Estimates in us.  Here: the weights once from memory at 6 TB/s, again for every
// further 16 rows and the rows for every 16 columns from the caches at 11, and 3.  The
// tiles: 6, and 1 and 0.8 a block of 128 for each round of them, or the weights at 5.6
// TB/s and 3 if that is longer.  Measured (here / tiles): one token of 8 experts above 44 /
// 63; 4 rows of each of 32, 7168 -> 2048 gated 158 / 166, 2048 -> 7168 90 / 98; 16 rows
// of each 119 / 99; 2 of each of 64, 1024 -> 4096 57 / 64; 1 or 16 rows of one, 4096 ->
// 4096 9.5 / 28.  Coded by the workgroup itself (whole_blocks), a call also
// takes what 128 columns do at 30 GB/s, so 16 rows of one, 4096 <- 4096, take 38 (30 in
// tiles); over the workspace they take 15, but another kernel and 4 us more of any
// call (8 of 65 rows, 272 <- 512 through SwiGLU: 15 against 11).  dx else:
// 515 rows of 8, 272 <- 512, 10 / 14; one token of 8, 7168 <- 2 x 2048, 58 / 61; 2 of
// each of 64, 4096 <- 1024, 66 / 88; 16 of each of 32, 7168 <- 2 x 2048, 274 / 181.
static double few_us(int wide, int E, int64_t max_rows, int R, int C, bool whole_blocks)
{
    const int64_t live = max_rows < E ? max_rows : E, tiles = max_row_tiles(max_rows, E, 16);
    const double each = 1.0 * wide * C * R;
    const double us = live * each / 6e6 + ((tiles - live) * each + (C / 16.0) * max_rows * R) / 11e6 + 3;
    const double group = R * 128.0 * (wide + (max_rows < 16 ? max_rows / 16.0 : 1)) / 3e4 + 3;  // of a workgroup
    return whole_blocks && us < group ? group : us;
}

bool few_fp8_pay(int wide, int E, int64_t max_rows, int R, int C, bool whole_blocks)
{
    if (!grid_fits(max_row_tiles(max_rows, E, 16) * code_blocks(C), 512))  // (the largest of its three)
        return false;
    const double weights = 1.0 * (max_rows < E ? max_rows : E) * wide * C * R;
    const int cols = 256 / wide;
    const int64_t coarse = max_row_tiles(max_rows, E, 64) * ((C + cols - 1) / cols);
    const double there = ((coarse + kCus - 1) / kCus) * (1 + code_blocks(R) * 0.8) + 6;
    const double here = few_us(wide, E, max_rows, R, C, whole_blocks);
    return here < (there > weights / 5.6e6 + 3 ? there : weights / 5.6e6 + 3);
}

int64_t few_fp8_bytes(int wide, int halves, int E, int64_t max_rows, int R, int C)
{
    const bool pays = max_row_tiles(max_rows, E, 16) * code_blocks(C) < kCus &&
                      few_us(wide, E, max_rows, R, C, true) > few_us(wide, E, max_rows, R, C, false) + 4;
    return pays ? max_rows * halves * C * 4 : 0;
}

hipError_t launch_fp8_few(Kind kind, Fp8 &a, int64_t max_rows, void *workspace, hipStream_t stream)
{
    switch (kind) {
    case kPlain: return launch<kPlain>(a, max_rows, workspace, stream);
    case kGated: return launch<kGated>(a, max_rows, workspace, stream);
    case kBack: return launch<kBack>(a, max_rows, workspace, stream);
    default: return launch<kBackGated>(a, max_rows, workspace, stream);
    }
}

}  // namespace moe
