// The experts' products of E4M3 rows and weights, and the gradient of their rows:
//
//   forward   z = sum over blocks b of 128 of  xs[p, b] ws[n / 128, b] (xc wc)_b + bias,  y = act(z) + residual
//   dx        g = the same of dy's codes and the transposed weights',  dx = act'(z_prev) g
//
// The results leave in bf16, in codes with a scale for each 128, or both.
#include "fp8_tile.hpp"
#include "launch.hpp"

namespace moe {
namespace {

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
};

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

// Codes of 16 rows of a wave's columns, through LDS into whole pieces.
template <int BLOCKS>
__device__ __forceinline__ void store_codes(MOE_LDS char *__restrict__ lds, const f32x4 (&v)[BLOCKS], float scale,
                                            const Pieces<BLOCKS> &to, int row)
{
    const int lane = to.lane, r = lane % 16;
#pragma unroll
    for (int c = 0; c < BLOCKS; ++c)
        *reinterpret_cast<MOE_LDS uint32_t *>(lds + r * 256 + (c ^ r) * 16 + lane / 16 * 4) =
            codes4(v[c][0], v[c][1], v[c][2], v[c][3], scale);
#pragma unroll
    for (int j = 0; j < BLOCKS / 4; ++j)
        to.store(row, j, *reinterpret_cast<const MOE_LDS u32x4 *>(lds + Place::piece<BLOCKS>(j, lane)));
}

// Where a tile's results go: its rows first .. first + n - 1, this wave's columns
// from c on, `inside` of them (or more) the array's.
struct Where {
    int e, first, n, c, inside, lane;
};

// The scale of the block that this wave's columns begin, of the 16 rows from `row`.
__device__ __forceinline__ void store_scale(const Fp8 &a, const Where &at, int row, int halves, int half, float scale)
{
    const int r = row + at.lane % 16;
    if (at.lane < 16 && r < at.n && at.inside > 0)
        a.scales[((static_cast<int64_t>(at.first) + r) * halves + half) * code_blocks(a.C) + at.c / kCodeBlock] = scale;
}

// Loaded pieces of 16 rows, eight a row, into LDS: as the first or the second eight.
__device__ __forceinline__ void put_pieces(MOE_LDS char *__restrict__ lds, const u32x4 (&in)[2], int second, int lane)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int row = 8 * j + lane / 8;
        *reinterpret_cast<MOE_LDS u32x4 *>(lds + row * 256 + ((lane % 8 + 8 * second) ^ row) * 16) = in[j];
    }
}
__device__ __forceinline__ f32x4 get_block(const MOE_LDS char *__restrict__ lds, int c, int lane)
{
    return widen4(*reinterpret_cast<const MOE_LDS u32x2 *>(lds + Place::half(c, lane)));
}

// Forward: bias, pre-activations, activation, residual.  The accumulators are
// changed in place, a block of 64 rows after the other: beside 128 of them there is
// no room for copies.  GATED: blocks 0, 1, 4, 5 are the gate's, 2, 3, 6, 7 the up
// half's.
template <bool GATED, int NB>
__device__ __forceinline__ void finish_forward(const Fp8 &a, const CodeTile<GATED> &t,
                                               const typename CodeTile<GATED>::template Regs<NB> &f, const Where &at,
                                               MOE_LDS char *lds)
{
    constexpr int kBlocks = GATED ? 4 : 8, P = 2 * kBlocks, wide = GATED ? 2 : 1;
    MOE_LDS char *place = t.out_place(lds);
    const Pieces<P> out(a.out, at.first, at.n, a.C, 2, at.c, at.inside, at.lane), res(a.residual, at.first, at.n, a.C, 2, at.c, at.inside, at.lane);
    const Pieces<P> pre(a.preact, at.first, at.n, wide * a.C, 2, at.c, at.inside, at.lane);
    const Pieces<P> pre_up(a.preact, at.first, at.n, wide * a.C, 2, GATED ? at.c + a.C : at.c, at.inside, at.lane);
    const Pieces<kBlocks> codes(a.codes, at.first, at.n, a.C, 1, at.c, at.inside, at.lane);
    const float *bias = a.bias + static_cast<int64_t>(at.e) * wide * a.C + at.c + at.lane / 16 * 4;
    u32x4 ahead[P / 4];  // the residual's next 16 rows
    auto load = [&](int row) {
        if (a.residual)
#pragma unroll
            for (int j = 0; j < P / 4; ++j)
                ahead[j] = res.load(row, j);
    };
    load(t.row0(0));
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        if (b * 64 >= at.n)
            break;
        const int row = t.row0(b);
        f32x4 g[kBlocks], u[GATED ? kBlocks : 1];
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            g[i] = f.acc[GATED ? i / 2 * 4 + i % 2 : i][b];
            if (GATED)
                u[i] = f.acc[(i / 2 * 4 + i % 2 + 2) % 8][b];
            if (a.bias && i * 16 < at.inside) {
                g[i] += *reinterpret_cast<const f32x4 *>(bias + i * 16);
                if (GATED)
                    u[i] += *reinterpret_cast<const f32x4 *>(bias + a.C + i * 16);
            }
        }
        if (a.preact) {
            store_blocks<P>(place, g, pre, row);
            if constexpr (GATED)
                store_blocks<P>(place, u, pre_up, row);
        }
        if (GATED) {
#pragma unroll
            for (int i = 0; i < 4 * kBlocks; ++i)
                g[i / 4][i % 4] *= sigmoid(g[i / 4][i % 4]) * u[GATED ? i / 4 : 0][i % 4];
        } else {
            apply_act(g, a.act);
        }
        if (a.residual) {
#pragma unroll
            for (int j = 0; j < P / 4; ++j)
                *reinterpret_cast<MOE_LDS u32x4 *>(place + Place::piece<P>(j, at.lane)) = ahead[j];
            load(t.row0(min(b + 1, NB - 1)));  // in front of this block's stores: waiting for it is then not waiting for them
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
                g[i] += get_block(place, i, at.lane);
        }
        if (a.out)
            store_blocks<P>(place, g, out, row);
        if (a.codes) {
            uint32_t top = row_top(g);
            if (GATED)
                top = t.both_halves(lds, b, top, at.lane);
            const float scale = scale_of(top);
            store_codes(place, g, scale, codes, row);
            if (!GATED || t.col0() == 0)
                store_scale(a, at, row, 1, 0, scale);
        }
    }
}

// dx: through the activation that made the product's input, 64 columns at a time.
template <int NB>
__device__ __forceinline__ void finish_dx(const Fp8 &a, const CodeTile<false> &t, const CodeTile<false>::Regs<NB> &f,
                                          const Where &at, MOE_LDS char *lds)
{
    MOE_LDS char *place = t.out_place(lds);
    const bool gated = a.act == MOE_ACT_SWIGLU;
    const int cols = gated ? 2 * a.C : a.C, up = gated ? at.c + a.C : at.c;
    const Pieces<16> out(a.out, at.first, at.n, cols, 2, at.c, at.inside, at.lane), out_up(a.out, at.first, at.n, cols, 2, up, at.inside, at.lane);
    const Pieces<8> codes(a.codes, at.first, at.n, cols, 1, at.c, at.inside, at.lane), codes_up(a.codes, at.first, at.n, cols, 1, up, at.inside, at.lane);
    const Pieces<8> pre(a.z, at.first, at.n, cols, 2, at.c, at.inside, at.lane), pre_r(a.z, at.first, at.n, cols, 2, at.c + 64, at.inside - 64, at.lane);
    const Pieces<8> pre_up(a.z, at.first, at.n, cols, 2, up, at.inside, at.lane), pre_up_r(a.z, at.first, at.n, cols, 2, up + 64, at.inside - 64, at.lane);
    u32x4 ahead[2], ahead_up[2];
    auto load = [&](int row, bool right) {
        if (a.act != MOE_ACT_NONE)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                ahead[j] = right ? pre_r.load(row, j) : pre.load(row, j);
        if (gated)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                ahead_up[j] = right ? pre_up_r.load(row, j) : pre_up.load(row, j);
    };
    load(t.row0(0), false);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        if (b * 64 >= at.n)
            break;
        const int row = t.row0(b);
        f32x4 v[8], u[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
            v[c] = u[c] = f.acc[c][b];
        if (a.act != MOE_ACT_NONE)
#pragma unroll
            for (int right = 0; right < 2; ++right) {
                put_pieces(place, ahead, 0, at.lane);
                if (gated)
                    put_pieces(place, ahead_up, 1, at.lane);
                load(right ? t.row0(min(b + 1, NB - 1)) : row, !right);
                if (gated) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const f32x4 z = get_block(place, c, at.lane), zu = get_block(place, 4 + c, at.lane);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float g = z[j], x = v[right * 4 + c][j], s = sigmoid(g);
                            v[right * 4 + c][j] = x * zu[j] * (s * (1.0f + g * (1.0f - s)));
                            u[right * 4 + c][j] = x * (g * s);
                        }
                    }
                } else {
                    f32x4 z[4], w[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        z[c] = get_block(place, c, at.lane);
                        w[c] = v[right * 4 + c];
                    }
                    apply_slope(w, z, a.act);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        v[right * 4 + c] = w[c];
                }
            }
        if (a.out) {
            store_blocks<16>(place, v, out, row);
            if (gated)
                store_blocks<16>(place, u, out_up, row);
        }
        if (a.codes) {
            const float scale = scale_of(row_top(v));
            store_codes(place, v, scale, codes, row);
            store_scale(a, at, row, gated ? 2 : 1, 0, scale);
            if (gated) {
                const float scale_up = scale_of(row_top(u));
                store_codes(place, u, scale_up, codes_up, row);
                store_scale(a, at, row, 2, 1, scale_up);
            }
        }
    }
}

// A workgroup's walk over its list of tiles.
template <bool DX, bool GATED>
struct Walk {
    typedef CodeTile<GATED> T;
    static constexpr int kCols = GATED ? 128 : 256;  // output columns of a tile
    typedef TileList<DX ? kDx : kForward, kCols, Fp8> List;
    const Fp8 &a;
    MOE_LDS char *lds;
    List list;
    T t;
    int i;
    Work k;
    bool more;

    // blocks of 64 rows that the tile is run for
    __device__ __forceinline__ int blocks() const { return k.n <= 64 ? 1 : k.n <= 128 ? 2 : 4; }

    // Goes to the next tile, if there is one, and starts its first loads.
    __device__ __forceinline__ void next()
    {
        more = list.next(a, i, k);
        ++i;
        if (!more)
            return;
        T::keep_uniform(k.e);
        T::keep_uniform(k.first);
        T::keep_uniform(k.n);
        T::keep_uniform(k.c0);
        const int nbc = code_blocks(a.C), pitch = a.R * a.segments;
        const int64_t half = static_cast<int64_t>(k.e) * (GATED ? 2 : 1);
        const uint8_t *w = a.w + (half * a.C + k.c0) * pitch;
        t.init(w, w + static_cast<int64_t>(a.C) * pitch, min(kCols, a.C - k.c0), a.q + static_cast<int64_t>(k.first) * pitch,
               k.n, a.xs + static_cast<int64_t>(k.first) * a.xs_cols, a.xs_cols, a.R, a.segments);
        // (a wave past the last column takes the last block's)
        const int block = min(k.c0 / kCodeBlock + (GATED ? 0 : t.wave() % 2), nbc - 1);
#pragma unroll
        for (int g = 0; g < (GATED ? 2 : 1); ++g)
            t.ws[g] = (const MOE_SCALAR float *)(a.ws + ((half + g) * nbc + block) * t.steps);
        t.start(lds, blocks());
    }

    // A tile of at most NB blocks, from its first loads' arrival; the next one's
    // loads run beside its results.
    template <int NB>
    __device__ __forceinline__ void tile()
    {
        typename T::template Regs<NB> f;
        t.all_uniform();
        t.run(f, lds);
        const int c = k.c0 + t.col0() / (GATED ? 2 : 1);
        const Where at{k.e, k.first, k.n, c, a.C - c, fresh_lane()};
        next();
        if constexpr (DX)
            finish_dx(a, t, f, at, lds);
        else
            finish_forward<GATED>(a, t, f, at, lds);
    }
};

template <bool DX, bool GATED>
__global__ __launch_bounds__(512) void expert_fp8_kernel(Fp8 a)
{
    typedef Walk<DX, GATED> W;
    __shared__ __align__(1024) char shared[W::T::kLdsBytes + W::List::kBytes];
    W w{a, (MOE_LDS char *)shared};
    w.list.build(a, reinterpret_cast<int32_t *>(shared + W::T::kLdsBytes));
    w.i = 0;
    w.next();
    while (w.more) {
        const int nb = w.blocks();
        if (nb == 4)
            w.template tile<4>();
        else if (nb == 2)
            w.template tile<2>();
        else
            w.template tile<1>();
    }
}

// Rows of a tile of 256 columns (128 of a gated product): the smallest of which
// the call has no more than CUs.
int tile_height(int E, int64_t max_rows, int col_tiles)
{
    for (int h = 64; h < 256; h *= 2)
        if (max_row_tiles(max_rows, E, h) * col_tiles <= kCus)
            return h;
    return 256;
}

// As grid_for of the bf16 products.
dim3 grid_for(int64_t n) { return dim3(static_cast<unsigned>(n + 14 < kCus ? (n + 14) / 8 * 8 : kCus)); }

template <bool DX, bool GATED>
hipError_t launch(Fp8 &a, int64_t max_rows, hipStream_t stream)
{
    const int col_tiles = (a.C + (GATED ? 127 : 255)) / (GATED ? 128 : 256);
    a.max_rows = static_cast<int>(max_rows);
    a.height = tile_height(a.E, max_rows, col_tiles);
    expert_fp8_kernel<DX, GATED><<<grid_for(max_row_tiles(max_rows, a.E, a.height) * col_tiles), 512, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_fp8(const void *x, const float *xs, int xs_cols, const int32_t *offsets, const void *w,
                             const float *ws, const float *bias, int act, const void *residual, int E, int64_t max_rows,
                             int K, int N, void *out, void *codes, float *scales, void *preact, hipStream_t stream)
{
    Fp8 a{};
    a.q = static_cast<const uint8_t *>(x), a.xs = xs, a.xs_cols = xs_cols, a.offsets = offsets;
    a.w = static_cast<const uint8_t *>(w), a.ws = ws, a.bias = bias, a.act = act;
    a.residual = static_cast<const uint16_t *>(residual), a.E = E, a.R = K, a.segments = 1, a.C = N;
    a.out = out, a.codes = static_cast<uint8_t *>(codes), a.scales = scales, a.preact = static_cast<uint16_t *>(preact);
    return act == MOE_ACT_SWIGLU ? launch<false, true>(a, max_rows, stream) : launch<false, false>(a, max_rows, stream);
}

hipError_t launch_expert_fp8_dx(const void *dy, const float *dys, const int32_t *offsets, const void *wt,
                                const float *wts, int halves, int act, const void *z, int E, int64_t max_rows, int K,
                                int N, void *dx, void *codes, float *scales, hipStream_t stream)
{
    Fp8 a{};
    a.q = static_cast<const uint8_t *>(dy), a.xs = dys, a.xs_cols = halves * code_blocks(N), a.offsets = offsets;
    a.w = static_cast<const uint8_t *>(wt), a.ws = wts, a.act = act, a.z = static_cast<const uint16_t *>(z);
    a.E = E, a.R = N, a.segments = halves, a.C = K;
    a.out = dx, a.codes = static_cast<uint8_t *>(codes), a.scales = scales;
    return launch<true, false>(a, max_rows, stream);
}

}  // namespace moe
