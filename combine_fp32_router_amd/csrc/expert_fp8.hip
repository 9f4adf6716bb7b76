// The experts' products of E4M3 rows and weights, and the gradient of their rows:
//
//   forward   z = sum over blocks b of 128 of  xs[p, b] ws[n / 128, b] (xc wc)_b + bias,  y = act(z) + residual
//   dx        g = the same of dy's codes and the transposed weights',  dx = act'(z_prev) g
//
// The results leave in bf16, in codes with a scale for each 128, or both.
//
// Many rows an expert are bound by the matrix cores' power (fp8_tile.hpp) and by the
// results, which leave from all CUs at once while no matrix core works (the next tile's
// first loads are under way then, but stand in one count with the stores): 16384 rows of 8,
// 7168 -> 2048 gated with z kept, then 2048 -> 7168: 802 us, 1.8 PFLOP/s.  dx of 16384 rows,
// 2048 <- 7168: 267 us, and through SwiGLU with its codes 325, 335 MB in place of 67 (6%
// more with its inputs' lines asked for ahead of the product).  Few and some rows are bound by the weights: 64 rows of each of 64, 2048 -> 4096: 123 us, 4.7 TB/s.  (A kernel
// that streams weights to registers past 64 rows in LDS, two workgroups a CU, took 120
// there, but 191 against 173 for 32 x 64 rows, 7168 -> 2048 gated.)
#include "fp8_args.hpp"
#include "fp8_tile.hpp"
#include "launch.hpp"

#include <type_traits>

namespace moe {
namespace {

// Where a tile's results go: its rows first .. first + n - 1, this wave's columns
// from c on, `inside` of them (or more) the array's.
struct Where {
    int e, first, n, c, inside, lane;
};

// The results of 16 rows of a wave at a time, 64 columns of bf16 or all of the
// codes, through LDS into 16-byte pieces of whole rows, P a row (expert_finish.hpp).
// A lane's offsets into parts of arrays of one pitch are the same ones; the parts'
// places are in their descriptors.
struct Part {
    __amdgpu_buffer_rsrc_t rsrc;
    int pitch, inside;  // bytes of a row, from this part's column on
    // The part of p [.., cols] from column c on, of the tile's rows.
    __device__ __forceinline__ Part(const Where &at, const void *p, int cols, int size, int c, int inside_)
        : rsrc(row_rsrc(const_cast<char *>(static_cast<const char *>(p)) + (static_cast<int64_t>(at.first) * cols + c) * size,
                        p ? max(0, (at.n * cols - c) * size) : 0)),
          pitch(cols * size), inside(inside_ * size)
    {
    }
    template <int P>
    __device__ __forceinline__ int offset(const Where &at, int row, int j, int lane) const
    {
        const int r = row + 64 / P * j + lane / P;
        return r < at.n && lane % P * 16 < inside ? r * pitch + lane % P * 16 : kOutside;
    }
    template <int P>
    __device__ __forceinline__ void load(const Where &at, int row, int lane, u32x4 (&v)[P / 4]) const
    {
#pragma unroll
        for (int j = 0; j < P / 4; ++j)
            v[j] = load_cached(rsrc, offset<P>(at, row, j, lane));
    }
    template <int P>
    __device__ __forceinline__ void store(const Where &at, int row, int lane, const MOE_LDS char *__restrict__ place) const
    {
#pragma unroll
        for (int j = 0; j < P / 4; ++j)
            __builtin_amdgcn_raw_buffer_store_b128(*reinterpret_cast<const MOE_LDS u32x4 *>(place + Place::piece<P>(j, lane)),
                                                   rsrc, offset<P>(at, row, j, lane), 0, 0);
    }
};

__device__ __forceinline__ void put_bf16(MOE_LDS char *__restrict__ place, const f32x4 *v, int lane)
{
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<MOE_LDS u32x2 *>(place + Place::half(c, lane)) = round4(v[c]);
}
template <int BLOCKS>
__device__ __forceinline__ void put_codes(MOE_LDS char *__restrict__ place, const f32x4 (&v)[BLOCKS], float scale, int lane)
{
    const int r = lane % 16;
    const Coder coder(scale);
#pragma unroll
    for (int c = 0; c < BLOCKS; ++c)
        *reinterpret_cast<MOE_LDS uint32_t *>(place + r * 256 + (c ^ r) * 16 + lane / 16 * 4) =
            coder.codes4(v[c][0], v[c][1], v[c][2], v[c][3]);
}
// Loaded pieces of 16 rows, eight a row, into LDS: as the first or the second eight.
__device__ __forceinline__ void put_pieces(MOE_LDS char *__restrict__ place, const u32x4 (&in)[2], int second, int lane)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int row = 8 * j + lane / 8;
        *reinterpret_cast<MOE_LDS u32x4 *>(place + row * 256 + ((lane % 8 + 8 * second) ^ row) * 16) = in[j];
    }
}
__device__ __forceinline__ f32x4 get_block(const MOE_LDS char *__restrict__ place, int c, int lane)
{
    return widen4(*reinterpret_cast<const MOE_LDS u32x2 *>(place + Place::half(c, lane)));
}

// The scale of the block that this wave's columns begin, of the 16 rows from `row`.
__device__ __forceinline__ void store_scale(const Fp8 &a, const Where &at, int row, int halves, int half, float scale, int lane)
{
    const int r = row + lane % 16;
    if (lane < 16 && r < at.n && at.inside > 0)
        a.scales[((static_cast<int64_t>(at.first) + r) * halves + half) * code_blocks(a.C) + at.c / kCodeBlock] = scale;
}

// What a tile's results take from memory, a piece of 16 rows by 64 columns (of one or
// two arrays) after the other.  All of it is there before the product where the tile
// is short; beside 256 rows' accumulators there is room for one piece ahead, the first
// asked for in front of the next tile's first loads: behind them, it would come after.
template <int ARRAYS, int PIECES>
struct Ahead {
    static constexpr int kDepth = PIECES <= 4 ? PIECES : 1;
    u32x4 v[kDepth][ARRAYS][2];
};

// Forward: bias, pre-activations, activation, residual.  The accumulators are
// changed in place, a block of 64 rows after the other: beside 128 of them there is
// no room for copies, nor for addresses kept from one 64 columns to the next (hence
// the lane as a value of its own in each).  GATED: blocks 0, 1, 4, 5 are the gate's,
// 2, 3, 6, 7 the up half's.
template <bool GATED, int NB>
struct Forward {
    static constexpr int kHalves = GATED ? 1 : 2, wide = GATED ? 2 : 1;  // of 64 columns
    typedef CodeTile<GATED> T;
    const Fp8 &a;
    const T &t;
    const Where &at;
    Ahead<1, NB * kHalves> ahead;
    static constexpr bool kKept = NB < 4;  // the bias, for all of the tile
    f32x4 bias[kKept ? 8 : 1];

    // Of 16 columns: block i of the wave's, or of the up half's after the gate's four.
    __device__ __forceinline__ f32x4 bias_of(int i, int lane) const
    {
        const __amdgpu_buffer_rsrc_t r = row_rsrc(
            const_cast<float *>(a.bias) + static_cast<int64_t>(at.e) * wide * a.C + at.c, max(0, at.inside + (wide - 1) * a.C) * 4);
        const int c = (GATED ? i % 4 : i) * 16;
        return __builtin_bit_cast(f32x4, load_cached(r, c < at.inside ? (c + lane / 16 * 4 + (GATED ? i / 4 * a.C : 0)) * 4 : kOutside));
    }
    __device__ __forceinline__ void load(int piece, int lane)
    {
        if (piece < NB * kHalves && a.residual) {
            const int right = piece % kHalves;
            Part(at, a.residual, a.C, 2, at.c + 64 * right, at.inside - 64 * right)
                .template load<8>(at, t.row0(piece / kHalves), lane, ahead.v[piece % ahead.kDepth][0]);
        }
    }
    __device__ __forceinline__ void begin()
    {
#pragma unroll
        for (int i = 0; i < ahead.kDepth; ++i)
            load(i, at.lane);
        if (kKept && a.bias)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                bias[kKept ? i : 0] = bias_of(i, at.lane);
    }

    __device__ __forceinline__ void finish(const typename T::template Regs<NB> &f, MOE_LDS char *lds)
    {
        MOE_LDS char *place = t.out_place(lds);
        int lane = at.lane;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (b * 64 >= at.n)
                break;
            const int row = t.row0(b);
            f32x4 y[4 * kHalves];
#pragma unroll
            for (int right = 0; right < kHalves; ++right) {
                asm volatile("" : "+v"(lane));
                f32x4 g[4], u[GATED ? 4 : 1];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    g[i] = f.acc[GATED ? i / 2 * 4 + i % 2 : right * 4 + i][b];
                    if (GATED)
                        u[i] = f.acc[(i / 2 * 4 + i % 2 + 2) % 8][b];
                    if (a.bias) {
                        g[i] += kKept ? bias[kKept ? right * 4 + i : 0] : bias_of(right * 4 + i, lane);
                        if (GATED)
                            u[i] += kKept ? bias[kKept ? 4 + i : 0] : bias_of(4 + i, lane);
                    }
                }
                if (a.preact) {
                    put_bf16(place, g, lane);
                    Part(at, a.preact, wide * a.C, 2, at.c + 64 * right, at.inside - 64 * right).template store<8>(at, row, lane, place);
                    if (GATED) {
                        put_bf16(place, u, lane);
                        Part(at, a.preact, wide * a.C, 2, at.c + a.C, at.inside).template store<8>(at, row, lane, place);
                    }
                }
                if (GATED) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        g[i / 4][i % 4] *= sigmoid(g[i / 4][i % 4]) * u[GATED ? i / 4 : 0][i % 4];
                } else {
                    apply_act(g, a.act);
                }
                if (a.residual) {
                    const int piece = b * kHalves + right;
                    put_pieces(place, ahead.v[piece % ahead.kDepth][0], 0, lane);
                    // (in front of this block's stores: waiting for it is then not waiting for them)
                    load(piece + ahead.kDepth, lane);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        g[i] += get_block(place, i, lane);
                }
                if (a.out) {
                    put_bf16(place, g, lane);
                    Part(at, a.out, a.C, 2, at.c + 64 * right, at.inside - 64 * right).template store<8>(at, row, lane, place);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[right * 4 + i] = g[i];
            }
            if (a.codes) {
                asm volatile("" : "+v"(lane));
                uint32_t top = row_top(y);
                if (GATED)
                    top = t.both_halves(lds, b, top, lane);
                const float scale = scale_of(top);
                put_codes(place, y, scale, lane);
                Part(at, a.codes, a.C, 1, at.c, at.inside).template store<4 * kHalves>(at, row, lane, place);
                if (!GATED || t.col0() == 0)
                    store_scale(a, at, row, 1, 0, scale, lane);
            }
        }
    }
};

// dx: through the activation that made the product's input (SWIGLU: MOE_ACT_SWIGLU).
template <bool SWIGLU, int NB>
struct Back {
    typedef CodeTile<false> T;
    static constexpr int halves = SWIGLU ? 2 : 1;
    const Fp8 &a;
    const T &t;
    const Where &at;
    Ahead<halves, 2 * NB> ahead;

    __device__ __forceinline__ void load(int piece, int lane)
    {
        if (piece < 2 * NB && (SWIGLU || a.act != MOE_ACT_NONE)) {
            const int right = piece % 2;
#pragma unroll
            for (int h = 0; h < halves; ++h)
                Part(at, a.z, halves * a.C, 2, at.c + h * a.C + 64 * right, at.inside - 64 * right)
                    .template load<8>(at, t.row0(piece / 2), lane, ahead.v[piece % ahead.kDepth][h]);
        }
    }
    __device__ __forceinline__ void begin()
    {
#pragma unroll
        for (int i = 0; i < ahead.kDepth; ++i)
            load(i, at.lane);
    }
    __device__ __forceinline__ void store(MOE_LDS char *place, const f32x4 *v, int row, int right, int half, int lane) const
    {
        put_bf16(place, v, lane);
        Part(at, a.out, halves * a.C, 2, at.c + half * a.C + 64 * right, at.inside - 64 * right).template store<8>(at, row, lane, place);
    }
    __device__ __forceinline__ void store_coded(MOE_LDS char *place, const f32x4 (&v)[8], int row, int half, int lane) const
    {
        const float scale = scale_of(row_top(v));
        put_codes(place, v, scale, lane);
        Part(at, a.codes, halves * a.C, 1, at.c + half * a.C, at.inside).template store<8>(at, row, lane, place);
        store_scale(a, at, row, halves, half, scale, lane);
    }

    __device__ __forceinline__ void finish(const typename T::template Regs<NB> &f, MOE_LDS char *lds)
    {
        MOE_LDS char *place = t.out_place(lds);
        int lane = at.lane;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if (b * 64 >= at.n)
                break;
            const int row = t.row0(b);
            f32x4 v[8], u[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
                v[c] = f.acc[c][b];
#pragma unroll
            for (int right = 0; right < 2; ++right) {
                asm volatile("" : "+v"(lane));
                if (SWIGLU || a.act != MOE_ACT_NONE) {
                    const int piece = 2 * b + right;
#pragma unroll
                    for (int h = 0; h < halves; ++h)
                        put_pieces(place, ahead.v[piece % ahead.kDepth][h], h, lane);
                    load(piece + ahead.kDepth, lane);
#pragma unroll
                    for (int c = 4 * right; c < 4 * right + 4; ++c) {
                        const f32x4 z[1] = {get_block(place, c % 4, lane)};
                        if constexpr (SWIGLU) {
                            swiglu_slopes(v[c], u[c], z[0], get_block(place, 4 + c % 4, lane));
                        } else {
                            f32x4 w[1] = {v[c]};
                            apply_slope(w, z, a.act);
                            v[c] = w[0];
                        }
                        __builtin_amdgcn_sched_barrier(0);  // (read together, the blocks take registers that are not there)
                    }
                }
                if (a.out) {
                    store(place, v + 4 * right, row, right, 0, lane);
                    if (SWIGLU)
                        store(place, u + 4 * right, row, right, 1, lane);
                }
            }
            if (a.codes) {
                asm volatile("" : "+v"(lane));
                store_coded(place, v, row, 0, lane);
                if (SWIGLU) {
                    asm volatile("" : "+v"(lane));
                    store_coded(place, u, row, 1, lane);
                }
            }
        }
    }
};

// A workgroup's walk over its list of tiles.
template <Kind KIND>
struct Walk {
    static constexpr bool GATED = KIND == kGated, DX = KIND >= kBack;
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
        const int c = k.c0 + t.col0() / (GATED ? 2 : 1);
        Where at{k.e, k.first, k.n, c, a.C - c, fresh_lane()};
        std::conditional_t<DX, Back<KIND == kBackGated, NB>, Forward<GATED, NB>> results{a, t, at};
        if (NB < 4)
            results.begin();
        t.run(f, lds);
        if (NB == 4)
            results.begin();
        next();
        T::keep_uniform(at.e);
        T::keep_uniform(at.first);
        T::keep_uniform(at.n);
        T::keep_uniform(at.c);
        T::keep_uniform(at.inside);
        results.finish(f, lds);
    }
};

template <Kind KIND>
__global__ __launch_bounds__(512) void expert_fp8_kernel(Fp8 a)
{
    typedef Walk<KIND> W;
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

template <Kind KIND>
hipError_t launch(Fp8 &a, int64_t max_rows, hipStream_t stream)
{
    const int col_tiles = (a.C + Walk<KIND>::kCols - 1) / Walk<KIND>::kCols;
    a.max_rows = static_cast<int>(max_rows);
    a.height = tile_height(a.E, max_rows, col_tiles);
    expert_fp8_kernel<KIND><<<grid_for(max_row_tiles(max_rows, a.E, a.height) * col_tiles), 512, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_fp8(const void *x, const float *xs, int xs_cols, const int32_t *offsets, const void *w,
                             const float *ws, const float *bias, int act, const void *residual, int E, int64_t max_rows,
                             int K, int N, void *out, void *codes, float *scales, void *preact, void *workspace,
                             hipStream_t stream)
{
    Fp8 a{};
    a.q = static_cast<const uint8_t *>(x), a.xs = xs, a.xs_cols = xs_cols, a.offsets = offsets;
    a.w = static_cast<const uint8_t *>(w), a.ws = ws, a.bias = bias, a.act = act;
    a.residual = static_cast<const uint16_t *>(residual), a.E = E, a.R = K, a.segments = 1, a.C = N;
    a.out = out, a.codes = static_cast<uint8_t *>(codes), a.scales = scales, a.preact = static_cast<uint16_t *>(preact);
    const Kind kind = act == MOE_ACT_SWIGLU ? kGated : kPlain;
    const int wide = kind == kGated ? 2 : 1;
    const bool room = workspace && few_fp8_bytes(wide, 1, E, max_rows, K, N);
    if (few_fp8_pay(wide, E, max_rows, K, N, codes && !room))
        return launch_fp8_few(kind, a, max_rows, workspace, stream);
    return act == MOE_ACT_SWIGLU ? launch<kGated>(a, max_rows, stream) : launch<kPlain>(a, max_rows, stream);
}

size_t expert_fp8_workspace_bytes(int act, int E, int64_t max_rows, int K, int N)
{
    const int wide = act == MOE_ACT_SWIGLU ? 2 : 1;
    const bool few = max_rows > 0 && few_fp8_pay(wide, E, max_rows, K, N, false);
    return few ? static_cast<size_t>(few_fp8_bytes(wide, 1, E, max_rows, K, N)) : 0;
}

size_t expert_fp8_dx_workspace_bytes(int halves, int act, int E, int64_t max_rows, int K, int N)
{
    const bool few = max_rows > 0 && few_fp8_pay(1, E, max_rows, halves * N, K, false);
    return few ? static_cast<size_t>(few_fp8_bytes(1, act == MOE_ACT_SWIGLU ? 2 : 1, E, max_rows, halves * N, K)) : 0;
}

hipError_t launch_expert_fp8_dx(const void *dy, const float *dys, const int32_t *offsets, const void *wt,
                                const float *wts, int halves, int act, const void *z, int E, int64_t max_rows, int K,
                                int N, void *dx, void *codes, float *scales, void *workspace, hipStream_t stream)
{
    Fp8 a{};
    a.q = static_cast<const uint8_t *>(dy), a.xs = dys, a.xs_cols = halves * code_blocks(N), a.offsets = offsets;
    a.w = static_cast<const uint8_t *>(wt), a.ws = wts, a.act = act, a.z = static_cast<const uint16_t *>(z);
    a.E = E, a.R = N, a.segments = halves, a.C = K;
    a.out = dx, a.codes = static_cast<uint8_t *>(codes), a.scales = scales;
    const bool room = workspace && few_fp8_bytes(1, act == MOE_ACT_SWIGLU ? 2 : 1, E, max_rows, halves * N, K);
    if (few_fp8_pay(1, E, max_rows, halves * N, K, codes && !room))
        return launch_fp8_few(act == MOE_ACT_SWIGLU ? kBackGated : kBack, a, max_rows, workspace, stream);
    return act == MOE_ACT_SWIGLU ? launch<kBackGated>(a, max_rows, stream) : launch<kBack>(a, max_rows, stream);
}

}  // namespace moe
