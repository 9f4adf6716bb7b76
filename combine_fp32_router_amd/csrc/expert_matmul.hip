// The experts' products and their gradients: one matrix product per
// contiguous run of rows (moe_recv.h's grouped buffer), all runs in one launch.
//
//   forward   z = x W_e^T + b_e,  y = act(z) + residual
//   dx        g = dy W_e,         dx = act'(z_prev) g
//   dw        dW_e = dy_e^T x_e,  db_e = column sums of dy_e
//
// Large calls are bound by the matrix cores at the clock that the card's power
// leaves (one run of 8192 rows, 8192 x 7168: 735 us, 1.31 PFLOP/s), small ones by
// reading the weights, and small dw by writing them.  Eight uneven runs of 16384
// rows: K = 7168, N = 2048 gated, z kept, 810 us, 1.19 PFLOP/s; dx of N = 7168, K =
// 2048 through SwiGLU 485, its dw 445, 1.0 and 1.1 PFLOP/s.  64 uneven runs of 4099
// rows, K = 1024, N = 4096, bias and residual: 138 us, 4.4 TB/s.  dw in bf16 takes
// 0.8 to 0.9 of its fp32 time, accumulated 0.9 to 1.1 of it.  Where
// all tiles fit the card at once a call takes one tile's time: 8 uneven runs of
// 8192 rows, K = 768, N = 2048: dx 44 us, dw 46.
//
// Each is a tile of outputs, C[row, col] = sum_r Q[row, r] P[col, r], with
// `col` the output's contiguous dimension.  The MFMA's first operand is P, so
// a lane ends with four consecutive columns of one row and stores them at
// once.  An operand lies in memory with r contiguous (x, dy, and W in the
// forward pass) or with its own index contiguous (W in dx, both in dw).
#include "expert_tile.hpp"
#include "launch.hpp"

namespace moe {
namespace {

enum Op { kForward, kDx, kDw };

constexpr float kCutAbove = 1.7f;  // (TileList)
constexpr int kPartExperts = 256;   // (PartList)

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
    int height;             // forward, dx: rows of a tile
    // in parts: how many, their sums in the MFMA's layout, those of db
    int parts, tiles;       // (tiles: the most that the workspace is for)
    f32x4 *part;
    float *part_db;
};

// Results leave 16 rows of a wave's columns at a time.  A lane's share is
// four columns of each of FR blocks of 16 (the MFMA's layout); memory is
// read and written in 16-byte pieces of whole rows.  The two meet in 4 KiB of
// LDS a wave, rows of 256 bytes, piece p of row r kept at p ^ r: stored
// straight from the MFMA's layout, in pieces of 8 bytes, a tile's results cost
// L2 four requests a line (8192 x 8192, K = 1024: 165 us instead of 138; now 130).
// Rows and columns outside a tile are given offsets outside the buffer
// descriptors, whose reads return 0 and whose writes are dropped, so that the
// number of memory operations in flight is always known.
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x4 widen4(u32x2 v)
{
    return f32x4{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)};
}
__device__ __forceinline__ u32x2 round4(f32x4 f)
{
    const bf16x2 a = __builtin_convertvector((f32x2{f.x, f.y}), bf16x2);
    const bf16x2 b = __builtin_convertvector((f32x2{f.z, f.w}), bf16x2);
    return u32x2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
}

// The wave's LDS: 16 rows of up to sixteen 16-byte pieces.
struct Place {
    MOE_LDS char *base;
    // MFMA layout: four columns of block c, as bf16 or fp32 (c < 4)
    static __device__ __forceinline__ int half(int c)
    {
        const int lane = lane_id();
        return lane % 16 * 256 + ((c * 2 + lane / 32) ^ (lane % 16)) * 16 + lane / 16 % 2 * 8;
    }
    static __device__ __forceinline__ int whole(int c)
    {
        const int lane = lane_id();
        return lane % 16 * 256 + ((c * 4 + lane / 16) ^ (lane % 16)) * 16;
    }
    // row layout: piece lane%P of row (64 / P) j + lane/P
    template <int P>
    static __device__ __forceinline__ int piece(int j)
    {
        const int lane = lane_id(), row = 64 / P * j + lane / P;
        return row * 256 + ((lane % P) ^ row) * 16;
    }
};

// A row-major array in memory, from a tile's first row on: 16-byte pieces of
// its rows, P of them a wave's columns.
template <int P>
struct Pieces {
    __amdgpu_buffer_rsrc_t rsrc;
    int pitch, col, n;  // bytes of a row, this lane's offset in a row (kOutside past the columns), rows

    // Rows first .. first + n - 1 of `cols` columns of `size` bytes; the wave's
    // pieces start at column c, `inside` of its columns are the array's.
    __device__ __forceinline__ Pieces(const void *p, int64_t first, int n_, int cols, int size, int c, int inside)
        : rsrc(row_rsrc(const_cast<char *>(static_cast<const char *>(p)) + first * cols * size, n_ * cols * size)),
          pitch(cols * size), n(n_)
    {
        const int in_wave = lane_id() % P * (16 / size);
        col = in_wave < inside ? (c + in_wave) * size : kOutside;
    }
    static constexpr int kCount = P / 4;  // loads or stores for 16 rows
    // offset of the j-th of them, for the 16 rows from `row`
    __device__ __forceinline__ int at(int row, int j) const
    {
        const int r = row + 64 / P * j + lane_id() / P;
        return r < n && col != kOutside ? r * pitch + col : kOutside;
    }
    __device__ __forceinline__ u32x4 load(int row, int j) const
    {
        return __builtin_amdgcn_raw_buffer_load_b128(rsrc, at(row, j), 0, 0);
    }
    __device__ __forceinline__ void store(int row, int j, u32x4 v) const
    {
        __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, at(row, j), 0, 0);
    }
};

// Loaded pieces of 16 rows -> the MFMA layout (blocks first, first + step, ...
// of v), and back.
template <int P, int BLOCKS>
__device__ __forceinline__ void to_blocks(MOE_LDS char *__restrict__ lds, const u32x4 (&in)[P / 4], f32x4 (&v)[BLOCKS])
{
#pragma unroll
    for (int j = 0; j < P / 4; ++j)
        *reinterpret_cast<MOE_LDS u32x4 *>(lds + Place::piece<P>(j)) = in[j];
#pragma unroll
    for (int c = 0; c < BLOCKS; ++c)
        v[c] = widen4(*reinterpret_cast<const MOE_LDS u32x2 *>(lds + Place::half(c)));
}
template <int P, int BLOCKS>
__device__ __forceinline__ void store_blocks(MOE_LDS char *__restrict__ lds, const f32x4 (&v)[BLOCKS],
                                             const Pieces<P> &out, int row)
{
#pragma unroll
    for (int c = 0; c < BLOCKS; ++c)
        *reinterpret_cast<MOE_LDS u32x2 *>(lds + Place::half(c)) = round4(v[c]);
#pragma unroll
    for (int j = 0; j < P / 4; ++j)
        out.store(row, j, *reinterpret_cast<const MOE_LDS u32x4 *>(lds + Place::piece<P>(j)));
}

// Forward: bias, pre-activations, activation, residual.  GATED: blocks 0, 1, 4,
// 5 of v are the gate's, 2, 3, 6, 7 the up half's.
template <int FR, bool GATED>
struct FinishForward {
    static constexpr int kBlocks = GATED ? FR / 2 : FR, P = 2 * kBlocks;
    const Args &a;
    MOE_LDS char *lds;
    Pieces<P> out, res, pre, pre_up;
    f32x4 bias[FR];
    u32x4 ahead[P / 4];  // the residual's next 16 rows

    __device__ __forceinline__ FinishForward(const Args &a_, MOE_LDS char *lds_, int e, int first, int n, int c, int inside, int row)
        : a(a_), lds(lds_), out(a.out, first, n, a.C, 2, c, inside), res(a.residual ? a.residual : a.q, first, n, a.C, 2, c, inside),
          pre(a.preact ? a.preact : a.q, first, n, GATED ? 2 * a.C : a.C, 2, c, inside),
          pre_up(a.preact ? a.preact : a.q, first, n, GATED ? 2 * a.C : a.C, 2, GATED ? c + a.C : c, inside)
    {
        if (a.bias) {
            const float *b = a.bias + static_cast<int64_t>(e) * (GATED ? 2 : 1) * a.C + c + lane_id() / 16 * 4;
#pragma unroll
            for (int i = 0; i < FR; ++i) {
                const int o = GATED ? i / 4 * 32 + i % 2 * 16 : i * 16;
                bias[i] = f32x4{};
                if (o < inside)
                    bias[i] = *reinterpret_cast<const f32x4 *>(b + o + (GATED && i / 2 % 2 ? a.C : 0));
            }
        }
        if (a.residual)
            load(row);
    }
    __device__ __forceinline__ void load(int row)
    {
#pragma unroll
        for (int j = 0; j < P / 4; ++j)
            ahead[j] = res.load(row, j);
    }
    __device__ __forceinline__ void operator()(int row, int next, f32x4 (&v)[FR])
    {
        f32x4 y[kBlocks], add[kBlocks];
        if (a.residual) {
            to_blocks<P>(lds, ahead, add);
            load(next);  // in front of this block's stores: waiting for it is then not waiting for them
        }
        if (a.bias)
#pragma unroll
            for (int i = 0; i < FR; ++i)
                v[i] += bias[i];
        if constexpr (GATED) {
            f32x4 g[kBlocks], u[kBlocks];
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                g[i] = v[i / 2 * 4 + i % 2];
                u[i] = v[i / 2 * 4 + i % 2 + 2];
            }
            if (a.preact) {
                store_blocks<P>(lds, g, pre, row);
                store_blocks<P>(lds, u, pre_up, row);
            }
#pragma unroll
            for (int i = 0; i < 4 * kBlocks; ++i) {
                const float x = g[i / 4][i % 4];
                y[i / 4][i % 4] = x * sigmoid(x) * u[i / 4][i % 4];
            }
        } else {
            if (a.preact)
                store_blocks<P>(lds, v, pre, row);
            apply_act(v, a.act);
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
                y[i] = v[i];
        }
        if (a.residual)
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
                y[i] += add[i];
        store_blocks<P>(lds, y, out, row);
    }
};

// dx: through the activation that made the product's input.
template <int FR>
struct FinishDx {
    static constexpr int P = 2 * FR;
    const Args &a;
    MOE_LDS char *lds;
    const bool gated;
    Pieces<P> out, out_up, pre, pre_up;
    u32x4 ahead[P / 4], ahead_up[P / 4];

    __device__ __forceinline__ FinishDx(const Args &a_, MOE_LDS char *lds_, int first, int n, int c, int inside, int row)
        : a(a_), lds(lds_), gated(a_.act == MOE_ACT_SWIGLU), out(a.out, first, n, gated ? 2 * a.C : a.C, 2, c, inside),
          out_up(a.out, first, n, gated ? 2 * a.C : a.C, 2, gated ? c + a.C : c, inside),
          pre(a.z ? a.z : a.q, first, n, gated ? 2 * a.C : a.C, 2, c, inside),
          pre_up(a.z ? a.z : a.q, first, n, gated ? 2 * a.C : a.C, 2, gated ? c + a.C : c, inside)
    {
        load(row);
    }
    __device__ __forceinline__ void load(int row)
    {
        if (a.act == MOE_ACT_NONE)
            return;
#pragma unroll
        for (int j = 0; j < P / 4; ++j)
            ahead[j] = pre.load(row, j);
        if (gated)
#pragma unroll
            for (int j = 0; j < P / 4; ++j)
                ahead_up[j] = pre_up.load(row, j);
    }
    __device__ __forceinline__ void operator()(int row, int next, f32x4 (&v)[FR])
    {
        if (a.act != MOE_ACT_NONE) {
            f32x4 z[FR];
            to_blocks<P>(lds, ahead, z);
            if (gated) {
                f32x4 u[FR];
                to_blocks<P>(lds, ahead_up, u);
                load(next);
#pragma unroll
                for (int i = 0; i < 4 * FR; ++i) {
                    const float g = z[i / 4][i % 4], up = u[i / 4][i % 4], x = v[i / 4][i % 4], s = sigmoid(g);
                    v[i / 4][i % 4] = x * up * (s * (1.0f + g * (1.0f - s)));
                    u[i / 4][i % 4] = x * (g * s);
                }
                store_blocks<P>(lds, u, out_up, row);
            } else {
                load(next);
                apply_slope(v, z, a.act);
            }
        }
        store_blocks<P>(lds, v, out, row);
    }
};

template <int FR>
struct FinishDw {
    const Args &a;
    MOE_LDS char *lds;
    const bool half;
    Pieces<2 * FR> out;      // bf16: all columns
    Pieces<16> lower, upper;  // fp32: 64 columns each

    __device__ __forceinline__ FinishDw(const Args &a_, MOE_LDS char *lds_, int64_t first, int n, int c, int inside)
        : a(a_), lds(lds_), half((a_.flags & MOE_GRAD_BF16) != 0), out(a.out, first, n, a.C, 2, c, inside),
          lower(a.out, first, n, a.C, 4, c, inside), upper(a.out, first, n, a.C, 4, c + 64, inside - 64)
    {
    }
    __device__ __forceinline__ void operator()(int row, int, f32x4 (&v)[FR])
    {
        if (half) {
            store_blocks<2 * FR>(lds, v, out, row);
            return;
        }
        fp32_half(lds, lower, row, v[0], v[1], v[2], v[3]);
        if constexpr (FR == 8)
            fp32_half(lds, upper, row, v[4], v[5], v[6], v[7]);
    }
    __device__ __forceinline__ void fp32_half(MOE_LDS char *__restrict__ place, const Pieces<16> &to, int row,
                                              f32x4 v0, f32x4 v1, f32x4 v2, f32x4 v3) const
    {
        const f32x4 v[4] = {v0, v1, v2, v3};
        u32x4 old[4];
        if (a.flags & MOE_GRAD_ACCUMULATE)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                old[j] = to.load(row, j);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<MOE_LDS f32x4 *>(place + Place::whole(c)) = v[c];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f32x4 x = *reinterpret_cast<const MOE_LDS f32x4 *>(place + Place::piece<16>(j));
            if (a.flags & MOE_GRAD_ACCUMULATE)
                x += __builtin_bit_cast(f32x4, old[j]);
            to.store(row, j, __builtin_bit_cast(u32x4, x));
        }
    }
};

// One tile of a workgroup's list.
struct Work {
    int e;           // expert
    int first, n;    // its rows of the output
    int c0;          // its first output column
    int r_first, R;  // dw: the expert's run
};

// The tiles of a call, in the order in which they are handed out: workgroup b
// takes entries b, b + gridDim.x, ...  Entry j runs on XCD j % 8, so every
// list is dealt out in eight contiguous parts (xcd_order).  Runs and list are
// worked out once, into LDS.
//
// forward, dx: tiles of `height` rows (256, 128 or 64, the host's choice), at
// first those of more than half of it, which all cost the same, then the runs'
// shorter ends.  The last round of whole tiles leaves workgroups idle: the
// ends go to them, 64 rows to each if they suffice, else whole and two at a
// time, or the round's tiles are cut to a half or a
// quarter of their rows and dealt out together with the ends, if by the
// tiles' costs that ends sooner (5000 rows, K = N = 4096, 320 tiles: 131 us
// against 171; 10000 rows, K = N = 2048, also 320: 76 against 97.  Ends of 33, 109,
// 25 and 52 rows behind 512 tiles: 432 us with the 109 cut, 455 without).
//
// dw (TileList<kDw>): an expert's tiles cost what its run is long, and the
// longest run's could outlast all others: up to 64 experts' are cut to 128 or 64
// rows where one of 256 would take too much of the whole call, ordered by
// their cost, and every second round is dealt out backwards.
template <Op OP, int COLS>
struct TileList {
    static constexpr int kBytes = 4 * (3 * MOE_MAX_EXPERTS + 2);
    int32_t *starts;  // [E + 1] first rows of the runs
    int32_t *upto;    // [E] entries up to an expert's last (of whole tiles; dw: in the order of `experts`)
    int32_t *second;  // [E] the same of the ends, then their rows; dw: experts, those to come first first
    int E, height, end_rows, whole, ends, col_tiles;
    int nw, nw8, ne, end;  // entries: whole tiles, rounded up, ends, all
    int cut, full, parts;  // pieces that the last round's tiles are cut to, tiles before them, pieces

    __device__ __forceinline__ void build(const Args &a, int32_t *lds)
    {
        E = a.E;
        height = a.height;
        starts = lds;
        upto = lds + E + 1;
        second = upto + E;
        col_tiles = (a.C + COLS - 1) / COLS;
        for (int e = threadIdx.x; e <= E; e += blockDim.x)
            starts[e] = run_start(a.offsets, e, a.max_rows);
        __syncthreads();
        // (a branch on it that is not known to be a wave's makes the compiler take the
        // tiles' addresses for lanes' own, in loops around every load)
        const int w = static_cast<int>(uniform(threadIdx.x / kWave)), lane = lane_id();
        if (OP == kDw) {
            if (w == 0)
                order(a);
        } else if (w == 0) {
            const int all = count(upto, [&](int n) { return (n + height - 1) / height - short_end(n); });
            const int idle = static_cast<int>(gridDim.x) - all * col_tiles % static_cast<int>(gridDim.x);
            end_rows = height / 2;
            if (count(second, [&](int n) { return end_tiles(n, 64); }) * col_tiles <= idle)
                end_rows = 64;
            else
                count(second, [&](int n) { return short_end(n); });
            if (lane == 0)
                second[E] = end_rows;
        }
        __syncthreads();
        if (OP == kDw) {
            end = static_cast<int>(uniform(upto[E - 1]));
        } else {
            whole = static_cast<int>(uniform(upto[E - 1]));
            ends = static_cast<int>(uniform(second[E - 1]));
            end_rows = static_cast<int>(uniform(second[E]));
            nw = whole * col_tiles;
            ne = ends * col_tiles;
            const int groups = gridDim.x, left = nw % groups;
            full = nw - left;
            cut = 1;
            if (height == 256 && groups == kCus && left) {
                auto rounds = [&](int n) { return (n + kCus - 1) / kCus; };
                int least = 100 + rounds(max(ne - 2 * (groups - left), 0)) * 63;
                if (rounds(2 * left + ne) * 63 < least)
                    least = rounds(2 * left + ne) * 63, cut = 2;
                if (rounds(4 * left + ne) * 50 < least)
                    cut = 4;
            }
            parts = cut > 1 ? left * cut : 0;
            nw8 = cut > 1 ? full + (parts + 7) / 8 * 8 : (nw + 7) / 8 * 8;
            end = nw8 + (ne + 7) / 8 * 8;
        }
    }

    __device__ __forceinline__ ExpertRun run(int e) const
    {
        const int first = starts[e];
        return {first, max(starts[e + 1] - first, 0)};
    }

    // Writes the experts' counts, added up; the sum of all.
    template <typename F>
    __device__ __forceinline__ int count(int32_t *list, F of) const
    {
        int before = 0;
        for (int e0 = 0; e0 < E; e0 += kWave) {
            const int e = e0 + lane_id(), sum = before + wave_inclusive_scan(e < E ? of(run(e).n) : 0);
            if (e < E)
                list[e] = sum;
            before = static_cast<int>(lane_value(sum, kWave - 1));
        }
        return before;
    }

    // Whether the run's last tile is one of the ends.
    __device__ __forceinline__ int short_end(int n) const
    {
        return height > 64 && n % height > 0 && n % height <= height / 2;
    }
    __device__ __forceinline__ int end_tiles(int n, int rows) const
    {
        return short_end(n) ? (n % height + rows - 1) / rows : 0;
    }

    // dw.  Cost of a tile of 256 >> cut rows, in 1/16 of 64 r of a tile of 256:
    // the products' and the results'.
    static __device__ __forceinline__ int cost(int n, int cut)
    {
        const int steps = (n + kStep - 1) / kStep;
        return cut == 0 ? 16 * steps + 64 : cut == 1 ? 10 * steps + 40 : 7 * steps + 28;
    }
    __device__ __forceinline__ void order(const Args &a)
    {
        const int lane = lane_id();
        int before = 0;
        for (int e0 = 0; e0 < E; e0 += kWave) {
            const int e = e0 + lane, n = e < E ? run(e).n : 0;
            int cut = 0, at = e;
            if (E <= kWave) {
                const int tiles = ((a.rows + 255) / 256) * col_tiles;
                float share = e < E ? static_cast<float>(cost(n, 0)) * tiles / kCus : 0.0f;
#pragma unroll
                for (int o = 1; o < kWave; o <<= 1)
                    share += __shfl_xor(share, o);
                while (cut < 2 && cost(n, cut) > kCutAbove * share)
                    ++cut;
                const int c = e < E ? cost(n, cut) : -1;
                at = 0;
                for (int j = 0; j < E; ++j) {
                    const int other = lane_value(c, j);
                    at += other > c || (other == c && j < lane);
                }
            }
            if (e < E) {
                second[at] = e | cut << 16;
                upto[at] = (((a.rows + (256 >> cut) - 1) >> (8 - cut)) * col_tiles + 7) / 8 * 8;
            }
            // (this wave's own writes)
            const int sum = before + wave_inclusive_scan(e < E ? upto[e] : 0);
            if (e < E)
                upto[e] = sum;
            before = lane_value(sum, kWave - 1);
        }
    }

    // First i whose upto[i] is past entry j.
    __device__ __forceinline__ int holder(const int32_t *list, int j) const
    {
        int i = 0;
        for (int e0 = 0; e0 < E; e0 += kWave) {
            const int at = e0 + lane_id();
            i += __builtin_popcountll(__ballot(at < E && list[at] <= j));
        }
        return static_cast<int>(uniform(i));
    }

    // Moves this workgroup's count i to its next entry with work; false at the
    // end of its list.
    __device__ __forceinline__ bool next(const Args &a, int &i, Work &t) const
    {
        const int groups = gridDim.x, b = blockIdx.x;
        for (;; ++i) {
            int j = i * groups + (OP == kDw && i % 2 ? (groups / 8 - 1 - b / 8) * 8 + b % 8 : b);
            if (OP == kDw) {
                if (i * groups >= end)
                    return false;
                if (j >= end)
                    continue;
                const int at = holder(upto, j), entry = static_cast<int>(uniform(second[at]));
                const int before = at ? static_cast<int>(uniform(upto[at - 1])) : 0;
                const int shift = 8 - (entry >> 16), h = 1 << shift, row_tiles = (a.rows + h - 1) >> shift;
                const int id = xcd_order(j - before, row_tiles * col_tiles);
                if (id < 0)
                    continue;
                t.e = entry & 0xffff;
                const TileAt tile = grouped_order(id, row_tiles, col_tiles);
                const ExpertRun r = run(t.e);
                t.first = static_cast<int>(uniform(tile.row * h));
                t.n = min(h, a.rows - t.first);
                t.c0 = static_cast<int>(uniform(tile.col * COLS));
                t.r_first = static_cast<int>(uniform(r.first));
                t.R = static_cast<int>(uniform(r.n));
            } else {
                if (j >= nw8 && cut == 1) {
                    // the short ends: i0 whole tiles of this workgroup lie behind it
                    const int idle = groups - nw8 % groups, i0 = nw8 / groups + (b < nw8 % groups);
                    const int turn = i - i0;  // of this workgroup's ends
                    j = nw8 + (b < groups - idle ? 2 * idle + turn * groups + b
                               : turn < 2        ? turn * idle + b - (groups - idle)
                                                 : 2 * idle + (turn - 2) * groups + b);
                }
                if (j >= end)
                    return false;
                const bool end_tile = j >= nw8, part = cut > 1 && j >= full && !end_tile;
                int id = end_tile ? xcd_order(j - nw8, ne)
                         : part   ? xcd_order(j - full, parts)
                                  : xcd_order(j, cut > 1 ? full : nw);
                if (id < 0)
                    continue;
                int rows = height, skip = 0;  // of the tile, and in front of a piece of it
                if (part) {
                    rows = height / cut;
                    skip = id % cut * rows;
                    id = full + id / cut;
                }
                const TileAt at = grouped_order(id, end_tile ? ends : whole, col_tiles);
                const int32_t *list = end_tile ? second : upto;
                t.e = holder(list, at.row);
                const ExpertRun r = run(t.e);
                const int before = t.e ? list[t.e - 1] : 0;
                if (end_tile)
                    rows = end_rows, skip = r.n / height * height;
                const int in_run = static_cast<int>(uniform((at.row - before) * (end_tile ? rows : height) + skip));
                t.n = min(rows, static_cast<int>(uniform(r.n)) - in_run);
                if (t.n <= 0)  // a piece behind its run
                    continue;
                t.first = static_cast<int>(uniform(r.first)) + in_run;
                t.c0 = at.col * COLS;
                t.R = a.R;
            }
            return true;
        }
        return false;
    }
};

template <Op OP, bool GATED, int TILE_COLS>
__global__ __launch_bounds__(64 * kTileWaves) void expert_kernel(Args a)
{
    typedef Tile<TILE_COLS, OP == kForward, OP != kDw, GATED> T;
    constexpr int kCols = GATED ? T::kCols / 2 : T::kCols;  // output columns of a tile
    // one array: for two the compiler would wait for all loads before a read
    typedef TileList<OP, kCols> List;
    __shared__ __align__(1024) char shared[T::kLdsBytes + List::kBytes];
    MOE_LDS char *lds = (MOE_LDS char *)shared;
    List list;
    list.build(a, reinterpret_cast<int32_t *>(shared + T::kLdsBytes));

    T t;
    auto start = [&](const Work &k) {  // the loads of a tile's first stages
        t.R = k.R;
        if (OP == kForward) {
            const int64_t rows = static_cast<int64_t>(k.e) * (GATED ? 2 : 1) * a.C + k.c0;
            t.p.init(a.p + rows * a.R, a.p + (rows + a.C) * a.R, a.R, min(kCols, a.C - k.c0));
        } else if (OP == kDx) {
            t.p.init(a.p + static_cast<int64_t>(k.e) * a.C * a.R + k.c0, nullptr, a.C, min(kCols, a.C - k.c0));
        } else {
            t.p.init(a.p + static_cast<int64_t>(k.r_first) * a.C + k.c0, nullptr, a.C, min(kCols, a.C - k.c0));
        }
        if (OP == kDw)
            t.q.init(a.q + static_cast<int64_t>(k.r_first) * a.rows + k.first, nullptr, a.rows, k.n);
        else
            t.q.init(a.q + static_cast<int64_t>(k.first) * a.R, nullptr, a.R, k.n);
        t.start_rows(k.n, lds);
    };

    int i = 0;
    Work k;
    if (!list.next(a, i, k))
        return;
    start(k);
    for (;;) {
        t.clear();
        const bool sums = OP == kDw && a.db && k.c0 == 0;
        if (sums)
            t.template run_rows<OP == kDw>(k.n, lds);
        else
            t.template run_rows<false>(k.n, lds);
        Work after = k;
        ++i;
        const bool more = list.next(a, i, after);
        if (more)
            start(after);  // runs beside the rest of this tile
        if (sums) {
            // lanes l, l + 16, l + 32 and l + 48 hold parts of row l's and row l + 16's sums
            const int lane = lane_id();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float sum[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    sum[h] = t.sum[b][h] + __shfl_xor(t.sum[b][h], 16);
                    sum[h] += __shfl_xor(sum[h], 32);
                }
                const int row = t.row0(t.wave() % 2 * 2 + b) + lane % 32;
                if (lane < 32 && row < k.n) {
                    float *db = a.db + static_cast<int64_t>(k.e) * a.rows + k.first + row;
                    *db = ((a.flags & MOE_GRAD_ACCUMULATE) ? *db : 0.0f) + sum[lane / 16];
                }
            }
        }
        const int c = k.c0 + t.col0() / (GATED ? 2 : 1), inside = a.C - c;
        MOE_LDS char *place = t.out_place(lds);
        if constexpr (OP == kForward) {
            FinishForward<T::kFrags, GATED> f(a, place, k.e, k.first, k.n, c, inside, t.row0(0));
            t.finish(k.n, f);
        } else if constexpr (OP == kDx) {
            FinishDx<T::kFrags> f(a, place, k.first, k.n, c, inside, t.row0(0));
            t.finish(k.n, f);
        } else {
            FinishDw<T::kFrags> f(a, place, static_cast<int64_t>(k.e) * a.rows + k.first, k.n, c, inside);
            t.finish(k.n, f);
        }
        if (!more)
            return;
        k = after;
    }
}

// Few outputs of a long reduced length: every tile, of 64 x 128, is
// shared by up to `parts` workgroups, each of which takes a piece of the
// length and leaves its sums, as its accumulators hold them, in the workspace; a
// second kernel adds them in order and finishes the tile.  Two workgroups
// share a CU (THIN).  dw of 16384 rows, 512 x 512: 23 us, 100 in whole tiles;
// 8192 rows, 128 x 2048: 19 and 54; dx of 512 rows, 8192 -> 256: 21 and 54.
template <Op OP, bool GATED>
struct PartList {
    static constexpr int kCols = GATED ? 64 : 128;  // output columns of a tile
    static constexpr int kBytes = 4 * (2 * kPartExperts + 1);
    int32_t *starts, *upto;  // as in TileList; upto: not for dw
    int E, tiles, col_tiles, row_tiles;

    __device__ __forceinline__ void build(const Args &a, int32_t *lds)
    {
        E = a.E;
        starts = lds;
        upto = lds + E + 1;
        col_tiles = (a.C + kCols - 1) / kCols;
        row_tiles = (a.rows + 63) / 64;  // dw
        for (int e = threadIdx.x; e <= E; e += blockDim.x)
            starts[e] = run_start(a.offsets, e, a.max_rows);
        __syncthreads();
        tiles = E * row_tiles * col_tiles;
        if (OP != kDw) {
            if (uniform(threadIdx.x / kWave) == 0) {
                int before = 0;
                for (int e0 = 0; e0 < E; e0 += kWave) {
                    const int e = e0 + lane_id();
                    const int sum = before + wave_inclusive_scan(e < E ? (run(e).n + 63) / 64 : 0);
                    if (e < E)
                        upto[e] = sum;
                    before = lane_value(sum, kWave - 1);
                }
            }
            __syncthreads();
            tiles = min(static_cast<int>(uniform(upto[E - 1])) * col_tiles, a.tiles);
        }
    }
    __device__ __forceinline__ ExpertRun run(int e) const
    {
        const int first = starts[e];
        return {first, max(starts[e + 1] - first, 0)};
    }
    __device__ __forceinline__ ExpertRun uniform_run(int e) const
    {
        const ExpertRun r = run(e);
        return {static_cast<int>(uniform(r.first)), static_cast<int>(uniform(r.n))};
    }
    __device__ __forceinline__ Work at(const Args &a, int tile) const
    {
        Work t;
        t.c0 = tile % col_tiles * kCols;
        const int row = tile / col_tiles;
        if (OP != kDw) {
            t.e = 0;
            for (int e0 = 0; e0 < E; e0 += kWave) {
                const int e = e0 + lane_id();
                t.e += __builtin_popcountll(__ballot(e < E && upto[e] <= row));
            }
            t.e = static_cast<int>(uniform(t.e));
            const ExpertRun r = uniform_run(t.e);
            const int in_run = (row - (t.e ? static_cast<int>(uniform(upto[t.e - 1])) : 0)) * 64;
            t.first = r.first + in_run;
            t.n = min(64, r.n - in_run);
            t.R = a.R;
        } else {
            t.e = row / row_tiles;
            const ExpertRun r = uniform_run(t.e);
            t.first = row % row_tiles * 64;
            t.n = min(64, a.rows - t.first);
            t.r_first = r.first;
            t.R = r.n;
        }
        return t;
    }
    // r of a tile's part
    static __device__ __forceinline__ int share(const Args &a, int R)
    {
        return ((R + kStep - 1) / kStep + a.parts - 1) / a.parts * kStep;
    }
};

template <Op OP, bool GATED>
__global__ __launch_bounds__(64 * kTileWaves, 2) void expert_part_kernel(Args a)
{
    typedef Tile<128, OP == kForward, OP != kDw, GATED, true> T;
    typedef PartList<OP, GATED> List;
    __shared__ __align__(1024) char shared[T::kLdsBytes + List::kBytes];
    MOE_LDS char *lds = (MOE_LDS char *)shared;
    List list;
    list.build(a, reinterpret_cast<int32_t *>(shared + T::kLdsBytes));
    T t;
    for (int j = blockIdx.x; j < list.tiles * a.parts; j += gridDim.x) {
        const int tile = j / a.parts, part = j % a.parts;
        const Work k = list.at(a, tile);
        const int share = List::share(a, k.R), r0 = part * share;
        if (r0 >= k.R)
            continue;
        t.R = min(share, k.R - r0);
        if (OP != kDw) {
            if (OP == kForward) {
                const int64_t rows = static_cast<int64_t>(k.e) * (GATED ? 2 : 1) * a.C + k.c0;
                t.p.init(a.p + rows * a.R + r0, a.p + (rows + a.C) * a.R + r0, a.R, min(List::kCols, a.C - k.c0));
            } else {
                t.p.init(a.p + (static_cast<int64_t>(k.e) * a.R + r0) * a.C + k.c0, nullptr, a.C, min(128, a.C - k.c0));
            }
            t.q.init(a.q + static_cast<int64_t>(k.first) * a.R + r0, nullptr, a.R, k.n);
        } else {
            t.p.init(a.p + (static_cast<int64_t>(k.r_first) + r0) * a.C + k.c0, nullptr, a.C, min(128, a.C - k.c0));
            t.q.init(a.q + (static_cast<int64_t>(k.r_first) + r0) * a.rows + k.first, nullptr, a.rows, k.n);
        }
        t.start_rows(k.n, lds);
        t.clear();
        const bool sums = OP == kDw && a.db && k.c0 == 0;
        if (sums)
            t.template run_rows<OP == kDw>(k.n, lds);
        else
            t.template run_rows<false>(k.n, lds);
        f32x4 *to = a.part + ((static_cast<int64_t>(tile) * a.parts + part) * kTileWaves + t.wave()) * (2 * T::kFrags * kWave) +
                    lane_id();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < T::kFrags; ++c)
                to[(i * T::kFrags + c) * kWave] = T::read_acc(t.acc[c][0][i]);
        if (sums && t.wave() % 2 == 0) {  // (as in expert_kernel)
            const int lane = lane_id();
            float sum[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                sum[h] = t.sum[0][h] + __shfl_xor(t.sum[0][h], 16);
                sum[h] += __shfl_xor(sum[h], 32);
            }
            if (lane < 32)
                a.part_db[(static_cast<int64_t>(tile / list.col_tiles) * a.parts + part) * 64 + t.row0(0) + lane] =
                    sum[lane / 16];
        }
    }
}

// One wave for each 16 rows that a wave of the parts' kernel held: most of it
// is waiting for the parts.
template <Op OP, bool GATED>
__global__ __launch_bounds__(kWave) void expert_join_kernel(Args a)
{
    constexpr int kFrags = 4, kUnits = 2 * kTileWaves, kUnit = kFrags * kWave;  // of a tile's part, in f32x4
    typedef PartList<OP, GATED> List;
    __shared__ __align__(1024) char shared[4096 + List::kBytes];
    List list;
    list.build(a, reinterpret_cast<int32_t *>(shared + 4096));
    const int tile = blockIdx.x / kUnits, unit = blockIdx.x % kUnits, wave = unit / 2, lane = lane_id();
    if (tile >= list.tiles)
        return;
    const Work k = list.at(a, tile);
    const int share = List::share(a, k.R), live = k.R > 0 ? (k.R + share - 1) / share : 0;
    if (OP == kDw && a.db && k.c0 == 0 && unit == 0 && lane < k.n) {
        float sum = 0.0f;
        for (int p = 0; p < live; ++p)
            sum += a.part_db[(static_cast<int64_t>(tile / list.col_tiles) * a.parts + p) * 64 + lane];
        float *db = a.db + static_cast<int64_t>(k.e) * a.rows + k.first + lane;
        *db = ((a.flags & MOE_GRAD_ACCUMULATE) ? *db : 0.0f) + sum;
    }
    const int row = wave / 2 * 32 + unit % 2 * 16, c = k.c0 + wave % 2 * (64 / (GATED ? 2 : 1)), inside = a.C - c;
    if (row >= k.n)
        return;
    const f32x4 *from = a.part + (static_cast<int64_t>(tile) * a.parts * kUnits + unit) * kUnit + lane;
    f32x4 v[kFrags] = {};
#pragma unroll 4
    for (int p = 0; p < live; ++p)
#pragma unroll
        for (int b = 0; b < kFrags; ++b)
            v[b] += from[p * (kUnits * kUnit) + b * kWave];
    MOE_LDS char *place = (MOE_LDS char *)shared;
    if constexpr (OP == kForward) {
        FinishForward<kFrags, GATED> f(a, place, k.e, k.first, k.n, c, inside, row);
        f(row, row, v);
    } else if constexpr (OP == kDx) {
        FinishDx<kFrags> f(a, place, k.first, k.n, c, inside, row);
        f(row, row, v);
    } else {
        FinishDw<kFrags> f(a, place, static_cast<int64_t>(k.e) * a.rows + k.first, k.n, c, inside);
        f(row, row, v);
    }
}

// In how many parts a tile's reduced length R is best taken (1: not at all): as
// many as fill the card, of at least four steps of 64 each, where they save 16
// steps or more, of about 0.45 us, against the 5 us of the second kernel.
int parts_of(int64_t tiles, int E, int64_t R)
{
    const int64_t steps = R / kStep;
    if (tiles < 1 || tiles > kCus / 2 || E > kPartExperts)
        return 1;
    const int64_t n = steps / 4 < 2 * kCus / tiles ? steps / 4 : 2 * kCus / tiles;
    return n >= 2 && steps - steps / n >= 16 ? static_cast<int>(n) : 1;
}
constexpr int64_t kPartBytes = 64 * 128 * 4, kPartDbBytes = 64 * 4;  // of a part of a tile, and of a row of tiles

// Workgroups of a call of at most n tiles: one for each of the card's 256
// CUs, whose LDS it fills, each with a list of tiles.  (Each of the two lists
// is a whole number for each XCD: spare entries.)
dim3 grid_for(int64_t n) { return dim3(static_cast<unsigned>(n + 14 < kCus ? (n + 14) / 8 * 8 : kCus)); }

#define MOE_EXPERT(OP, GATED, COLS, TILES)                                                     \
    if ((COLS) == 128)                                                                         \
        expert_kernel<OP, GATED, 128><<<grid_for(TILES), 64 * kTileWaves, 0, stream>>>(a);     \
    else                                                                                       \
        expert_kernel<OP, GATED, 256><<<grid_for(TILES), 64 * kTileWaves, 0, stream>>>(a)

}  // namespace

Parts row_parts(int E, int64_t max_rows, int R, int C, int unit)
{
    Parts g{};
    g.tiles = max_row_tiles(max_rows, E, 64) * ((C + unit - 1) / unit);
    g.parts = parts_of(g.tiles, E, R);
    g.bytes = g.parts > 1 ? g.tiles * g.parts * kPartBytes : 0;
    return g;
}

Parts forward_parts(int act, int E, int64_t max_rows, int K, int N)
{
    const Parts g = row_parts(E, max_rows, K, N, act == MOE_ACT_SWIGLU ? 64 : 128);
    return g.parts > 1 && !few_rows_pay(act, E, max_rows, K, N, g.parts) ? g : Parts{1, g.tiles, 0};
}

Parts dw_parts(int E, int64_t max_rows, int K, int N)
{
    Parts g{};
    const int64_t rows = static_cast<int64_t>(E) * ((N + 63) / 64);
    g.tiles = rows * ((K + 127) / 128);
    g.parts = parts_of(g.tiles, E, max_rows / E);
    g.bytes = g.parts > 1 ? g.parts * (g.tiles * kPartBytes + rows * kPartDbBytes) : 0;
    return g;
}

template <Op OP, bool GATED>
static hipError_t launch_parts(Args &a, const Parts &g, void *workspace, hipStream_t stream)
{
    a.parts = g.parts, a.tiles = static_cast<int>(g.tiles);
    a.part = static_cast<f32x4 *>(workspace);
    a.part_db = reinterpret_cast<float *>(static_cast<char *>(workspace) + g.tiles * g.parts * kPartBytes);
    const int64_t n = g.tiles * g.parts;
    expert_part_kernel<OP, GATED><<<dim3(static_cast<unsigned>(n < 2 * kCus ? n : 2 * kCus)), 64 * kTileWaves, 0, stream>>>(a);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return err;
    expert_join_kernel<OP, GATED><<<dim3(static_cast<unsigned>(g.tiles * 2 * kTileWaves)), kWave, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_expert_matmul(const void *x, const int32_t *offsets, const void *w,
                                const float *bias, int act, const void *residual, int E,
                                int64_t max_rows, int K, int N, void *out, void *preact,
                                void *workspace, hipStream_t stream)
{
    Args a{};
    a.p = static_cast<const uint16_t *>(w);
    a.q = static_cast<const uint16_t *>(x);
    a.offsets = offsets, a.E = E, a.max_rows = static_cast<int>(max_rows), a.R = K, a.C = N;
    a.act = act, a.bias = bias, a.residual = static_cast<const uint16_t *>(residual);
    a.out = out, a.preact = static_cast<uint16_t *>(preact);
    const bool gated = act == MOE_ACT_SWIGLU;
    const Parts parts = forward_parts(act, E, max_rows, K, N);
    const bool shared = workspace && parts.parts > 1;
    if (!shared && few_rows_pay(act, E, max_rows, K, N, 1))
        return launch_expert_few(x, offsets, w, bias, act, residual, E, max_rows, K, N, out, preact, stream);
    if (shared)
        return gated ? launch_parts<kForward, true>(a, parts, workspace, stream)
                     : launch_parts<kForward, false>(a, parts, workspace, stream);
    const TileShape shape = tile_shape(E, max_rows, N, gated ? 64 : 128);
    a.height = shape.rows;
    if (gated) {
        MOE_EXPERT(kForward, true, shape.cols, shape.tiles);
    } else {
        MOE_EXPERT(kForward, false, shape.cols, shape.tiles);
    }
    return hipGetLastError();
}

hipError_t launch_expert_matmul_dx(const void *dy, const int32_t *offsets, const void *w, int act,
                                   const void *z, int E, int64_t max_rows, int K, int N, void *dx,
                                   void *workspace, hipStream_t stream)
{
    Args a{};
    a.p = static_cast<const uint16_t *>(w);
    a.q = static_cast<const uint16_t *>(dy);
    a.offsets = offsets, a.E = E, a.max_rows = static_cast<int>(max_rows), a.R = N, a.C = K;
    a.act = act, a.z = static_cast<const uint16_t *>(z), a.out = dx;
    const Parts parts = row_parts(E, max_rows, N, K, 128);
    if (workspace && parts.parts > 1)
        return launch_parts<kDx, false>(a, parts, workspace, stream);
    const TileShape shape = tile_shape(E, max_rows, K, 128);
    a.height = shape.rows;
    MOE_EXPERT(kDx, false, shape.cols, shape.tiles);
    return hipGetLastError();
}

hipError_t launch_expert_matmul_dw(const void *dy, const void *x, const int32_t *offsets, int E,
                                   int64_t max_rows, int K, int N, int flags, void *dw, float *db,
                                   void *workspace, hipStream_t stream)
{
    Args a{};
    a.p = static_cast<const uint16_t *>(x);
    a.q = static_cast<const uint16_t *>(dy);
    a.offsets = offsets, a.E = E, a.max_rows = static_cast<int>(max_rows), a.C = K, a.rows = N;
    a.out = dw, a.db = db, a.flags = flags;
    const Parts parts = dw_parts(E, max_rows, K, N);
    if (workspace && parts.parts > 1)
        return launch_parts<kDw, false>(a, parts, workspace, stream);
    const int64_t n = static_cast<int64_t>(E) * ((N + 255) / 256) * ((K + 255) / 256);  // cut into up to 4 each
    MOE_EXPERT(kDw, false, 2 * n <= kCus ? 128 : 256, 8 * n);
    return hipGetLastError();
}

}  // namespace moe
