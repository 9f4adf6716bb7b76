// The residual's addition with the root-mean-square norm, and its gradient.
//
//   s = x + r,   y = s R w,   R = (mean(s^2) + eps)^(-1/2)
//   d_x = d_s + R g - s R^3 mean(g s),  g = d_y w;   d_w = sum over rows of d_y s R
//
// A row is read once and held in registers (THREADS threads, VPT 16-byte vectors
// each) between its sums and its results, and the next row's loads are in flight
// meanwhile; above 16384 columns neither the next row nor, in the gradient, this one is
// held.  Sixteen lanes hold the 128 values of a block of codes, a row of the DPP moves.
// The gradient of w stays in registers over all rows of a workgroup; the workgroups'
// sums meet in a second kernel, in a fixed order.  Bound by memory (16384 x 7168, all
// outputs: 191 us, 5.5 TB/s; the gradient 163, 5.8 TB/s), small calls by the launch (1 x 7168:
// 4 us).  Wide rows lack registers: 4096 x 32768 215 us and 268 (4.0 TB/s); above
// that some go to scratch, 27 a lane of the norm's and 233 of the gradient's (2048 x
// 65536: 246 us, 4.9 TB/s, and 632, 1.7 TB/s), and 7 of the gradient's from 8208 to 16384
// columns (4096 x 16384: 117 us and 101, 5.3 TB/s).
#include "fp8_codes.hpp"
#include "launch.hpp"

namespace moe {
namespace {

struct Norm {
    const uint16_t *x, *residual;
    const float *weight;
    float eps;
    int64_t T;
    int H;
    float n, per_n;  // H, 1 / H
    uint16_t *sum, *y;
    uint8_t *codes;
    float *scales;
    bool blocks;  // a scale for each block of 128, else for the row
};

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1)
        v += __shfl_xor(v, o);
    return v;
}

// N sums over the row's threads (THREADS of them, one wave or the workgroup);
// `red` holds 2 * N * 16 floats.  `turn` alternates between its halves, so that one
// barrier a row is enough.
template <int THREADS, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float *red, int turn)
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = wave_sum(v[i]);
    if (THREADS == kWave)
        return;
    float *mine = red + turn * N * 16;
    if (lane_id() == 0)
#pragma unroll
        for (int i = 0; i < N; ++i)
            mine[i * 16 + threadIdx.x / kWave] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < THREADS / kWave; ++w)
            v[i] += mine[i * 16 + w];
    }
}

template <int THREADS>
__device__ __forceinline__ uint32_t row_top(uint32_t v, uint32_t *red, int turn)
{
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1)
        v = umax(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), o)));
    if (THREADS == kWave)
        return v;
    uint32_t *mine = red + turn * 16;
    if (lane_id() == 0)
        mine[threadIdx.x / kWave] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / kWave; ++w)
        v = umax(v, mine[w]);
    return v;
}

// Rows of a workgroup at once, and its threads.
constexpr int rows_of(int threads) { return threads == kWave ? 4 : 1; }
constexpr int group_of(int threads) { return threads == kWave ? 4 * kWave : threads; }

// A row's bytes; a row past the last is empty.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_of(const void *p, int64_t t, int bytes, bool live)
{
    return row_rsrc(const_cast<char *>(static_cast<const char *>(p)) + t * bytes, p && live ? bytes : 0);
}

// VPT vectors of a row from lane l on; STREAM: rows that no cache will keep.
template <int THREADS, int VPT, bool STREAM>
__device__ __forceinline__ void load_row(const __amdgpu_buffer_rsrc_t &r, int l, u32x4 (&v)[VPT])
{
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        v[i] = STREAM ? load_stream16(r, (l + i * THREADS) * 16) : load_cached(r, (l + i * THREADS) * 16);
}
template <bool STREAM, typename V>
__device__ __forceinline__ void store_vector(const __amdgpu_buffer_rsrc_t &r, int offset, V v)
{
    constexpr int policy = STREAM ? kCpolStream : kCpolDefault;
    if constexpr (sizeof(V) == 16)
        __builtin_amdgcn_raw_buffer_store_b128(v, r, offset, 0, policy);
    else
        __builtin_amdgcn_raw_buffer_store_b64(v, r, offset, 0, policy);
}

// A row's sums are taken of c s, c = 1 at first; where the mean of squares leaves fp32,
// or is so small (2^-60) that squares do, once more with another power of two: R = c
// (mean((c s)^2) + c^2 eps)^(-1/2).  The squares of c s are then 2^-106 .. 2^96 for all
// values that bf16 has, 2^-133 .. 2^128, and a row's sum is below 2^117.
constexpr float kUp = 0x1p80f, kDown = 0x1p-80f;
constexpr uint32_t kLeastSquares = (127 - 60) << 23, kInfinity = 0x7f800000u;  // of fp32, as bits
__device__ __forceinline__ bool in_range(uint32_t squares) { return squares - kLeastSquares < kInfinity - kLeastSquares; }

constexpr int kNowhere = static_cast<int>(0x80000000u);  // an offset past every row

// A value that all of a row's threads have, for branches that they take together.
__device__ __forceinline__ uint32_t uniform_bits(float v) { return uniform(__float_as_uint(v)); }

// This lane's weights (1 where there are none).
template <int THREADS, int VPT>
__device__ __forceinline__ void load_weights(const float *weight, int H, int l, float (&w)[VPT][8])
{
    const __amdgpu_buffer_rsrc_t r = row_of(weight, 0, H * 4, true);
#pragma unroll
    for (int i = 0; i < 2 * VPT; ++i) {
        const u32x4 v = load_cached(r, (l + i / 2 * THREADS) * 32 + i % 2 * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[i / 2][i % 2 * 4 + j] = weight ? __uint_as_float(v[j]) : 1.0f;
    }
}

template <int THREADS, int VPT, bool STREAM>
__global__ __launch_bounds__(group_of(THREADS)) void add_norm_kernel(Norm a)
{
    constexpr int kRows = rows_of(THREADS);
    __shared__ float red[2 * 16];
    __shared__ uint32_t tops[2 * 16];
    const int l = THREADS == kWave ? lane_id() : static_cast<int>(threadIdx.x);
    const int first = THREADS == kWave ? static_cast<int>(uniform(threadIdx.x / kWave)) : 0;
    constexpr bool kHold = THREADS < 1024;  // the weights, beside the row and the next one
    const int nb = code_blocks(a.H);
    float w[kHold ? VPT : 1][8];
    u32x4 v[VPT], u[VPT];
    auto load = [&](int64_t t) {
        load_row<THREADS, VPT, STREAM>(row_of(a.x, t, a.H * 2, t < a.T), l, v);
        if (a.residual)
            load_row<THREADS, VPT, STREAM>(row_of(a.residual, t, a.H * 2, t < a.T), l, u);
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    if (kHold) {
        load(static_cast<int64_t>(blockIdx.x) * kRows + first);
        load_weights<THREADS, kHold ? VPT : 1>(a.weight, a.H, l, w);
    }
    int turn = 0;
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows; t0 < a.T; t0 += step) {
        const int64_t t = t0 + first;
        const bool live = t < a.T;
        if (!kHold)
            load(t);
        float s[VPT][8], c = 1.0f, ss[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            unpack8(v[i], s[i]);
            if (a.residual) {
                float f[8];
                unpack8(u[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    s[i][j] += f[j];
            }
            if (kHold)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    ss[0] = fmaf(s[i][j], s[i][j], ss[0]);
        }
        if (kHold)
            load(t + step);
        if (a.sum) {
            const __amdgpu_buffer_rsrc_t to = row_of(a.sum, t, a.H * 2, live);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                store_vector<STREAM>(to, (l + i * THREADS) * 16, pack8(s[i]));
        }
        for (bool sum = !kHold;; sum = true) {
            if (sum) {
                ss[0] = 0.0f;
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float f = s[i][j] * c;
                        ss[0] = fmaf(f, f, ss[0]);
                    }
            }
            row_sums<THREADS, 1>(ss, red, turn);
            const uint32_t squares = uniform_bits(fmaf(ss[0], a.per_n, a.eps));
            if (__builtin_expect(in_range(squares), true))
                break;
            if (c != 1.0f)
                break;
            c = squares < kLeastSquares ? kUp : kDown;
            turn ^= 1;
        }
        const float r = 1.0f / sqrtf(ss[0] / a.n + a.eps * c * c) * c;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (!kHold)
                load_weights<THREADS, 1>(a.weight, a.H, l + i * THREADS, reinterpret_cast<float(&)[1][8]>(w[0]));
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[i][j] = s[i][j] * r * w[kHold ? i : 0][j];
        }
        if (a.y) {
            const __amdgpu_buffer_rsrc_t to = row_of(a.y, t, a.H * 2, live);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                store_vector<STREAM>(to, (l + i * THREADS) * 16, pack8(s[i]));
        }
        if (a.codes) {
            const __amdgpu_buffer_rsrc_t to = row_of(a.codes, t, a.H, live);
            uint32_t top[VPT], all = 0;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                top[i] = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j)  // (past the row w has zeros, but an infinite r would make them NaN)
                    top[i] = umax(top[i], (l + i * THREADS) * 8 < a.H ? size_bits(s[i][j]) : 0u);
                all = umax(all, top[i]);
            }
            if (!a.blocks) {
                all = row_top<THREADS>(all, tops, turn);
                if (l == 0 && live)
                    a.scales[t] = scale_of(all);
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = l + i * THREADS;
                if (c / 16 >= nb)  // (zeros; the Coder would take them for scales to divide by)
                    continue;
                const float scale = scale_of(a.blocks ? row_umax(top[i]) : all);
                if (a.blocks && c % 16 == 0 && c * 8 < a.H && live)
                    a.scales[t * nb + c / 16] = scale;
                store_vector<STREAM>(to, c * 8, Coder(scale).codes8(s[i]));
            }
        }
        turn ^= 1;
    }
}

struct NormGrad {
    const uint16_t *dy, *dsum, *sum;
    const float *weight;
    float eps;
    int64_t T;
    int H;
    float n, per_n;  // H, 1 / H
    uint16_t *dx;
    float *part;  // [workgroups][H], or null
};

// HOLD: a row stays in registers between its sums and its results, beside the
// weights and the next row; else it is read again (from cache: 128 KiB of each array at
// the longest).
template <int THREADS, int VPT, bool STREAM>
__global__ __launch_bounds__(group_of(THREADS)) void add_norm_grad_kernel(NormGrad a)
{
    constexpr bool HOLD = THREADS < 1024;
    constexpr int kRows = rows_of(THREADS), kHeld = HOLD ? VPT : 1;
    __shared__ float red[2 * 2 * 16];
    const int l = THREADS == kWave ? lane_id() : static_cast<int>(threadIdx.x);
    const int first = THREADS == kWave ? static_cast<int>(uniform(threadIdx.x / kWave)) : 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    auto rows_at = [&](const uint16_t *p, int64_t t) { return row_of(p, t, a.H * 2, t < a.T); };
    float held[kHeld][8], dw[VPT][8] = {};
    u32x4 sv[kHeld], yv[kHeld], dv[kHeld], sn[kHeld], yn[kHeld], dn[kHeld];
    auto load_next = [&](int64_t t) {
        load_row<THREADS, kHeld, STREAM>(rows_at(a.sum, t), l, sn);
        load_row<THREADS, kHeld, STREAM>(rows_at(a.dy, t), l, yn);
        // (of a null array no memory is read; behind a branch a lone vector is waited for at
        // once, 131072 x 512: 109 us instead of 95, but 16384 x 7168: 163 instead of 167)
        if (VPT == 1 || a.dsum)
            load_row<THREADS, kHeld, STREAM>(rows_at(a.dsum, t), l, dn);
    };
    if (HOLD) {
        load_next(static_cast<int64_t>(blockIdx.x) * kRows + first);
        load_weights<THREADS, kHeld>(a.weight, a.H, l, held);
    }
    // vector i of an array of the row, and of the weights
    auto vector = [&](const u32x4 (&kept)[kHeld], const __amdgpu_buffer_rsrc_t &r, int i) {
        return HOLD ? kept[HOLD ? i : 0] : load_cached(r, (l + i * THREADS) * 16);
    };
    auto weights = [&](int i, float(&w)[8]) {
        if constexpr (HOLD) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j] = held[i][j];
        } else {
            load_weights<THREADS, 1>(a.weight, a.H, l + i * THREADS, reinterpret_cast<float(&)[1][8]>(w));
        }
    };
    // the sums of (c s)^2 and of g c s
    auto sum_up = [&](const u32x4 &sv, const u32x4 &yv, const float(&w)[8], float c, float(&sums)[2]) {
        float s[8], g[8];
        unpack8(sv, s);
        unpack8(yv, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[j] *= c;
            sums[0] = fmaf(s[j], s[j], sums[0]);
            sums[1] = fmaf(g[j] * w[j], s[j], sums[1]);
        }
    };
    // d_x, `back` of s R off it, and d_w's share if the row has one
    auto gradient = [&](const u32x4 &sv, const u32x4 &yv, const u32x4 &dv, const float(&w)[8], float r, float back, bool add,
                        float(&sum)[8]) {
        float s[8], g[8], d[8];
        unpack8(sv, s);
        unpack8(yv, g);
        unpack8(dv, d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = s[j] * r;
            sum[j] = add ? fmaf(g[j], x, sum[j]) : sum[j];  // (of a missing row r may be infinite)
            const float v = fmaf(g[j] * w[j], r, -x * back);
            d[j] = a.dsum ? d[j] + v : v;
        }
        return pack8(d);
    };
    int turn = 0;
    for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows; t0 < a.T; t0 += step) {
        const int64_t t = t0 + first;
        const bool live = t < a.T;
        const __amdgpu_buffer_rsrc_t sr = rows_at(a.sum, t), yr = rows_at(a.dy, t), dr = rows_at(a.dsum, t);
        if (HOLD) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                sv[i] = sn[i], yv[i] = yn[i], dv[i] = dn[i];
            load_next(t + step);
        }
        float sums[2] = {0.0f, 0.0f};  // of s^2 and of g s
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float w[8];
            weights(i, w);
            sum_up(vector(sv, sr, i), vector(yv, yr, i), w, 1.0f, sums);
            if (!HOLD)
                __builtin_amdgcn_sched_barrier(0);  // (all vectors at once would not fit)
        }
        row_sums<THREADS, 2>(sums, red, turn);
        turn ^= 1;
        const uint32_t squares = __float_as_uint(fmaf(sums[0], a.per_n, a.eps));
        const bool good = in_range(squares) & (__float_as_uint(fabsf(sums[1])) < kInfinity);
        const float r = 1.0f / sqrtf(sums[0] / a.n + a.eps);
        const __amdgpu_buffer_rsrc_t to = rows_at(a.dx, t);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float w[8];
            weights(i, w);
            const u32x4 d = a.dsum ? vector(dv, dr, i) : u32x4{};
            const u32x4 dx = gradient(vector(sv, sr, i), vector(yv, yr, i), d, w, r, r * (r * (sums[1] / a.n)), live && good, dw[i]);
            store_vector<STREAM>(to, good ? (l + i * THREADS) * 16 : kNowhere, dx);
            if (!HOLD)
                __builtin_amdgcn_sched_barrier(0);
        }
        if (__builtin_expect(uniform(!good), false)) {
            // Nothing of the row is stored or counted yet.  (A branch in front of the results
            // would hold back their loads: 4096 x 32768 281 us instead of 268.)  Where g s alone
            // is too large, a power of two brings s to some 2^-20.
            const float c = squares < kLeastSquares ? kUp
                            : squares < kInfinity   ? __uint_as_float(__float_as_uint(r * 0x1p-20f) & kInfinity)
                                                    : kDown;
            sums[0] = sums[1] = 0.0f;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float w[8];
                load_weights<THREADS, 1>(a.weight, a.H, l + i * THREADS, reinterpret_cast<float(&)[1][8]>(w));
                const int at = (l + i * THREADS) * 16;
                sum_up(load_cached(sr, at), load_cached(yr, at), w, c, sums);
                __builtin_amdgcn_sched_barrier(0);
            }
            row_sums<THREADS, 2>(sums, red, turn);
            turn ^= 1;
            const float rc = 1.0f / sqrtf(sums[0] / a.n + a.eps * c * c);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float w[8];
                load_weights<THREADS, 1>(a.weight, a.H, l + i * THREADS, reinterpret_cast<float(&)[1][8]>(w));
                const int at = (l + i * THREADS) * 16;
                const u32x4 d = a.dsum ? load_cached(dr, at) : u32x4{};
                store_vector<STREAM>(to, at, gradient(load_cached(sr, at), load_cached(yr, at), d, w, rc * c,
                                                      rc * c * (rc * (sums[1] / a.n)), live, dw[i]));
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    if (!a.part)
        return;
    if constexpr (kRows > 1) {  // the waves' sums, wave 0's first, in its registers
        __shared__ float sums[kRows - 1][VPT][8][kWave];
        if (first > 0)
#pragma unroll
            for (int i = 0; i < VPT * 8; ++i)
                sums[first - 1][i / 8][i % 8][l] = dw[i / 8][i % 8];
        __syncthreads();
        if (first > 0)
            return;
#pragma unroll
        for (int w = 0; w < kRows - 1; ++w)
#pragma unroll
            for (int i = 0; i < VPT * 8; ++i)
                dw[i / 8][i % 8] += sums[w][i / 8][i % 8][l];
    }
    const __amdgpu_buffer_rsrc_t to = row_of(a.part, blockIdx.x, a.H * 4, true);
#pragma unroll
    for (int i = 0; i < 2 * VPT; ++i) {
        u32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = __float_as_uint(dw[i / 2][i % 2 * 4 + j]);
        __builtin_amdgcn_raw_buffer_store_b128(v, to, (l + i / 2 * THREADS) * 32 + i % 2 * 16, 0, 0);
    }
}

// d_w from the workgroups' sums: 32 columns a workgroup, its 32 groups of threads
// every 32nd part each.
__global__ __launch_bounds__(1024) void norm_weight_kernel(const float *__restrict__ part, int parts, int H,
                                                           bool accumulate, float *__restrict__ dw)
{
    __shared__ float sums[32][33];
    const int x = threadIdx.x % 32, y = threadIdx.x / 32, c = blockIdx.x * 32 + x;
    float sum = 0.0f;
    if (c < H)
        for (int p = y; p < parts; p += 32)
            sum += part[static_cast<int64_t>(p) * H + c];
    sums[y][x] = sum;
    __syncthreads();
    if (y == 0 && c < H) {
        float all = accumulate ? dw[c] : 0.0f;
        for (int i = 0; i < 32; ++i)
            all += sums[i][x];
        dw[c] = all;
    }
}

// Threads and vectors of a row.
struct NormTiling {
    int threads, vpt;
};
NormTiling norm_tiling(int H)
{
    const int vecs = H / 8;
    NormTiling n{kWave, 1};
    if (vecs > 4 * kWave)
        n.threads = vecs > 4 * 512 ? 1024 : vecs > 4 * 256 ? 512 : 256;
    while (n.threads * n.vpt < vecs)
        n.vpt *= 2;
    return n;
}
int norm_groups(int64_t T, int rows, int most)
{
    const int64_t n = (T + rows - 1) / rows;
    return static_cast<int>(n < most ? n : most);
}
// Workgroups of the gradient's first kernel.
// One a CU, whose next row is on its way while it works on one, is enough, and more
// leave more sums to the second kernel (16384 x 7168: 163 us; 173 with two, 177 with
// four; 4096 x 16384 101, 105 and 117); rows of a wave, four at once, take two (65536 x
// 1024: 96 us; 113 with one, 108 with four; 131072 x 512 95, 135 and 103.  From 1040 to 2048
// columns a wave's registers let one be on a CU at a time: 32768 x 2048 95 us, 90 with
// one).
int grad_groups(int64_t T, const NormTiling &n) { return norm_groups(T, rows_of(n.threads), n.threads == kWave ? 2 * kCus : kCus); }

}  // namespace

size_t norm_grad_workspace_bytes(int64_t T, int H)
{
    const NormTiling n = norm_tiling(H);
    return static_cast<size_t>(grad_groups(T, n)) * H * 4;
}

// Whether a call's arrays, `bytes` a value, are more than the last-level cache
// keeps for whoever reads them next: its rows then pass the caches by (16384 x 7168,
// all outputs: 191 us against 198; its gradient 163 against 182).
static bool streams(int64_t T, int H, int bytes) { return T * H * bytes > kCacheBytes; }

#define MOE_NORM(THREADS, VPT)                                                                          \
    if (n.threads == THREADS && n.vpt == VPT) {                                                         \
        const dim3 grid(norm_groups(T, rows_of(THREADS), THREADS == 1024 ? 2 * kCus : 16 * kCus));       \
        if (stream_rows)                                                                                \
            add_norm_kernel<THREADS, VPT, true><<<grid, group_of(THREADS), 0, stream>>>(a);             \
        else                                                                                            \
            add_norm_kernel<THREADS, VPT, false><<<grid, group_of(THREADS), 0, stream>>>(a);            \
    }

hipError_t launch_add_norm(const void *x, const void *residual, const float *weight, float eps, int64_t T, int H,
                           void *sum, void *y, bool blocks, void *codes, float *scales, hipStream_t stream)
{
    Norm a{};
    a.x = static_cast<const uint16_t *>(x), a.residual = static_cast<const uint16_t *>(residual);
    a.weight = weight, a.eps = eps, a.T = T, a.H = H, a.n = static_cast<float>(H), a.per_n = 1.0f / a.n;
    a.sum = static_cast<uint16_t *>(sum), a.y = static_cast<uint16_t *>(y);
    a.codes = static_cast<uint8_t *>(codes), a.scales = scales, a.blocks = blocks;
    const NormTiling n = norm_tiling(H);
    const bool stream_rows = streams(T, H, 2 + (residual ? 2 : 0) + (sum ? 2 : 0) + (y ? 2 : 0) + (codes ? 1 : 0));
    MOE_NORM(64, 1)
    MOE_NORM(64, 2)
    MOE_NORM(64, 4)
    MOE_NORM(256, 2)
    MOE_NORM(256, 4)
    MOE_NORM(512, 4)
    MOE_NORM(1024, 4)
    MOE_NORM(1024, 8)
    return hipGetLastError();
}

#define MOE_NORM_GRAD(THREADS, VPT)                                                                     \
    if (n.threads == THREADS && n.vpt == VPT) {                                                         \
        if (stream_rows)                                                                                \
            add_norm_grad_kernel<THREADS, VPT, true><<<dim3(groups), group_of(THREADS), 0, stream>>>(a); \
        else                                                                                            \
            add_norm_grad_kernel<THREADS, VPT, false><<<dim3(groups), group_of(THREADS), 0, stream>>>(a); \
    }

hipError_t launch_add_norm_grad(const void *d_y, const void *d_sum, const void *sum, const float *weight, float eps,
                                int64_t T, int H, void *d_x, float *d_weight, bool accumulate, void *workspace,
                                hipStream_t stream)
{
    NormGrad a{};
    a.dy = static_cast<const uint16_t *>(d_y), a.dsum = static_cast<const uint16_t *>(d_sum);
    a.sum = static_cast<const uint16_t *>(sum), a.weight = weight, a.eps = eps, a.T = T, a.H = H, a.n = static_cast<float>(H), a.per_n = 1.0f / a.n;
    a.dx = static_cast<uint16_t *>(d_x), a.part = d_weight ? static_cast<float *>(workspace) : nullptr;
    const NormTiling n = norm_tiling(H);
    const int groups = grad_groups(T, n);
    const bool stream_rows = streams(T, H, d_sum ? 8 : 6);
    if (T > 0) {
        MOE_NORM_GRAD(64, 1)
        MOE_NORM_GRAD(64, 2)
        MOE_NORM_GRAD(64, 4)
        MOE_NORM_GRAD(256, 2)
        MOE_NORM_GRAD(256, 4)
        MOE_NORM_GRAD(512, 4)
        MOE_NORM_GRAD(1024, 4)
        MOE_NORM_GRAD(1024, 8)
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    if (d_weight)
        norm_weight_kernel<<<dim3((H + 31) / 32), 1024, 0, stream>>>(a.part, groups, H, accumulate, d_weight);
    return hipGetLastError();
}

}  // namespace moe
