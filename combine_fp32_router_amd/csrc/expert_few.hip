// The experts' forward product for few rows an expert, as serving single
// tokens has it:  z = x W_e^T + b_e,  y = act(z) + residual.
//
// Every live expert's weights are read once and multiplied with up to 16 MB
// rows, so the reading bounds it.  A workgroup has 16 output columns of one
// tile of rows; its four waves share the reduced length K, each wave every
// fourth 64 of it, and add their sums in LDS, in wave order.  Each wave is on
// its own: its loads go from memory to a ring of three chunks in its part of
// LDS, 16 weight rows by 128 bytes each two loads of eight whole lines, and
// it waits for its oldest ones only; no barrier before the sums.
// One token at 8 of 32 experts, K = 7168, N = 2048 gated (470 MB of weights):
// 78 us, 6.0 TB/s, against 80 us of the tiles of 64 x 128; loads straight into
// the MFMA's operands, each touching 16 lines of which it uses half, took 89 us,
// rings of four and six chunks 80 and 82.
#include "expert_rows.hpp"
#include "launch.hpp"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4, kDepth = 3;
#define MOE_LDS __attribute__((address_space(3)))
constexpr int kOutside = static_cast<int>(0x80000000u);

struct Few {
    const uint16_t *x, *w;
    const int32_t *offsets;
    const float *bias;
    const uint16_t *residual;
    uint16_t *out, *preact;
    int act, E, max_rows, K, N;
};

// One wave's stream: 16 weight rows (GATED: 16 gate and 16 up) and 16 MB rows
// of x, 64 of K a chunk, through a ring of kDepth chunks in its own LDS.  An
// image is 16 rows of 128 bytes, piece c of row i at c ^ (i / 2) % 8.
template <bool GATED, int MB>
struct Stream {
    static constexpr int wide = GATED ? 2 : 1, kImages = wide + MB, kChunkBytes = kImages * 2048;
    static constexpr int kLoads = 2 * kImages, kRingBytes = kDepth * kChunkBytes;
    const char *w[wide], *x;
    int K, pitch, xbytes;
    int off[2], piece[2];  // of this lane's two loads of an image
    f32x4 acc[wide][MB];

    // Chunk at k0 into `chunk`.
    __device__ __forceinline__ void fetch(MOE_LDS char *chunk, int k0) const
    {
        const int left = (K - k0) * 2;  // bytes of a row from k0 on
        const int64_t at = static_cast<int64_t>(k0) * 2;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int o = piece[h] < left ? off[h] : kOutside;
#pragma unroll
            for (int i = 0; i < kImages; ++i) {
                const char *src = (i < wide ? w[i < wide ? i : 0] : x) + at;
                const int bytes = (i < wide ? 16 * pitch : xbytes) - k0 * 2;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    row_rsrc(const_cast<char *>(src), left > 0 ? max(bytes, 0) : 0),
                    (MOE_LDS void *)(chunk + i * 2048 + h * 1024), 16,
                    o + (i < wide ? 0 : (i - wide) * 16 * pitch), 0, 0, 0);
            }
        }
    }
    // Multiplies the chunk at `rd` (this wave's oldest loads) and refills the
    // chunk before it, once the last step's reads of that are done.
    __device__ __forceinline__ void step(const MOE_LDS char *__restrict__ rd, MOE_LDS char *__restrict__ wr, int k0)
    {
        asm volatile("" ::: "memory");
        constexpr int left = (kDepth - 2) * kLoads;  // younger loads
        __builtin_amdgcn_s_waitcnt(0x0070 | (left & 15) | (left >> 4) << 14);
        asm volatile("" ::: "memory");
        const int lane = lane_id();
        bf16x8 f[kImages][2];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < kImages; ++i)
                f[i][s] = *reinterpret_cast<const MOE_LDS bf16x8 *>(
                    rd + i * 2048 + lane % 16 * 128 + ((4 * s + lane / 16) ^ (lane % 16 / 2)) * 16);
        fetch(wr, k0);
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int g = 0; g < wide; ++g)
                    acc[g][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f[g][s], f[wide + m][s], acc[g][m], 0, 0, 0);
    }
};

template <bool GATED, int MB>
__global__ __launch_bounds__(64 * kWaves) void few_rows_kernel(Few a)
{
    typedef Stream<GATED, MB> S;
    constexpr int wide = S::wide;
    static_assert(S::kRingBytes >= wide * MB * kWave * 16, "the sums fit the ring");
    __shared__ __align__(1024) char rings[kWaves][S::kRingBytes];
    const int groups = a.N / 16, lane = lane_id(), w = static_cast<int>(uniform(threadIdx.x / kWave));
    const RowTile t = find_row_tile(a.offsets, a.E, a.max_rows, 16 * MB, blockIdx.x / groups);
    if (t.n <= 0)
        return;
    const int c0 = blockIdx.x % groups * 16;
    S s;
    s.K = a.K;
    s.pitch = 2 * a.K;
    s.xbytes = t.n * s.pitch;
    const uint16_t *we = a.w + (static_cast<int64_t>(t.e) * wide * a.N + c0) * a.K;
#pragma unroll
    for (int g = 0; g < wide; ++g)
        s.w[g] = reinterpret_cast<const char *>(we + static_cast<int64_t>(g) * a.N * a.K);
    s.x = reinterpret_cast<const char *>(a.x + static_cast<int64_t>(t.first) * a.K);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = h * 8 + lane / 8;
        s.piece[h] = ((lane % 8) ^ (row / 2)) * 16;
        s.off[h] = row * s.pitch + s.piece[h];
    }
#pragma unroll
    for (int g = 0; g < wide; ++g)
#pragma unroll
        for (int m = 0; m < MB; ++m)
            s.acc[g][m] = f32x4{};
    MOE_LDS char *ring = (MOE_LDS char *)rings[w];
    constexpr int kStride = 64 * kWaves;
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i)
        s.fetch(ring + i * S::kChunkBytes, w * 64 + i * kStride);
    int rd = 0, wr = (kDepth - 1) * S::kChunkBytes;
#pragma unroll 1
    for (int k0 = w * 64; k0 < a.K; k0 += kStride) {
        s.step(ring + rd, ring + wr, k0 + (kDepth - 1) * kStride);
        wr = rd;
        rd = rd + S::kChunkBytes == S::kRingBytes ? 0 : rd + S::kChunkBytes;
    }
    // the sums take the rings' place
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070);  // no load is still to land there
    asm volatile("" ::: "memory");
    auto part = [&](int wave, int g, int m) {
        return reinterpret_cast<f32x4 *>(rings[wave]) + (g * MB + m) * kWave + lane;
    };
#pragma unroll
    for (int g = 0; g < wide; ++g)
#pragma unroll
        for (int m = 0; m < MB; ++m)
            *part(w, g, m) = s.acc[g][m];
    __syncthreads();
    // wave m finishes rows 16 m .. + 15: four columns of one row a lane
    for (int m = w; m < MB; m += kWaves) {
        f32x4 v[wide];
#pragma unroll
        for (int g = 0; g < wide; ++g) {
            v[g] = *part(0, g, m);
#pragma unroll
            for (int i = 1; i < kWaves; ++i)
                v[g] += *part(i, g, m);
        }
        const int in_tile = m * 16 + lane % 16, c = c0 + lane / 16 * 4;
        if (in_tile >= t.n)
            continue;
        const int64_t r = t.first + in_tile;
        auto store4 = [](uint16_t *p, f32x4 f) {
            *reinterpret_cast<u32x2 *>(p) = u32x2{pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w)};
        };
#pragma unroll
        for (int g = 0; g < wide; ++g) {
            if (a.bias)
                v[g] += *reinterpret_cast<const f32x4 *>(a.bias + (static_cast<int64_t>(t.e) * wide + g) * a.N + c);
            if (a.preact)
                store4(a.preact + (r * wide + g) * a.N + c, v[g]);
        }
        f32x4 y[1] = {v[0]};
        if (GATED) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[0][j] = v[0][j] * sigmoid(v[0][j]) * v[wide - 1][j];
        } else {
            apply_act(y, a.act);
        }
        if (a.residual) {
            const u32x2 s = *reinterpret_cast<const u32x2 *>(a.residual + r * a.N + c);
            y[0] += f32x4{bf16_lo(s.x), bf16_hi(s.x), bf16_lo(s.y), bf16_hi(s.y)};
        }
        store4(a.out + r * a.N + c, y[0]);
    }
}

}  // namespace

// Rows of a tile: enough for the average run.
static int few_height(int E, int64_t max_rows)
{
    const int64_t live = max_rows < E ? max_rows : E;
    return max_rows <= 16 * live ? 16 : max_rows <= 32 * live ? 32 : 64;
}

// Estimates in us.  Here: the weights from memory at 6.2 TB/s, the rows once
// for every 16 columns at 17 TB/s, or 6.2 where they are more than the L2s hold,
// 2, and 0.8 for each round of the workgroups that fit the card.  The tiles: 8
// for each round of them and 0.75 for 64 of K (in parts: 12, and 0.45 for 64 of
// a part's), or the weights and 5 if that is longer.  They are rough: 64 rows of
// 1 expert, K = N = 4096, go in parts where a workspace allows it, 19, though 11
// are enough here.  Measured (here / tiles): 1 token of 8 experts above 78 / 80; 64
// rows of 1 expert, K = N = 4096 11 / 30; 256 rows of it 37 / 28; 128 rows of each of
// 8, K = 2048, N = 768 gated 27 / 23; 64 rows of each of 8, K = 7168, N = 2048
// gated 126 / 113; 2 rows of each of 64, K = 1024, N = 4096 108 / 95; 1 row of each
// of 8, K = 2048, N = 7168 52 / 37; 4 of each of 32, K = 2048, N = 1024 32 / 24.
bool few_rows_pay(int act, int E, int64_t max_rows, int K, int N, int parts)
{
    const int wide = act == MOE_ACT_SWIGLU ? 2 : 1;
    const int64_t live = max_rows < E ? max_rows : E;
    const int height = few_height(E, max_rows);
    const int64_t groups = max_row_tiles(max_rows, E, height) * (N / 16);
    if (!grid_fits(groups, 64 * kWaves))
        return false;
    const int fit = kCus * (163840 / (kWaves * kDepth * 2048 * (wide + height / 16)));  // by their LDS
    const double weights = 2.0 * live * wide * N * K / 6.2e6, rows = 2.0 * max_rows * K;
    const double here = weights + (N / 16) * rows / (rows > 32e6 ? 6.2e6 : 17e6) + 2 + 0.8 * ((groups + fit - 1) / fit);
    const TileShape shape = tile_shape(E, max_rows, N, 128 / wide);
    const double there = parts > 1 ? 12 + K / 64 * 0.45 / parts
                                   : ((shape.tiles + kCus - 1) / kCus) * (8 + K / 64 * 0.0075 * shape.percent);
    return here < (there > weights + 5 ? there : weights + 5);
}

hipError_t launch_expert_few(const void *x, const int32_t *offsets, const void *w, const float *bias, int act,
                             const void *residual, int E, int64_t max_rows, int K, int N, void *out, void *preact,
                             hipStream_t stream)
{
    Few a{};
    a.x = static_cast<const uint16_t *>(x), a.w = static_cast<const uint16_t *>(w), a.offsets = offsets;
    a.bias = bias, a.residual = static_cast<const uint16_t *>(residual), a.out = static_cast<uint16_t *>(out);
    a.preact = static_cast<uint16_t *>(preact), a.act = act, a.E = E, a.max_rows = static_cast<int>(max_rows);
    a.K = K, a.N = N;
    const int height = few_height(E, max_rows);
    const dim3 grid(static_cast<unsigned>(max_row_tiles(max_rows, E, height) * (N / 16)));
#define MOE_FEW(MB)                                                                            \
    if (act == MOE_ACT_SWIGLU)                                                                 \
        few_rows_kernel<true, MB><<<grid, 64 * kWaves, 0, stream>>>(a);                        \
    else                                                                                       \
        few_rows_kernel<false, MB><<<grid, 64 * kWaves, 0, stream>>>(a)
    if (height == 16) {
        MOE_FEW(1);
    } else if (height == 32) {
        MOE_FEW(2);
    } else {
        MOE_FEW(4);
    }
#undef MOE_FEW
    return hipGetLastError();
}

}  // namespace moe
