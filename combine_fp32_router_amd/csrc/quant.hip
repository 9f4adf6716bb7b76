// E4M3 codes and scales of bf16 rows (a scale for each 128 values of a row) and
// of weights (one for each 128 x 128, the transposed codes beside them), as the
// 8-bit products take them.  Both read every value once and are bound by memory:
// 4099 x 7168 rows 17.2 us, 5.2 TB/s; 8 x 4096 x 7168 weights with the transposed codes
// 174 us, 5.4 TB/s.
#include "expert_rows.hpp"
#include "fp8_codes.hpp"
#include "launch.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256, kAtOnce = 4;  // vectors of a thread at a time

struct QuantRows {
    const uint16_t *x;       // or
    const float *wide;       // in fp32
    const int32_t *offsets;  // or null: all rows
    int E, max_rows, n;      // values of a segment (a row, or a half of one)
    int halves, lanes;       // threads of a segment: 16 times a power of two
    uint8_t *codes;
    float *scales;
};

template <bool STREAM, typename V>
__device__ __forceinline__ void store(V v, V *p)
{
    if (STREAM)
        __builtin_nontemporal_store(v, p);
    else
        *p = v;
}
template <bool STREAM>
__device__ __forceinline__ u32x4 load(const u32x4 *p)
{
    return STREAM ? __builtin_nontemporal_load(p) : *p;
}

// `lanes` threads take a segment's 16-byte vectors in turn, four each at a time,
// 16 lanes a block.
template <bool STREAM, bool WIDE>
__global__ __launch_bounds__(kThreads) void quant_rows_kernel(QuantRows a)
{
    const int rows = a.offsets ? run_start(a.offsets, a.E, a.max_rows) : a.max_rows;
    const int64_t segments = static_cast<int64_t>(rows) * a.halves;
    const int each = kThreads / a.lanes, l = threadIdx.x & (a.lanes - 1), vecs = a.n / 8, nb = code_blocks(a.n);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * each + threadIdx.x / a.lanes; i < segments;
         i += static_cast<int64_t>(gridDim.x) * each) {
        const u32x4 *x = WIDE ? reinterpret_cast<const u32x4 *>(a.wide + i * a.n) : reinterpret_cast<const u32x4 *>(a.x + i * a.n);
        u32x2 *codes = reinterpret_cast<u32x2 *>(a.codes + i * a.n);
        for (int c0 = l; c0 < nb * 16; c0 += kAtOnce * a.lanes) {
            constexpr int kLoads = WIDE ? 2 : 1;  // of eight values
            u32x4 v[kAtOnce][kLoads];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int c = c0 + k * a.lanes;
#pragma unroll
                for (int h = 0; h < kLoads; ++h)
                    v[k][h] = c < vecs ? load<STREAM>(x + c * kLoads + h) : u32x4{};
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int c = c0 + k * a.lanes;
                if (c >= nb * 16)
                    break;
                float f[8];
                if (WIDE) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        f[j] = __uint_as_float(v[k][j / 4 % kLoads][j % 4]);
                } else {
                    unpack8(v[k][0], f);
                }
                uint32_t top = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    top = umax(top, size_bits(f[j]));
                const float scale = scale_of(row_umax(top));
                const u32x2 q = Coder(scale).codes8(f);
                if (c < vecs)
                    store<STREAM>(q, codes + c);
                if (c % 16 == 0 && c < vecs)
                    a.scales[i * nb + c / 16] = scale;
            }
        }
    }
}

struct QuantWeights {
    const uint16_t *w;
    int N, K, halves;
    uint8_t *codes, *codes_t;
    float *scales, *scales_t;
};

// One workgroup for 128 x 128: a thread has 8 x 8 of them, so that its codes turn
// in registers and the transposed tile passes LDS in 8-byte pieces.  (256 x 256 and
// 1024 threads, for longer pieces of rows: 183 us where this takes 175.)
template <bool STREAM>
__global__ __launch_bounds__(kThreads) void quant_weights_kernel(QuantWeights a)
{
    __shared__ uint32_t tops[kThreads / kWave];
    __shared__ __align__(16) uint8_t turned[128][128 + 16];
    const int nbn = code_blocks(a.N), nbk = code_blocks(a.K);
    const int bn = blockIdx.x % nbn, bk = blockIdx.x / nbn % nbk, m = blockIdx.x / nbk / nbn;  // m: e * halves + half
    const int k = bk * 128 + threadIdx.x % 16 * 8, n0 = bn * 128 + threadIdx.x / 16 * 8;
    const int64_t matrix = static_cast<int64_t>(m) * a.N * a.K;
    u32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = n0 + i < a.N && k < a.K
                   ? load<STREAM>(reinterpret_cast<const u32x4 *>(a.w + matrix + static_cast<int64_t>(n0 + i) * a.K + k))
                   : u32x4{};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)  // the sizes of a pair of bf16 values, as fp32 bits
            top = umax(top, umax(v[i][j] << 16 & 0x7fffffffu, v[i][j] & 0x7fff0000u));
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1)
        top = umax(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), o)));
    if (lane_id() == 0)
        tops[threadIdx.x / kWave] = top;
    __syncthreads();
    top = umax(umax(tops[0], tops[1]), umax(tops[2], tops[3]));
    const float scale = scale_of(top);
    const int e = m / a.halves, half = m % a.halves;
    if (threadIdx.x == 0) {
        a.scales[(static_cast<int64_t>(m) * nbn + bn) * nbk + bk] = scale;
        if (a.codes_t)
            a.scales_t[((static_cast<int64_t>(e) * nbk + bk) * a.halves + half) * nbn + bn] = scale;
    }
    const Coder coder(scale);
    u32x2 q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f[8];
        unpack8(v[i], f);
        q[i] = coder.codes8(f);
        if (n0 + i < a.N && k < a.K)
            store<STREAM>(q[i], reinterpret_cast<u32x2 *>(a.codes + matrix + static_cast<int64_t>(n0 + i) * a.K + k));
    }
    if (!a.codes_t)
        return;
    // 4 x 4 bytes at a time: rows 4 r .. + 3, columns 4 c .. + 3
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t p0 = q[4 * r][c], p1 = q[4 * r + 1][c], p2 = q[4 * r + 2][c], p3 = q[4 * r + 3][c];
            const uint32_t lo01 = __builtin_amdgcn_perm(p1, p0, 0x05010400), hi01 = __builtin_amdgcn_perm(p1, p0, 0x07030602);
            const uint32_t lo23 = __builtin_amdgcn_perm(p3, p2, 0x05010400), hi23 = __builtin_amdgcn_perm(p3, p2, 0x07030602);
            const uint32_t t[4] = {__builtin_amdgcn_perm(lo23, lo01, 0x05040100), __builtin_amdgcn_perm(lo23, lo01, 0x07060302),
                                   __builtin_amdgcn_perm(hi23, hi01, 0x05040100), __builtin_amdgcn_perm(hi23, hi01, 0x07060302)};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint32_t *>(&turned[threadIdx.x % 16 * 8 + 4 * c + j][threadIdx.x / 16 * 8 + 4 * r]) = t[j];
        }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = threadIdx.x / 8 + 32 * i, kk = bk * 128 + row, n = bn * 128 + threadIdx.x % 8 * 16;
        if (kk < a.K && n < a.N)  // N is a multiple of 16
            store<STREAM>(*reinterpret_cast<const u32x4 *>(&turned[row][threadIdx.x % 8 * 16]),
                          reinterpret_cast<u32x4 *>(a.codes_t + ((static_cast<int64_t>(e) * a.K + kk) * a.halves + half) * a.N + n));
    }
}

}  // namespace

static hipError_t launch_rows(const void *x, const float *wide, const int32_t *offsets, int E, int64_t max_rows, int n,
                              int halves, void *codes, float *scales, hipStream_t stream)
{
    QuantRows a{};
    a.x = static_cast<const uint16_t *>(x), a.wide = wide, a.offsets = offsets, a.E = E, a.max_rows = static_cast<int>(max_rows);
    a.n = n, a.halves = halves, a.codes = static_cast<uint8_t *>(codes), a.scales = scales;
    a.lanes = 16;
    while (a.lanes < kThreads && kAtOnce * a.lanes < code_blocks(n) * 16)
        a.lanes *= 2;
    const int64_t groups = (max_rows * halves + kThreads / a.lanes - 1) / (kThreads / a.lanes);
    const dim3 grid(static_cast<unsigned>(groups < 16 * kCus ? groups : 16 * kCus));
    if (wide)
        quant_rows_kernel<false, true><<<grid, kThreads, 0, stream>>>(a);
    else if (max_rows * halves * n * 3 > kCacheBytes)
        quant_rows_kernel<true, false><<<grid, kThreads, 0, stream>>>(a);
    else
        quant_rows_kernel<false, false><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_quant_rows(const void *x, const int32_t *offsets, int E, int64_t max_rows, int n, int halves,
                             void *codes, float *scales, hipStream_t stream)
{
    return launch_rows(x, nullptr, offsets, E, max_rows, n, halves, codes, scales, stream);
}

hipError_t launch_quant_wide_rows(const float *x, const int32_t *offsets, int E, int64_t max_rows, int n, int halves,
                                  void *codes, float *scales, hipStream_t stream)
{
    return launch_rows(nullptr, x, offsets, E, max_rows, n, halves, codes, scales, stream);
}

int64_t quant_weights_groups(int E, int N, int K, int halves)
{
    return static_cast<int64_t>(E) * halves * code_blocks(N) * code_blocks(K);
}

hipError_t launch_quant_weights(const void *w, int E, int N, int K, int halves, void *codes, float *scales,
                                void *codes_t, float *scales_t, hipStream_t stream)
{
    QuantWeights a{};
    a.w = static_cast<const uint16_t *>(w), a.N = N, a.K = K, a.halves = halves;
    a.codes = static_cast<uint8_t *>(codes), a.scales = scales;
    a.codes_t = static_cast<uint8_t *>(codes_t), a.scales_t = scales_t;
    const dim3 grid(static_cast<unsigned>(quant_weights_groups(E, N, K, halves)));
    if (static_cast<int64_t>(E) * halves * N * K * (codes_t ? 4 : 3) > kCacheBytes)
        quant_weights_kernel<true><<<grid, kThreads, 0, stream>>>(a);
    else
        quant_weights_kernel<false><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace moe
