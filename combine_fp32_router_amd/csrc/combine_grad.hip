// Gradient of the combine: out[t] = sum_j w_tj * deq(row[pos_tj]) gives, for
// the gradient d of out[t],
//   d_row[pos_tj, h] = bf16_rne(w_tj * d_h)
//   d_w_tj           = sum_h d_h * deq(row[pos_tj])_h    (0 for a dropped slot)
// A quantised row's scale is taken out of the sum: sum_h d_h * code_h, times
// the scale once.
//
// gfx950 design.  One block per token; each thread holds VPT 16-byte vectors
// of d in registers as fp32, so d is read once for all k slots.  Per slot a
// thread reads its part of the row, adds its products to one fp32 partial
// and writes its part of w * d.  The partials of a group of slots reduce over
// the wave, then over the block through LDS in wave order: the same bits
// every time.
//
// HBM-bound: bf16 writes a row for every row it reads.  8192 tokens of 7168,
// 8 slots: gates alone (read) 149 us, 7.1 TB/s; rows alone (write) 183, 5.8;
// both in one kernel 376, since reads and writes then take turns in HBM
// throughout, and in two launches, first all reads, 332.  With rows of one
// byte or less that saves nothing (int8: 286 against 289; E4M3 285, int4 239).
// Few rows are written with ordinary stores and in one launch, many with
// streaming stores, which do not push other data out of the last-level cache
// (in turn over four sets of buffers, ordinary / streaming: 67 MB of rows
// 28.0 / 28.4 us, 34 MB 21.8 / 23.2, 134 MB int8 46.5 / 43.4, 117 MB 53.6 / 46.4,
// 235 MB 104 / 88; over one set, which the cache holds, ordinary ones take 36
// instead of 43 for the 134).
#include "common.hpp"
#include "launch.hpp"

namespace moe {
namespace {

constexpr int kSlotGroup = 4;  // slots whose row loads are in flight together
constexpr int kNarrowTokens = 4;  // of a block, short rows
constexpr int64_t kManyBytes = 100 << 20;  // of written rows: streaming stores

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1)
        v += __shfl_xor(v, o);
    return v;
}

// Eight elements of a row as fp32, without the scale.
template <int Q>
struct RowVec;
template <>
struct RowVec<0> {  // bf16
    typedef u32x4 vec;
    static __device__ __forceinline__ void get(vec v, float *f) { unpack8(v, f); }
};
template <>
struct RowVec<1> {  // int8
    typedef u32x2 vec;
    static __device__ __forceinline__ void get(vec v, float *f) { dequant8(v, 1.0f, f); }
};
template <>
struct RowVec<2> {  // int4
    typedef uint32_t vec;
    static __device__ __forceinline__ void get(vec v, float *f) { dequant4x8(v, 1.0f, f); }
};
template <>
struct RowVec<3> {  // E4M3
    typedef u32x2 vec;
    static __device__ __forceinline__ void get(vec v, float *f) { dequant_fp8x8(v, 1.0f, f); }
};

// ROWS: write d_row, with streaming stores if STREAM; GATES: read the rows and
// write d_w.
template <int Q, int VPT, bool ROWS, bool GATES, bool STREAM>
__global__ __launch_bounds__(1024) void combine_grad_kernel(
    const u32x4 *__restrict__ d_out, const void *__restrict__ rows_,
    const float *__restrict__ scales, const int32_t *__restrict__ pos,
    const float *__restrict__ w, int G, int k, u32x4 *__restrict__ d_rows, float *__restrict__ d_w)
{
    typedef RowVec<Q> RV;
    __shared__ float red[16][MOE_MAX_TOPK];  // [wave][slot]
    const typename RV::vec *rows = static_cast<const typename RV::vec *>(rows_);
    const int64_t t = blockIdx.x;
    const int nthr = blockDim.x, wv = threadIdx.x / kWave;
    const int32_t at = load_per_lane(pos + t * k, k);
    const float wts = load_per_lane(w + t * k, k);
    float d[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int g = threadIdx.x + i * nthr;
        unpack8(g < G ? d_out[t * G + g] : u32x4{0, 0, 0, 0}, d[i]);
    }
    for (int j0 = 0; j0 < k; j0 += kSlotGroup) {
        typename RV::vec v[kSlotGroup][VPT];
        if (GATES) {
#pragma unroll
            for (int q = 0; q < kSlotGroup; ++q) {
                const int32_t p = j0 + q < k ? lane_value(at, j0 + q) : -1;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int g = threadIdx.x + i * nthr;
                    v[q][i] = typename RV::vec{};
                    if (p >= 0 && g < G)
                        v[q][i] = __builtin_nontemporal_load(rows + static_cast<int64_t>(p) * G + g);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < kSlotGroup; ++q) {
            const int j = j0 + q;
            if (j >= k)
                break;
            const int32_t p = lane_value(at, j);
            if (ROWS && p >= 0) {
                const float wj = lane_value(wts, j);
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int g = threadIdx.x + i * nthr;
                    float f[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        f[c] = wj * d[i][c];
                    u32x4 *at_row = d_rows + static_cast<int64_t>(p) * G + g;
                    if (g < G && STREAM)
                        __builtin_nontemporal_store(pack8(f), at_row);
                    else if (g < G)
                        *at_row = pack8(f);
                }
            }
            if (GATES) {
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    float f[8];
                    RV::get(v[q][i], f);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        dot = fmaf(d[i][c], f[c], dot);
                }
                dot = wave_sum(dot);
                if (lane_id() == 0)
                    red[wv][j] = dot;
            }
        }
    }
    if (GATES) {
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < k) {
            const int32_t p = pos[t * k + threadIdx.x];
            float sum = 0.0f;
            for (int i = 0; i < nthr / kWave; ++i)
                sum += red[i][threadIdx.x];
            if (Q != 0 && p >= 0)
                sum *= scales[p];
            d_w[t * k + threadIdx.x] = p >= 0 ? sum : 0.0f;
        }
    }
}

// Short rows, of at most LG <= 16 groups of eight elements: a wave has one
// token, and each LG of its lanes a slot.  16 slots of 32 elements int8, 26560
// tokens: 26 us, 50 with a block a token; 8 of 64 bf16, 16000 tokens: 10 and 19; 8
// of 128 int4, 30000: 28 and 35; their bytes alone 7, 5.5 and 13.  (LG = 32, 8 of
// 256 int8, 30000: 60 and 45.)
template <int Q, int LG, bool ROWS, bool GATES>
__global__ __launch_bounds__(kNarrowTokens *kWave) void combine_grad_narrow_kernel(
    const u32x4 *__restrict__ d_out, const void *__restrict__ rows_,
    const float *__restrict__ scales, const int32_t *__restrict__ pos,
    const float *__restrict__ w, int64_t T, int G, int k, bool stream, u32x4 *__restrict__ d_rows,
    float *__restrict__ d_w)
{
    typedef RowVec<Q> RV;
    constexpr int kSlots = kWave / LG;
    const typename RV::vec *rows = static_cast<const typename RV::vec *>(rows_);
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kNarrowTokens + threadIdx.x / kWave;
    if (t >= T)
        return;
    const int g = lane_id() % LG, sub = lane_id() / LG;
    float d[8];
    unpack8(g < G ? d_out[t * G + g] : u32x4{0, 0, 0, 0}, d);
#pragma unroll 4
    for (int j0 = 0; j0 < k; j0 += kSlots) {
        const int j = j0 + sub;
        const int32_t p = j < k ? pos[t * k + j] : -1;
        const bool in = p >= 0 && g < G;
        typename RV::vec v{};
        float scale = 1.0f;
        if (GATES && in) {
            v = __builtin_nontemporal_load(rows + static_cast<int64_t>(p) * G + g);
            if (Q != 0)
                scale = scales[p];
        }
        if (ROWS && in) {
            const float wj = w[t * k + j];
            float f[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
                f[c] = wj * d[c];
            u32x4 *at_row = d_rows + static_cast<int64_t>(p) * G + g;
            if (stream)
                __builtin_nontemporal_store(pack8(f), at_row);
            else
                *at_row = pack8(f);
        }
        if (GATES) {
            float f[8], dot = 0.0f;
            RV::get(v, f);
#pragma unroll
            for (int c = 0; c < 8; ++c)
                dot = fmaf(d[c], f[c], dot);
#pragma unroll
            for (int o = LG / 2; o > 0; o >>= 1)
                dot += __shfl_xor(dot, o);
            if (g == 0 && j < k)
                d_w[t * k + j] = p < 0 ? 0.0f : Q != 0 ? dot * scale : dot;
        }
    }
}

template <int Q>
void launch_format(const void *d_out, const void *rows, const float *scales, const int32_t *pos,
                   const float *w, int64_t T, int H, int k, void *d_rows, float *d_w,
                   hipStream_t stream)
{
    const int G = H / 8;
    const bool large = T * k * H * 2 > kManyBytes;
    if (G <= 16) {
        const dim3 blocks(static_cast<unsigned>((T + kNarrowTokens - 1) / kNarrowTokens));
#define MOE_CG_NARROW(LG, R, W)                                                                \
    combine_grad_narrow_kernel<Q, LG, R, W><<<blocks, kNarrowTokens * kWave, 0, stream>>>(     \
        static_cast<const u32x4 *>(d_out), rows, scales, pos, w, T, G, k, large,               \
        static_cast<u32x4 *>(d_rows), d_w)
#define MOE_CG_NARROW_PARTS(LG)                                                                \
    if (d_rows && d_w) { MOE_CG_NARROW(LG, true, true); }                                      \
    else if (d_rows) { MOE_CG_NARROW(LG, true, false); }                                       \
    else { MOE_CG_NARROW(LG, false, true); }
        if (G <= 2) { MOE_CG_NARROW_PARTS(2) }
        else if (G <= 8) { MOE_CG_NARROW_PARTS(8) }
        else { MOE_CG_NARROW_PARTS(16) }
#undef MOE_CG_NARROW_PARTS
#undef MOE_CG_NARROW
        return;
    }
    const RowTiling rt = row_tiling(G);
    const dim3 grid(static_cast<unsigned>(T)), block(rt.threads);
#define MOE_CG(V, R, W, S)                                                                     \
    combine_grad_kernel<Q, V, R, W, S><<<grid, block, 0, stream>>>(                            \
        static_cast<const u32x4 *>(d_out), rows, scales, pos, w, G, k,                         \
        static_cast<u32x4 *>(d_rows), d_w)
#define MOE_CG_PARTS(V)                                                                        \
    if (d_w && (!d_rows || (Q == 0 && large))) { MOE_CG(V, false, true, false); }              \
    if (!d_rows) { return; }                                                                   \
    if (!large) {                                                                              \
        if (d_w) { MOE_CG(V, true, true, false); } else { MOE_CG(V, true, false, false); }     \
    } else if (Q != 0 && d_w) {                                                                \
        MOE_CG(V, true, true, Q != 0);                                                         \
    } else {                                                                                   \
        MOE_CG(V, true, false, true);                                                          \
    }
    switch (rt.vpt) {
    case 1: MOE_CG_PARTS(1); break;
    case 2: MOE_CG_PARTS(2); break;
    case 4: MOE_CG_PARTS(4); break;
    default: MOE_CG_PARTS(8); break;
    }
#undef MOE_CG_PARTS
#undef MOE_CG
}

}  // namespace

hipError_t launch_combine_grad(const void *d_out, const void *rows, const float *scales, int quant,
                               const int32_t *pos, const float *w, int64_t T, int H, int k,
                               void *d_rows, float *d_w, hipStream_t stream)
{
    switch (quant) {
    case 0: launch_format<0>(d_out, rows, scales, pos, w, T, H, k, d_rows, d_w, stream); break;
    case 1: launch_format<1>(d_out, rows, scales, pos, w, T, H, k, d_rows, d_w, stream); break;
    case 2: launch_format<2>(d_out, rows, scales, pos, w, T, H, k, d_rows, d_w, stream); break;
    default: launch_format<3>(d_out, rows, scales, pos, w, T, H, k, d_rows, d_w, stream); break;
    }
    return hipGetLastError();
}

}  // namespace moe
