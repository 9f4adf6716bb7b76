// Balance loss of the router with per-expert counts, and the router's
// gradient (through the gate weights and through the balance loss).
//
// With p = softmax(logits[t]) over the E experts, c_e the number of a
// segment's slots routed to expert e, S_e = sum_t p_te and n the segment's
// live (unmasked) tokens:
//   loss        = E / (k n^2) * sum_e c_e S_e
//   d loss/d l  = E / (k n^2) * p_te * (c_e - sum_e' c_e' p_te')
// (the counts are constants of the gradient) and, for the gate weights
// w = softmax of the k selected logits,
//   d l_{idx_j} += w_j (dw_j - sum_i w_i dw_i).
//
// gfx950 mapping.  L lanes own one token (a 16-lane DPP row for E <= 256,
// the wave above), each holding NE of its logits in registers, so a row is
// read once and its maximum, sum and products reduce in the VALU.  The
// forward pass keeps each lane's running sum of p over the tokens of its
// block in registers, joins the block's waves through LDS in wave order and
// leaves one row of partial sums and counts per block; a second launch adds
// the rows of a segment in block order (in double), so no result depends on
// the order in which blocks or atomics ran.  A segment that fits one block
// needs no second launch.
//
// HBM-bound from about 10^7 logits on: 131072 tokens of 512 experts take 49 us
// (5.5 TB/s) and 8 for the join, the gradient 92 (5.8 TB/s, half of it
// written); 16384 of 256 in four segments 7.6 + 6.4 and 8.4, latency; 256 of 8
// 4.4 and 3.8.
#include "common.hpp"
#include "launch.hpp"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

template <int CTRL>
__device__ __forceinline__ float dppf(float v)
{
    return __uint_as_float(dpp32<CTRL>(__float_as_uint(v)));
}

template <int L>
__device__ __forceinline__ float group_max(float v)
{
    v = fmaxf(v, dppf<0xB1>(v));
    v = fmaxf(v, dppf<0x4E>(v));
    v = fmaxf(v, dppf<0x141>(v));
    v = fmaxf(v, dppf<0x140>(v));
    if (L == 64) {
        v = fmaxf(v, __shfl_xor(v, 16));
        v = fmaxf(v, __shfl_xor(v, 32));
    }
    return v;
}

template <int L>
__device__ __forceinline__ float group_sum(float v)
{
    v += dppf<0xB1>(v);
    v += dppf<0x4E>(v);
    v += dppf<0x141>(v);
    v += dppf<0x140>(v);
    if (L == 64) {
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
    }
    return v;
}

// Expert held as element q of lane `sub`: runs of four per lane when the row
// is read as 16-byte vectors, else one expert per lane in turn.
template <int L, bool VEC>
__device__ __forceinline__ int expert_of(int q, int sub)
{
    return VEC ? (q / 4) * (4 * L) + 4 * sub + q % 4 : q * L + sub;
}

// A token's logits, -inf past E; all zero for a token that is not live
// (whose memory is not read).
template <int L, int NE, bool VEC, bool LAST = false>
__device__ __forceinline__ void load_row(const float *__restrict__ row, int E, int sub, bool live,
                                         float (&v)[NE])
{
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < NE / 4; ++i) {
            const int e = expert_of<L, VEC>(4 * i, sub);
            f32x4 x{};
            if (live && e < E) {
                const f32x4 *at = reinterpret_cast<const f32x4 *>(row + e);
                x = LAST ? __builtin_nontemporal_load(at) : *at;
            }
            const bool past = e >= E;
            v[4 * i + 0] = past ? -INFINITY : x.x;
            v[4 * i + 1] = past ? -INFINITY : x.y;
            v[4 * i + 2] = past ? -INFINITY : x.z;
            v[4 * i + 3] = past ? -INFINITY : x.w;
        }
    } else {
#pragma unroll
        for (int q = 0; q < NE; ++q) {
            const int e = expert_of<L, VEC>(q, sub);
            v[q] = e >= E ? -INFINITY : (live ? row[e] : 0.0f);
        }
    }
}

// p of the token in place of its logits; 0 everywhere if it is not live.  The
// exponential is the base-2 instruction behind a rounded product: off by about
// (max - z) 2^-23 of the result.
template <int L, int NE>
__device__ __forceinline__ void softmax_row(float (&v)[NE], bool live)
{
    constexpr float kLog2e = 1.44269504088896341f;
    float m = v[0];
#pragma unroll
    for (int q = 1; q < NE; ++q)
        m = fmaxf(m, v[q]);
    m = group_max<L>(m);
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < NE; ++q) {
        v[q] = __builtin_amdgcn_exp2f((v[q] - m) * kLog2e);
        s += v[q];
    }
    s = group_sum<L>(s);
    const float inv = live ? __builtin_amdgcn_rcpf(s) : 0.0f;  // 1 ulp
#pragma unroll
    for (int q = 0; q < NE; ++q)
        v[q] *= inv;
}

struct BalanceOut {
    float *loss;
    int32_t *counts;
    float *prob_sums;
    int32_t *live;
};

// A value that another block stored, and the store, past the XCD's L2.
template <typename V>
__device__ __forceinline__ V load_shared(const V *p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename V>
__device__ __forceinline__ void store_shared(V *p, V v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// loss of one segment from its sums; called by every thread of a block.
// SHARED: they are other blocks'.
template <bool SHARED>
__device__ void write_loss(const float *sums, const int32_t *counts, int live, int E, int k,
                           float *loss)
{
    __shared__ double red[16];
    double acc = 0.0;
    for (int e = threadIdx.x; e < E; e += blockDim.x)
        acc += static_cast<double>(SHARED ? load_shared(counts + e) : counts[e]) *
               static_cast<double>(SHARED ? load_shared(sums + e) : sums[e]);
    for (int o = kWave / 2; o > 0; o >>= 1)
        acc += __shfl_xor(acc, o);
    if (lane_id() == 0)
        red[threadIdx.x / kWave] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
        double total = 0.0;
        for (int w = 0; w < static_cast<int>(blockDim.x) / kWave; ++w)
            total += red[w];
        const double n = static_cast<double>(live);
        *loss = live > 0 ? static_cast<float>(total * E / (n * n * k)) : 0.0f;
    }
}

// One block: tokens [b*tpb, (b+1)*tpb) of segment blockIdx.y.  ONE: the
// block covers its whole segment and writes the results itself.
template <int L, int NE, bool VEC, bool ONE>
__global__ __launch_bounds__(1024) void balance_partial_kernel(
    const float *__restrict__ logits, const int32_t *__restrict__ idx,
    const uint8_t *__restrict__ mask, int64_t T, int64_t seg, int tpb, int E, int k, float *psum,
    int32_t *pcount, int32_t *plive, unsigned *done, BalanceOut out)
{
    extern __shared__ float lds[];  // [waves][E] sums, then [E] counts, then the live count
    const int nw = blockDim.x / kWave, w = threadIdx.x / kWave, lane = lane_id();
    int32_t *hist = reinterpret_cast<int32_t *>(lds + nw * E);
    for (int e = threadIdx.x; e <= E; e += blockDim.x)
        hist[e] = 0;
    __syncthreads();
    const int64_t s = blockIdx.y;
    const int64_t t0 = s * seg + static_cast<int64_t>(blockIdx.x) * tpb;
    const int64_t end = min(T, (s + 1) * seg);
    const int n = static_cast<int>(max(int64_t(0), min(static_cast<int64_t>(tpb), end - t0)));

    // counts of the live tokens' slots
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        if (!mask || mask[t0 + i])
            atomicAdd(&hist[E], 1);
    for (int i = threadIdx.x; i < n * k; i += blockDim.x) {
        const int e = idx[t0 * k + i];
        if (static_cast<unsigned>(e) < static_cast<unsigned>(E) && (!mask || mask[t0 + i / k]))
            atomicAdd(&hist[e], 1);
    }

    constexpr int G = kWave / L;  // tokens of a wave at a time
    const int sub = lane % L;
    float acc[NE];
#pragma unroll
    for (int q = 0; q < NE; ++q)
        acc[q] = 0.0f;
    for (int i = w * G; i < n; i += 2 * nw * G) {
        float v[2][NE];  // two tokens at a time: their loads and their sums run side by side
        bool live[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int in = i + u * nw * G + lane / L;
            const int64_t t = t0 + in;
            live[u] = in < n && (!mask || mask[t]);
            load_row<L, NE, VEC>(logits + t * E, E, sub, live[u], v[u]);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
            softmax_row<L, NE>(v[u], live[u]);
#pragma unroll
        for (int q = 0; q < NE; ++q)
            acc[q] += v[0][q] + v[1][q];
    }
#pragma unroll
    for (int q = 0; q < NE; ++q) {
        if (L == 16) {
            acc[q] += __shfl_xor(acc[q], 16);
            acc[q] += __shfl_xor(acc[q], 32);
        }
        const int e = expert_of<L, VEC>(q, sub);
        if (lane < L && e < E)
            lds[w * E + e] = acc[q];
    }
    __syncthreads();
    const int64_t row = s * gridDim.x + blockIdx.x;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        double sum = 0.0;
        for (int i = 0; i < nw; ++i)
            sum += static_cast<double>(lds[i * E + e]);
        if (ONE) {
            lds[e] = static_cast<float>(sum);  // row 0: this thread alone reads and writes entry e
            out.prob_sums[s * E + e] = static_cast<float>(sum);
            out.counts[s * E + e] = hist[e];
        } else {
            psum[row * E + e] = static_cast<float>(sum);
            pcount[row * E + e] = hist[e];
        }
    }
    if (ONE) {
        __syncthreads();
        write_loss<false>(lds, hist, hist[E], E, k, out.loss + s);
        if (threadIdx.x == 0)
            out.live[s] = hist[E];
    } else if (threadIdx.x == 0) {
        plive[row] = hist[E];
        if (blockIdx.x == 0)
            done[s] = 0;
    }
}

// Adds a segment's partial rows: a group of COLS threads for each of 1024 /
// COLS rows at a time, eight of them in flight, the groups' sums added in
// order.  ALL: block (0, s) takes every expert of its segment and forms the
// loss.  Else block (x, s) takes COLS experts, and the segment's last block to
// finish forms the loss.  Its results pass the L2 by themselves (store_shared)
// and are waited for before it counts itself done: a release fence would
// write back all of the L2, full of the partial rows (13 us instead of 5; by
// every wave of 1024 blocks, 370).
template <int COLS, bool ALL>
__global__ __launch_bounds__(1024) void balance_join_kernel(const float *__restrict__ psum,
                                                            const int32_t *__restrict__ pcount,
                                                            const int32_t *__restrict__ plive,
                                                            int rows, int E, int k, unsigned *done,
                                                            BalanceOut out)
{
    constexpr int kGroups = 1024 / COLS;
    __shared__ double sums[kGroups][COLS];
    __shared__ int32_t counts[kGroups][COLS], lives[16];
    __shared__ unsigned last;
    const int64_t s = blockIdx.y;
    const int col = threadIdx.x % COLS, g = threadIdx.x / COLS;
    int32_t live = 0;
    for (int r = threadIdx.x; r < rows; r += 1024)
        live += plive[s * rows + r];
    for (int o = kWave / 2; o > 0; o >>= 1)
        live += __shfl_xor(live, o);
    if (lane_id() == 0)
        lives[threadIdx.x / kWave] = live;
    for (int e0 = ALL ? 0 : blockIdx.x * COLS; e0 < (ALL ? E : (static_cast<int>(blockIdx.x) + 1) * COLS); e0 += COLS) {
        const int e = e0 + col;
        const int64_t at = s * rows * E + e;
        double sum = 0.0;
        int32_t count = 0;
        if (e < E)
            for (int r0 = g; r0 < rows; r0 += 8 * kGroups) {
                float v[8];
                int32_t c[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = r0 + i * kGroups;
                    v[i] = r < rows ? psum[at + static_cast<int64_t>(r) * E] : 0.0f;
                    c[i] = r < rows ? pcount[at + static_cast<int64_t>(r) * E] : 0;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    sum += static_cast<double>(v[i]);
                    count += c[i];
                }
            }
        __syncthreads();  // the last experts' sums were read
        sums[g][col] = sum;
        counts[g][col] = count;
        __syncthreads();
        if (g == 0 && e < E) {
            for (int i = 1; i < min(kGroups, rows); ++i) {
                sum += sums[i][col];
                count += counts[i][col];
            }
            if (ALL) {
                out.prob_sums[s * E + e] = static_cast<float>(sum);
                out.counts[s * E + e] = count;
            } else {
                store_shared(&out.prob_sums[s * E + e], static_cast<float>(sum));
                store_shared(&out.counts[s * E + e], count);
            }
        }
    }
    live = 0;
    for (int i = 0; i < 16; ++i)
        live += lives[i];
    if (!ALL) {
        static_assert(ALL || COLS <= kWave, "the first wave writes all results");
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the first wave's results are there
        if (threadIdx.x == 0)
            last = atomicAdd(&done[s], 1u) == gridDim.x - 1 ? 1u : 0u;
        __syncthreads();
        if (!last)
            return;
    }
    __syncthreads();
    write_loss<!ALL>(out.prob_sums + s * E, out.counts + s * E, live, E, k, out.loss + s);
    if (threadIdx.x == 0)
        out.live[s] = live;
}

// Tokens of a segment, two a group of lanes, whose loads and sums run side by
// side; the last ones first, for if the balance loss has just read the logits,
// what the last-level cache still has of them is their end.  So that it stays
// there, the gradient is written past it, and the logits are read for the last
// time.  Front to back with ordinary loads and stores both calls took 22 us longer
// for 131072 tokens of 512 experts (now 154 us), 15 for 256 (now 80).
constexpr int kGradTokens = 2;

template <int L, int NE, bool VEC>
__global__ __launch_bounds__(256) void route_grad_kernel(
    const float *logits, const int32_t *__restrict__ idx, const float *__restrict__ w,
    const float *__restrict__ dw, const uint8_t *__restrict__ mask, const float *__restrict__ dloss,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ live_tokens, int64_t T,
    int64_t seg, int E, int k, bool masked_gates, float *dlogits)  // dlogits may be logits
{
    constexpr int G = 256 / L, kRow = L * NE;  // tokens at a time; experts a row has room for
    __shared__ __align__(16) float rows[G * kRow];
    const int sub = threadIdx.x % L, group = threadIdx.x / L;
    const int64_t s = gridDim.y - 1 - blockIdx.y, end = min(T, (s + 1) * seg);
    const int64_t first = s * seg + static_cast<int64_t>(gridDim.x - 1 - blockIdx.x) * (G * kGradTokens) + group;
    float d[kGradTokens][NE];
    bool live[kGradTokens];
    int e[kGradTokens];
    float wj[kGradTokens], dwj[kGradTokens];
#pragma unroll
    for (int u = 0; u < kGradTokens; ++u) {
        const int64_t t = first + u * G;
        live[u] = t < end && (!mask || mask[t]);
        if (dloss)
            load_row<L, NE, VEC, true>(logits + t * E, E, sub, live[u], d[u]);
        // lane j of the token holds slot j
        const bool slot = dw && sub < k && (masked_gates ? t < end : live[u]);
        e[u] = slot ? idx[t * k + sub] : -1;
        wj[u] = slot ? w[t * k + sub] : 0.0f;
        dwj[u] = slot ? dw[t * k + sub] : 0.0f;
    }
    if (dloss) {
        float c[NE];
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < NE / 4; ++i) {
                const int ee = expert_of<L, VEC>(4 * i, sub);
                i32x4 x{};
                if (ee < E)
                    x = *reinterpret_cast<const i32x4 *>(counts + s * E + ee);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    c[4 * i + q] = static_cast<float>(x[q]);
            }
        } else {
#pragma unroll
            for (int q = 0; q < NE; ++q) {
                const int ee = expert_of<L, VEC>(q, sub);
                c[q] = ee < E ? static_cast<float>(counts[s * E + ee]) : 0.0f;
            }
        }
        const float n = fmaxf(static_cast<float>(live_tokens[s]), 1.0f);
        const float scale = dloss[s] * (static_cast<float>(E) / static_cast<float>(k)) / n / n;
#pragma unroll
        for (int u = 0; u < kGradTokens; ++u) {
            softmax_row<L, NE>(d[u], live[u]);
            float dot = 0.0f;
#pragma unroll
            for (int q = 0; q < NE; ++q)
                dot = fmaf(c[q], d[u][q], dot);
            dot = group_sum<L>(dot);
            const float by = live[u] ? scale : 0.0f;  // a masked row's 0 times an infinite scale would be NaN
#pragma unroll
            for (int q = 0; q < NE; ++q)
                d[u][q] = d[u][q] * (c[q] - dot) * by;
        }
    } else {
#pragma unroll
        for (int u = 0; u < kGradTokens; ++u)
#pragma unroll
            for (int q = 0; q < NE; ++q)
                d[u][q] = 0.0f;
    }
    // The gradients of the slots' logits reach the lanes that hold them through
    // a row of LDS, where an id that occurs twice adds up.
    float *row = rows + group * kRow;
#pragma unroll
    for (int u = 0; u < kGradTokens; ++u) {
        const int64_t t = first + u * G;
        if (dw) {
            const float g = wj[u] * (dwj[u] - group_sum<L>(wj[u] * dwj[u]));
#pragma unroll
            for (int q = 0; q < NE; q += NE >= 4 ? 4 : 1) {
                if (NE >= 4)
                    *reinterpret_cast<float4 *>(row + q * L + 4 * sub) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                else
                    row[q * L + sub] = 0.0f;
            }
            asm volatile("" ::: "memory");  // one wave's LDS operations run in order
            if (static_cast<unsigned>(e[u]) < static_cast<unsigned>(E))
                atomicAdd(row + e[u], g);
            asm volatile("" ::: "memory");
#pragma unroll
            for (int q = 0; q < NE; ++q)
                d[u][q] += row[expert_of<L, VEC>(q, sub)];
            asm volatile("" ::: "memory");
        }
        if (t >= end)
            continue;
        float *out = dlogits + t * E;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < NE / 4; ++i) {
                const int ee = expert_of<L, VEC>(4 * i, sub);
                if (ee < E)
                    __builtin_nontemporal_store(
                        f32x4{d[u][4 * i], d[u][4 * i + 1], d[u][4 * i + 2], d[u][4 * i + 3]},
                        reinterpret_cast<f32x4 *>(out + ee));
            }
        } else {
#pragma unroll
            for (int q = 0; q < NE; ++q) {
                const int ee = expert_of<L, VEC>(q, sub);
                if (ee < E)
                    out[ee] = d[u][q];
            }
        }
    }
}

// Blocks of a segment and their tokens: about 512 blocks over the batch (1024
// leave the join twice the rows: 131072 tokens of 256 experts 84 us instead of
// 79), none under 32 tokens.  Short segments have one block each, and no join, if
// they are many or of few logits (256 tokens of 8 experts: 4.4 us; 16 segments of
// 256 tokens of 256: 10.3, 11.7 with a join; but five of 235 tokens of 995: 57, 19
// with a join).
struct BalanceTiling {
    int tpb, blocks;
};
BalanceTiling balance_tiling(int64_t T, int64_t seg, int E)
{
    int64_t tpb = (T + 511) / 512;
    tpb = tpb < 32 ? 32 : (tpb + 15) / 16 * 16;
    if (tpb > seg || (seg <= 256 && (T >= (E <= 256 ? 16 : 128) * seg || seg * E <= 32768)))
        tpb = seg > 0 ? seg : 1;
    return {static_cast<int>(tpb), static_cast<int>(seg > 0 ? (seg + tpb - 1) / tpb : 1)};
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t balance_workspace_bytes(int64_t T, int64_t seg, int E)
{
    const size_t S = layout_chunks(T, seg), rows = S * balance_tiling(T, seg, E).blocks;
    return round256(rows * E * 4) * 2 + round256(rows * 4) + round256(S * 4);
}

// Calls F with the lanes per token, elements per lane and vector flag of a
// router over E experts.
#define MOE_ROUTER_SHAPE(E, VEC, F)                                                            \
    if (E <= 16) { F(16, 1, false); }                                                          \
    else if (E <= 32) { F(16, 2, false); }                                                     \
    else if (E <= 64) { if (VEC) { F(16, 4, true); } else { F(16, 4, false); } }               \
    else if (E <= 128) { if (VEC) { F(16, 8, true); } else { F(16, 8, false); } }              \
    else if (E <= 256) { if (VEC) { F(16, 16, true); } else { F(16, 16, false); } }            \
    else if (E <= 512) { if (VEC) { F(64, 8, true); } else { F(64, 8, false); } }              \
    else { if (VEC) { F(64, 16, true); } else { F(64, 16, false); } }

hipError_t launch_balance_loss(const float *logits, const int32_t *idx, const uint8_t *mask,
                               int64_t T, int64_t seg, int E, int k, float *loss, int32_t *counts,
                               float *prob_sums, int32_t *live, void *workspace,
                               hipStream_t stream)
{
    const int S = layout_chunks(T, seg);
    const BalanceTiling bt = balance_tiling(T, seg, E);
    const size_t rows = static_cast<size_t>(S) * bt.blocks;
    char *ws = static_cast<char *>(workspace);
    float *psum = reinterpret_cast<float *>(ws);
    int32_t *pcount = reinterpret_cast<int32_t *>(ws + round256(rows * E * 4));
    int32_t *plive = reinterpret_cast<int32_t *>(ws + 2 * round256(rows * E * 4));
    unsigned *done = reinterpret_cast<unsigned *>(ws + 2 * round256(rows * E * 4) + round256(rows * 4));
    const BalanceOut out{loss, counts, prob_sums, live};
    const bool vec = E % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0;
    const bool one = bt.blocks == 1;
    const int threads = one && E <= 256 ? 1024 : E <= 512 ? 512 : 256;
    const size_t lds = (static_cast<size_t>(threads / kWave) * E + E + 1) * 4;
    const dim3 grid(bt.blocks, S);
#define MOE_BALANCE(L, NE, V)                                                                  \
    if (one)                                                                                   \
        balance_partial_kernel<L, NE, V, true><<<grid, threads, lds, stream>>>(                \
            logits, idx, mask, T, seg, bt.tpb, E, k, psum, pcount, plive, done, out);          \
    else                                                                                       \
        balance_partial_kernel<L, NE, V, false><<<grid, threads, lds, stream>>>(               \
            logits, idx, mask, T, seg, bt.tpb, E, k, psum, pcount, plive, done, out)
    MOE_ROUTER_SHAPE(E, vec, MOE_BALANCE)
#undef MOE_BALANCE
    hipError_t err = hipGetLastError();
    if (err != hipSuccess || one)
        return err;
    // many segments fill the card with a block each
    if (S >= 16)
        balance_join_kernel<64, true><<<dim3(1, S), 1024, 0, stream>>>(psum, pcount, plive, bt.blocks, E, k, done, out);
    else
        balance_join_kernel<16, false><<<dim3((E + 15) / 16, S), 1024, 0, stream>>>(psum, pcount, plive, bt.blocks, E,
                                                                                    k, done, out);
    return hipGetLastError();
}

int64_t route_grad_blocks(int64_t seg, int E)
{
    const int per = (E <= 256 ? 16 : 4) * kGradTokens;
    return (seg + per - 1) / per;
}

hipError_t launch_route_grad(const float *logits, const int32_t *idx, const float *w,
                             const float *dw, const uint8_t *mask, const float *dloss,
                             const int32_t *counts, const int32_t *live, int64_t T, int64_t seg,
                             int E, int k, bool masked_gates, float *dlogits, hipStream_t stream)
{
    const bool vec = E % 4 == 0 && ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(counts) |
                                     reinterpret_cast<uintptr_t>(dlogits)) & 15) == 0;
    const dim3 grid(static_cast<unsigned>(route_grad_blocks(seg, E)), layout_chunks(T, seg));
#define MOE_ROUTE_GRAD(L, NE, V)                                                               \
    route_grad_kernel<L, NE, V><<<grid, 256, 0, stream>>>(                                     \
        logits, idx, w, dw, mask, dloss, counts, live, T, seg, E, k, masked_gates, dlogits)
    MOE_ROUTER_SHAPE(E, vec, MOE_ROUTE_GRAD)
#undef MOE_ROUTE_GRAD
    return hipGetLastError();
}

}  // namespace moe
