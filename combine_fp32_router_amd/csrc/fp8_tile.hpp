// One output tile of the 8-bit products on the matrix cores.
//
// C[row, col] = sum over blocks b of 128 r of s[row, b] t[col / 128, b] sum_{r in
// b} Q[row, r] P[col, r]: 256 rows by 256 columns a workgroup of eight waves, two
// on each SIMD, 64 x 128 a wave.  A block's codes are one 16x16x128 MFMA of C = 0,
// whose four results a lane are then scaled into fp32 accumulators: 16 cycles of
// the vector unit beside the MFMA's 32, which the two waves of a SIMD fill in turn.
// A result is scaled three MFMAs after its own, when it is there.
//
// Wave w has the columns' half w % 2 and, of every block of 64 rows, the 16 from
// 16 (w / 2), so that a short tile's rows are shared evenly.  GATED: columns come
// in blocks of 32, gate and up in turn.
//
// r is walked 128 at a time through two LDS stages, filled by loads that go from
// memory to LDS without passing registers, as in expert_tile.hpp: an image row is
// 128 bytes, its 16-byte pieces permuted so that the reads fall on different banks.
// A wave holds its rows' fragments over a stage and streams its columns'.
//
// 8192 rows, 7168 -> 8192, normal data: 2.05 PFLOP/s, the same of zeros 2.65: what the
// matrix cores draw sets the clock.  Left out for timing, the reads of LDS bring the
// 2.05 to 2.43 and the scaling to 2.25, so neither alone is what bounds it (a library
// product of the same codes under one scale: 3.1).  MFMAs of 32x32x64: 1.97.
#pragma once

#include "expert_finish.hpp"
#include "expert_list.hpp"
#include "fp8_codes.hpp"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// The lane, as a value of its own: what is worked out from it is not kept over the
// tiles' loop, where there are no registers for it (the reloads of spilled ones waited
// for every store of a tile's results: 30 us a tile.  One of the plain gradient's is still
// spilled, and reloaded there).
__device__ __forceinline__ int fresh_lane()
{
    int lane = lane_id();
    asm volatile("" : "+v"(lane));
    return lane;
}

#define MOE_SCALAR __attribute__((address_space(4)))

template <bool GATED>
struct CodeTile {
    static constexpr int kWaves = 8, kFrags = 8;  // blocks of 16 columns of a wave
    static constexpr int kImage = 8192;                        // 64 indices of 128 bytes
    static constexpr int kStage = 8 * kImage, kQ = 4 * kImage;
    static constexpr int kScales = 2 * kStage;                 // the rows' scales: of 4 steps, and of the next 4
    static constexpr int kOutBytes = 4096;
    static constexpr int kTops = kScales + 2 * 4096;           // rows' largest sizes, which two waves put together
    static constexpr int kLdsBytes = kTops + 1024;

    // where the operands are, for this lane
    const char *p, *q, *xs;
    int pitch, pn, n, R, steps, blocks;  // bytes of a row; columns and rows inside; a segment's length; steps in all, of a segment
    int p_off, q_off, piece;             // of the first load
    int xs_off, xs_lane, xs_step, xs_bytes, xs_pitch;
    const MOE_SCALAR float *ws[GATED ? 2 : 1];  // (uniform, and no kernel writes what it reads here)

    __device__ __forceinline__ int wave() const { return static_cast<int>(uniform(threadIdx.x / kWave)); }
    __device__ __forceinline__ int col0() const { return wave() % 2 * 128; }
    __device__ __forceinline__ int row0(int block) const { return block * 64 + wave() / 2 * 16; }
    // LDS of a wave's results, in what the next tile's second stage gets last: the
    // columns' second half, and the rows from 128 on.
    __device__ __forceinline__ MOE_LDS char *out_place(MOE_LDS char *lds) const
    {
        const int w = wave();
        return lds + kStage + (w < 2 ? kImage : w < 4 ? 3 * kImage : kQ + w / 2 * kImage) + w % 2 * kOutBytes;
    }

    static __device__ __forceinline__ int place_of(int c, int i) { return c ^ (i / 2 % 8); }

    // Columns at w (GATED: up weights at w_up), n_cols of them inside; n_rows rows
    // at x.  `segments` of R bytes each make a row.
    __device__ __forceinline__ void init(const uint8_t *w, const uint8_t *w_up, int n_cols, const uint8_t *x, int n_rows,
                                         const float *x_scales, int xs_cols, int R_, int segments)
    {
        const int v = wave(), lane = fresh_lane(), in64 = v * 8 + lane / 8;
        R = R_;
        pitch = R * segments;
        blocks = code_blocks(R);
        steps = blocks * segments;
        pn = n_cols;
        n = n_rows;
        piece = place_of(lane % 8, in64) * 16;
        p = reinterpret_cast<const char *>(GATED && v >= 4 ? w_up : w);
        q = reinterpret_cast<const char *>(x);
        p_off = (GATED ? in64 % 32 : in64) * pitch + piece;
        q_off = in64 * pitch + piece;
        xs = reinterpret_cast<const char *>(x_scales);
        xs_step = xs_cols == 1 ? 0 : 4;
        xs_bytes = n * xs_cols * 4;
        xs_pitch = xs_cols * 4;
        xs_off = (v / 2 * 16 + lane / 4) * xs_pitch + lane % 4 * xs_step;
        xs_lane = lane % 4;
    }

    // Everything but the lane's own offsets is the same in all lanes.  If the compiler
    // loses sight of that, every load gets a loop around it, so it is told again
    // in front of a tile's product.
    template <typename V>
    static __device__ __forceinline__ void keep_uniform(V &v)
    {
        if constexpr (sizeof(V) == 8) {
            const uint64_t u = (uint64_t)v;
            v = (V)(static_cast<uint64_t>(uniform(static_cast<uint32_t>(u >> 32))) << 32 | uniform(static_cast<uint32_t>(u)));
        } else {
            v = static_cast<V>(uniform(static_cast<uint32_t>(v)));
        }
    }
    __device__ __forceinline__ void all_uniform()
    {
        keep_uniform(p);
        keep_uniform(q);
        keep_uniform(xs);
        keep_uniform(pitch);
        keep_uniform(pn);
        keep_uniform(n);
        keep_uniform(R);
        keep_uniform(steps);
        keep_uniform(blocks);
        keep_uniform(xs_step);
        keep_uniform(xs_bytes);
        keep_uniform(xs_pitch);
#pragma unroll
        for (int g = 0; g < (GATED ? 2 : 1); ++g)
            keep_uniform(ws[g]);
    }

    // Bytes of a row in front of step k, and those of them that step has (<= 0 past
    // the end).
    __device__ __forceinline__ int first_of(int k) const { return k >= blocks ? k * kCodeBlock - (blocks * kCodeBlock - R) : k * kCodeBlock; }
    __device__ __forceinline__ int live_of(int k) const
    {
        return k >= steps ? 0 : R - (k >= blocks ? k - blocks : k) * kCodeBlock;
    }
    __device__ __forceinline__ void load_p(MOE_LDS char *__restrict__ stage, int k, int j) const
    {
        const int r0 = first_of(k);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(row_rsrc(const_cast<char *>(p) + r0, max(0, pn * pitch - r0)),
                                                 (MOE_LDS void *)(stage + j * kImage + wave() * 1024), 16,
                                                 piece < live_of(k) ? p_off + j * (GATED ? 32 : 64) * pitch : kOutside, 0, 0, 0);
    }
    __device__ __forceinline__ void load_q(MOE_LDS char *__restrict__ stage, int k, int j) const
    {
        const int r0 = first_of(k);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(row_rsrc(const_cast<char *>(q) + r0, max(0, n * pitch - r0)),
                                                 (MOE_LDS void *)(stage + kQ + j * kImage + wave() * 1024), 16,
                                                 piece < live_of(k) ? q_off + j * 64 * pitch : kOutside, 0, 0, 0);
    }
    // The i-th load of the rows' scales: of 16 rows (of row block i % 4) for the four
    // steps from i - i % 4, so that a row's line is asked for every fourth step: asked
    // for in every step, for 64 rows, the scales were a third of the requests to L2.
    // (Both waves of a group of rows write the same to the same place.)
    __device__ __forceinline__ void load_scales(MOE_LDS char *__restrict__ lds, int i) const
    {
        const int k = i & ~3, h = i & 3;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            row_rsrc(const_cast<char *>(xs), xs_bytes),
            (MOE_LDS void *)(lds + kScales + (i / 4 % 2) * 4096 + wave() / 2 * 1024 + h * 256), 4,
            k + xs_lane < steps ? xs_off + h * 64 * xs_pitch + k * xs_step : kOutside, 0, 0, 0);
    }

    // As Tile::join.
    template <int LEFT>
    static __device__ __forceinline__ void join()
    {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0x0070 | (LEFT & 15) | (LEFT >> 4) << 14);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }

    // 16 indices from i0 of an image, lane l's index l % 16: two pieces of its row,
    // the same ones for both operands.
    static __device__ __forceinline__ i32x8 frag(const MOE_LDS char *__restrict__ image, int i0)
    {
        const int lane = lane_id(), i = lane % 16;
        const MOE_LDS char *row = image + (i0 + i) * kCodeBlock;
        const i32x4 lo = *reinterpret_cast<const MOE_LDS i32x4 *>(row + place_of(lane / 16, i) * 16);
        const i32x4 hi = *reinterpret_cast<const MOE_LDS i32x4 *>(row + place_of(4 + lane / 16, i) * 16);
        return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }

    // NB: blocks of 64 rows that the tile has (1, 2 or 4).  For few of them the columns'
    // fragments are read further ahead.
    template <int NB>
    struct Regs {
        static constexpr int kBlocks = NB, kAhead = NB >= 3 ? 2 : 4;
        i32x8 pf[kAhead], qf[NB];
        f32x4 d[4];
        float xv[NB], s[GATED ? 2 : 1][NB];
        float wv[GATED ? 2 : 1];
        f32x4 acc[kFrags][NB];
    };
    template <int NB>
    __device__ __forceinline__ void read_p(Regs<NB> &f, int c, const MOE_LDS char *__restrict__ stage) const
    {
        f.pf[c % Regs<NB>::kAhead] = frag(stage, col0() + c * 16);
    }
    template <int NB>
    __device__ __forceinline__ void read_q(Regs<NB> &f, int h, const MOE_LDS char *__restrict__ stage) const
    {
        f.qf[h] = frag(stage + kQ, row0(h));
    }
    template <int NB>
    __device__ __forceinline__ void read_scales(Regs<NB> &f, const MOE_LDS char *__restrict__ lds, int k) const
    {
#pragma unroll
        for (int h = 0; h < NB; ++h)
            f.xv[h] = *reinterpret_cast<const MOE_LDS float *>(lds + kScales + (k / 4 % 2) * 4096 + wave() / 2 * 1024 +
                                                               h * 256 + lane_id() % 16 * 16 + k % 4 * 4);
    }
    __device__ __forceinline__ float scale_at(int g, int k) const { return ws[g][min(k, steps - 1)]; }

    // The loads that a tile's first steps expect to be in flight, of `nb` blocks of
    // rows; run() itself loads the second stage's rows from 128 on.
    __device__ __forceinline__ void start(MOE_LDS char *lds, int nb) const
    {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            MOE_LDS char *stage = lds + k * kStage;
#pragma unroll
            for (int j = 0; j < (k == 0 ? 4 : 2); ++j)
                if (j < nb)
                    load_q(stage, k, j);
            load_p(stage, k, 0);
            load_p(stage, k, 2);
#pragma unroll
            for (int i = 4 * k; i < 4 + k; ++i)
                load_scales(lds, i);
            if (k == 0) {
                load_p(stage, k, 1);
                load_p(stage, k, 3);
            }
        }
    }

    template <int NB>
    __device__ __forceinline__ void load_rest(const Regs<NB> &, MOE_LDS char *lds) const
    {
#pragma unroll
        for (int j = 2; j < NB; ++j)
            load_q(lds + kStage, 1, j);
    }

    // The scaled addition that is due after MFMA m of a step (m - 3 of the ring).
    template <int NB>
    static __device__ __forceinline__ void add(Regs<NB> &f, int m)
    {
        const int c = m / NB, h = m % NB;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            f.acc[c][h][j] = fmaf(f.d[m % 4][j], f.s[GATED ? c / 2 % 2 : 0][h], f.acc[c][h][j]);
    }

    // Step k, whose stage is at offset `cur`.  An image is refilled (rows and the
    // columns' first half for step k + 2, their second half for k + 1) as soon as a
    // join has shown that every wave has read it.
    template <int NB>
    __device__ __forceinline__ void step(Regs<NB> &f, const MOE_LDS char *__restrict__ rd, MOE_LDS char *__restrict__ wr,
                                         int cur, int nxt, int k) const
    {
        constexpr int A = Regs<NB>::kAhead, kSlots = 8 * NB;
        constexpr int kFirst = A == 2 ? 2 : 1;                     // column block at which the first join is
        constexpr int L1 = 2 + NB, L2 = 3;                         // loads behind the joins
        constexpr int T1 = (4 - kFirst) * NB, T2 = 3 * NB;         // slots for them
#pragma unroll
        for (int m = 0; m < kSlots; ++m) {
            const int c = m / NB, h = m % NB;
            if (h == 0 && c == kFirst)
                join<NB + 3>();  // the columns' second half of this step is here; that of the last was read
            if (h == 0 && c == 4) {
#pragma unroll
                for (int g = 0; g < (GATED ? 2 : 1); ++g)
                    f.wv[g] = scale_at(g, k + 1);
                join<2 + NB>();  // rows, scales and the columns' first half of the next step are here; these were read
            }
            f.d[m % 4] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f.pf[c % A], f.qf[h], f32x4{}, 0, 0, 0, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            if (h == 0) {
                const int to = c + A - 1;
                read_p(f, to % 8, rd + (to < 8 ? cur : nxt));
            }
            if (c == 7) {
                read_q(f, h, rd + nxt);
                if (h == NB - 1)
                    read_scales(f, rd, k + 1);
            }
            const int t1 = m - kFirst * NB, t2 = m - 4 * NB;
            if (t1 >= 0 && t1 < T1)
#pragma unroll
                for (int i = t1 * L1 / T1; i < (t1 + 1) * L1 / T1; ++i) {
                    if (i < 2)
                        load_p(wr + nxt, k + 1, 1 + 2 * i);
                    else
                        load_q(wr + cur, k + 2, i - 2);
                }
            if (t2 >= 0 && t2 < T2)
#pragma unroll
                for (int i = t2 * L2 / T2; i < (t2 + 1) * L2 / T2; ++i) {
                    if (i < 2)
                        load_p(wr + cur, k + 2, 2 * i);
                    else
                        load_scales(wr, k + 5);
                }
            // the scales of step k come into use with its first result
            if (m == 3) {
#pragma unroll
                for (int g = 0; g < (GATED ? 2 : 1); ++g)
#pragma unroll
                    for (int i = 0; i < NB; ++i)
                        f.s[g][i] = f.xv[i] * f.wv[g];
            }
            add(f, (m + kSlots - 3) % kSlots);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // The product of a tile of at most NB blocks whose start(lds, NB) is under way, in
    // f.acc.
    template <typename F>
    __device__ __forceinline__ void run(F &f, MOE_LDS char *lds) const
    {
        constexpr int NB = F::kBlocks;
#pragma unroll
        for (int g = 0; g < (GATED ? 2 : 1); ++g) {
            f.wv[g] = scale_at(g, 0);
#pragma unroll
            for (int h = 0; h < NB; ++h)
                f.s[g][h] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f.d[i] = f32x4{};
#pragma unroll
        for (int c = 0; c < kFrags; ++c)
#pragma unroll
            for (int h = 0; h < NB; ++h)
                f.acc[c][h] = f32x4{};
        join<2 + (NB > 2 ? 2 : NB) + 3>();  // all but the columns' second half
        load_rest(f, lds);
#pragma unroll
        for (int h = 0; h < NB; ++h)
            read_q(f, h, lds);
#pragma unroll
        for (int c = 0; c < Regs<NB>::kAhead - 1; ++c)
            read_p(f, c, lds);
        read_scales(f, lds, 0);
        int cur = 0, nxt = kStage;
#pragma unroll 1
        for (int k = 0; k < steps; ++k) {
            step(f, lds, lds, cur, nxt, k);
            const int t = cur;
            cur = nxt;
            nxt = t;
        }
#pragma unroll
        for (int m = 8 * NB - 3; m < 8 * NB; ++m)
            add(f, m);
        join<0>();
    }

    // The largest of both column halves' sizes of this lane's row, of row block i.
    __device__ __forceinline__ uint32_t both_halves(MOE_LDS char *lds, int i, uint32_t top, int lane) const
    {
        MOE_LDS uint32_t *tops = reinterpret_cast<MOE_LDS uint32_t *>(lds + kTops) + i % 2 * 128;
        const int at = wave() * 16 + lane % 16;
        tops[at] = top;  // (four lanes of a row, the same value)
        join<63>();
        return umax(top, tops[at ^ 16]);
    }
};

}  // namespace moe
