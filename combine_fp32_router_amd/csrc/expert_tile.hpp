// One output tile of the experts' products on the matrix cores.
//
// C[row, col] = sum over r < R of Q[row, r] * P[col, r], BR rows and BC
// columns, by WR x WC waves of (BR/WR) x (BC/WC) each, in 32x32x16 bf16
// MFMAs whose first operand is P: lane l then holds row l%32 and, in
// registers 4g..4g+3, columns 8g + 4(l/32).. of a 32x32 block.
//
// r is walked 64 at a time through two LDS stages, filled by loads that go
// from memory to LDS without passing registers.  Such a load writes 16 bytes
// a lane to consecutive LDS addresses, so the LDS image cannot be padded;
// instead a lane fetches a permuted 16-byte piece of its row, chosen so that
// the reads below fall on different banks:
//   r contiguous in memory:  image [index][64 r], piece c of row i at c ^ (i/2)%8;
//     a lane reads its eight r values with one 16-byte read.
//   index contiguous:        image [64 r][index], piece c of row r at c ^ 4(r%4);
//     two transposing 8-byte reads of four r rows give the same eight values.
// Out of range reads of the buffer descriptor return zeros, so short tiles
// and the end of r need no other care.
#pragma once

#include "expert_rows.hpp"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

#define MOE_LDS __attribute__((address_space(3)))

constexpr int kOutside = static_cast<int>(0x80000000u);  // an offset past every descriptor

// ---- order of the tiles

// Total tiles of `height` rows over all runs.
__device__ __forceinline__ int count_row_tiles(const int32_t *__restrict__ offsets, int E,
                                               int max_rows, int height)
{
    int n = 0;
    for (int e = lane_id(); e < E; e += kWave)
        n += (expert_run(offsets, e, max_rows).n + height - 1) / height;
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1)
        n += __shfl_xor(n, o);
    return static_cast<int>(uniform(n));
}

// Workgroup b runs on XCD b % 8, each with an L2 of its own: give every XCD a
// contiguous range of the n tiles.  -1 for the grid's spare workgroups.
__device__ __forceinline__ int xcd_order(int b, int n)
{
    const int x = b % 8, i = b / 8, each = n / 8, more = n % 8;
    if (i >= each + (x < more))
        return -1;
    return x * each + min(x, more) + i;
}

struct TileAt {
    int row, col;
};

// Groups of eight row tiles, all columns of a group before the next: tiles
// that run side by side share both operands' pieces in L2.
__device__ __forceinline__ TileAt grouped_order(int id, int row_tiles, int col_tiles)
{
    const int group = id / (8 * col_tiles), in = id % (8 * col_tiles);
    const int height = min(8, row_tiles - 8 * group);
    return {8 * group + in % height, in / height};
}

// ---- operands

// Tile of W indices of an operand, 64 r a stage, staged by NW waves.
// CONTIG: memory [index][r], else [r][index].  PAIR: indices come in blocks
// of 32 from two places in turn (gate and up weights).
template <int W, int NW, bool CONTIG, bool PAIR>
struct Operand {
    static constexpr int kBytes = W * 128;
    static constexpr int kLoads = W * 128 / 1024 / NW;  // of 1 KiB, per wave and stage
    static constexpr int kRowsLoad = CONTIG ? 8 : 512 / W;  // memory rows a load covers
    static_assert(W * 128 % (1024 * NW) == 0 && (CONTIG || !PAIR), "whole loads");
    static_assert(CONTIG || (kRowsLoad * NW) % 4 == 0, "a wave's loads permute alike");
    const char *base;
    int pitch, n;  // bytes a memory row, indices inside
    int off;       // this lane's offset in the wave's first load
    int piece;     // CONTIG: its first r within the stage, the same in each of its loads

    __device__ __forceinline__ void init(const uint16_t *p, const uint16_t *p2, int pitch_, int n_)
    {
        // PAIR: each of a wave's loads covers 8 indices of a block of the same kind
        static_assert(!PAIR || NW % 8 == 0, "whole pairs of blocks");
        base = reinterpret_cast<const char *>(PAIR && uniform(threadIdx.x / kWave) / 4 % 2 ? p2 : p);
        pitch = pitch_ * 2;
        n = n_;
        const int w = threadIdx.x / kWave, lane = lane_id();
        if (CONTIG) {
            const int i = w * 8 + lane / 8;
            const int row = PAIR ? i / 64 * 32 + i % 32 : i;
            static_assert(!CONTIG || NW % 2 == 0, "a wave's loads permute alike");
            piece = ((lane % 8) ^ (i / 2 % 8)) * 8;
            off = row * pitch + piece * 2;
        } else {
            constexpr int kPieces = W / 8;
            const int r = w * kRowsLoad + lane / kPieces;
            off = r * pitch + ((lane % kPieces) ^ (r % 4 * 4)) * 16;
        }
    }

    // Starts this wave's j-th load of r0 .. r0 + 63 into `image`.
    __device__ __forceinline__ void fetch(MOE_LDS char *__restrict__ image, int r0, int R, int j) const
    {
        const int load = static_cast<int>(uniform(threadIdx.x / kWave)) + j * NW;
        MOE_LDS void *to = (MOE_LDS void *)(image + load * 1024);
        if (CONTIG) {
            // the row's pieces past R; adding rows to kOutside stays outside
            const int at = (r0 + piece < R ? off : kOutside) + j * (PAIR ? NW * 4 : NW * 8) * pitch;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                row_rsrc(const_cast<char *>(base) + static_cast<int64_t>(r0) * 2, max(0, n * pitch - r0 * 2)), to, 16, at, 0, 0, 0);
        } else {
            const int rows = min(64, R - r0);  // <= 0 past the end: nothing is read
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                row_rsrc(const_cast<char *>(base) + static_cast<int64_t>(r0) * pitch, rows > 0 ? (rows - 1) * pitch + n * 2 : 0), to, 16,
                off + j * NW * kRowsLoad * pitch, 0, 0, 0);
        }
    }

    // This lane's place in the image for the fragments that start at index 0
    // and r = s.
    static __device__ __forceinline__ int lane_place(int s)
    {
        const int lane = lane_id();
        if (CONTIG)
            return lane % 32 * 128 + ((s / 8 + lane / 32) ^ (lane % 32 / 2 % 8)) * 16;
        const int r = s + lane / 32 * 8 + lane % 16 / 4, i = lane / 16 % 2 * 16 + lane % 4 * 4;
        return r * (2 * W) + ((i / 8) ^ (r % 4 * 4)) * 16 + i % 8 * 2;
    }

    // The fragment of indices i0 .. i0 + 31 (i0 a multiple of 32) and r = s ..
    // s + 15; `place` is lane_place(s).
    static __device__ __forceinline__ bf16x8 frag(const MOE_LDS char *__restrict__ image, int i0, int place)
    {
        if constexpr (CONTIG) {
            return *reinterpret_cast<const MOE_LDS bf16x8 *>(image + i0 * 128 + place);
        } else {
            // i0 adds 4 pieces a block of 32, under the same permutation
            const MOE_LDS char *p = image + (place ^ (i0 * 2));
            const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((MOE_LDS bf16x4 *)(p));
            const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((MOE_LDS bf16x4 *)(p + 4 * 2 * W));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
};

template <int BR, int BC, int WR, int WC, bool P_CONTIG, bool Q_CONTIG, bool GATED>
struct Tile {
    static constexpr int NW = WR * WC;
    static constexpr int kRowFrags = BR / WR / 32, kColFrags = BC / WC / 32;
    typedef Operand<BC, NW, P_CONTIG, GATED> P;
    typedef Operand<BR, NW, Q_CONTIG, false> Q;
    static constexpr int kStageBytes = P::kBytes + Q::kBytes;
    P p;
    Q q;
    int R;
    f32x16 acc[kColFrags][kRowFrags];
    f32x16 sums;  // SUMS: sums of Q over r, of the row block that this wave keeps

    __device__ __forceinline__ int wave() const { return static_cast<int>(uniform(threadIdx.x / kWave)); }
    __device__ __forceinline__ int col0() const { return wave() % WC * (BC / WC); }
    __device__ __forceinline__ int row0() const { return wave() / WC * (BR / WR); }

    __device__ __forceinline__ void init(const uint16_t *pp, const uint16_t *pp2, int ppitch, int pn,
                                         const uint16_t *qp, int qpitch, int qn, int R_)
    {
        p.init(pp, pp2, ppitch, pn);
        q.init(qp, nullptr, qpitch, qn);
        R = R_;
        sums = f32x16{};
#pragma unroll
        for (int r = 0; r < kRowFrags; ++r)
#pragma unroll
            for (int c = 0; c < kColFrags; ++c)
                acc[c][r] = f32x16{};
    }

    struct Frags {
        bf16x8 p[kColFrags], q[kRowFrags];
    };
    __device__ __forceinline__ void read(Frags &f, const MOE_LDS char *__restrict__ cur, int s) const
    {
        const int pl = P::lane_place(s), ql = Q::lane_place(s);
#pragma unroll
        for (int c = 0; c < kColFrags; ++c)
            f.p[c] = P::frag(cur, col0() + c * 32, pl);
#pragma unroll
        for (int r = 0; r < kRowFrags; ++r)
            f.q[r] = Q::frag(cur + P::kBytes, row0() + r * 32, ql);
    }

    // SUMS: wave column c also multiplies its row block c by ones.
    static_assert(kRowFrags <= WC, "a wave column for each row block");

    // Multiplies the stage at `cur` while the loads of the next one, at r0,
    // run into `nxt`.
    template <bool SUMS>
    __device__ __forceinline__ void step(const MOE_LDS char *__restrict__ cur, MOE_LDS char *__restrict__ nxt, int r0)
    {
        Frags f[2];
        read(f[0], cur, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = i * P::kLoads / 4; j < (i + 1) * P::kLoads / 4; ++j)
                p.fetch(nxt, r0, R, j);
#pragma unroll
            for (int j = i * Q::kLoads / 4; j < (i + 1) * Q::kLoads / 4; ++j)
                q.fetch(nxt + P::kBytes, r0, R, j);
            if (i < 3)
                read(f[(i + 1) % 2], cur, 16 * (i + 1));
#pragma unroll
            for (int c = 0; c < kColFrags; ++c)
#pragma unroll
                for (int r = 0; r < kRowFrags; ++r)
                    acc[c][r] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % 2].p[c], f[i % 2].q[r], acc[c][r], 0, 0, 0);
            if (SUMS) {
                const __bf16 one = static_cast<__bf16>(1.0f);
                const bf16x8 ones = {one, one, one, one, one, one, one, one};
                bf16x8 mine = f[i % 2].q[0];
#pragma unroll
                for (int r = 1; r < kRowFrags; ++r)
                    mine = wave() % WC == r ? f[i % 2].q[r] : mine;
                sums = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ones, mine, sums, 0, 0, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // Waits for the loads in flight and for the other waves.
    static __device__ __forceinline__ void join()
    {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }

    template <bool SUMS = false>
    __device__ __forceinline__ void run(char (&lds)[2][kStageBytes])
    {
        MOE_LDS char *cur = (MOE_LDS char *)lds[0], *nxt = (MOE_LDS char *)lds[1];
        if (R <= 0)
            return;
#pragma unroll
        for (int j = 0; j < P::kLoads; ++j)
            p.fetch(cur, 0, R, j);
#pragma unroll
        for (int j = 0; j < Q::kLoads; ++j)
            q.fetch(cur + P::kBytes, 0, R, j);
#pragma unroll 1
        for (int r0 = 0; r0 < R; r0 += 64) {
            join();
            step<SUMS>(cur, nxt, r0 + 64);
            MOE_LDS char *t = cur;
            cur = nxt;
            nxt = t;
        }
    }

    // Calls f(row, column, values, up values) for eight columns of one row at
    // a time: 32 rows of a wave's columns go through its part of LDS, so that
    // lanes take neighbouring columns and memory sees whole lines.  GATED:
    // `column` counts output columns, the gate's values and the up values.
    static constexpr int kWaveCols = BC / WC, kOutPitch = kWaveCols + 4;  // floats; rows 4 banks apart
    static_assert(NW * 32 * kOutPitch * 4 <= 2 * kStageBytes, "fits the stages");
    template <typename F>
    __device__ __forceinline__ void finish(char (&lds)[2][kStageBytes], F f)
    {
        join();
        const int lane = lane_id();
        float *mine = reinterpret_cast<float *>(lds[0]) + wave() * (32 * kOutPitch);
#pragma unroll
        for (int r = 0; r < kRowFrags; ++r) {
#pragma unroll
            for (int c = 0; c < kColFrags; ++c)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    *reinterpret_cast<float4 *>(mine + lane % 32 * kOutPitch + c * 32 + g * 8 + lane / 32 * 4) =
                        make_float4(acc[c][r][4 * g], acc[c][r][4 * g + 1], acc[c][r][4 * g + 2], acc[c][r][4 * g + 3]);
            constexpr int kOuts = kWaveCols / (GATED ? 2 : 1) / 8;  // of a row
#pragma unroll 1
            for (int i = lane; i < 32 * kOuts; i += kWave) {
                const int row = i / kOuts, o = i % kOuts * 8;
                // gated: blocks of 32 gate and 32 up columns in turn
                const float *src = mine + row * kOutPitch + (GATED ? o / 32 * 64 + o % 32 : o);
                float v[8], u[8];
#pragma unroll
                for (int h = 0; h < 8; h += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(src + h);
                    v[h] = x.x, v[h + 1] = x.y, v[h + 2] = x.z, v[h + 3] = x.w;
                    if (GATED) {
                        const float4 y = *reinterpret_cast<const float4 *>(src + 32 + h);
                        u[h] = y.x, u[h + 1] = y.y, u[h + 2] = y.z, u[h + 3] = y.w;
                    }
                }
                f(row0() + r * 32 + row, col0() / (GATED ? 2 : 1) + o, v, u);
            }
        }
    }
};

}  // namespace moe
