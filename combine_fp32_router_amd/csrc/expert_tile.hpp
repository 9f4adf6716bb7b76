// One output tile of the experts' products on the matrix cores.
//
// C[row, col] = sum over r < R of Q[row, r] * P[col, r]: 256 rows by 256
// columns (or 128, for calls of few tiles) a workgroup of four waves, one on
// each SIMD, 128 x 128 (64) a wave in 16x16x32 bf16 MFMAs.  Their first operand is P, so lane l holds columns
// 4 (l/16) .. + 3 of a block's row l%16.  The wave's 256 accumulator
// registers are the AGPR half of its 512: the MFMAs are written as inline
// assembly on "a" registers, because the compiler, given the builtin, copies
// accumulators between the two halves in the loop.
//
// Four waves of 128 x 128 read 128 KiB of LDS for 64 r, eight of 128 x 64
// would read 192; with real data, where the card's power limits the clock,
// that is worth 10% (8192 x 8192, r 7168, time of 64 r: 1.33 against 1.45 us).
//
// r is walked 64 at a time through two LDS stages, filled by loads that go
// from memory to LDS without passing registers.  Such a load writes 16 bytes
// a lane to consecutive LDS addresses, so the LDS image cannot be padded;
// instead a lane fetches a permuted 16-byte piece of its row, chosen so that
// the reads fall on different banks:
//   r contiguous in memory: image [index][64 r]; a lane reads its eight r
//     values with one 16-byte read.
//   index contiguous:       image [64 r][index]; two transposing 8-byte reads
//     of four r rows give the same eight values.
// Reads of a buffer descriptor outside its range return zeros, so short tiles
// and the end of r need no other care.
#pragma once

#include "expert_finish.hpp"
#include "expert_list.hpp"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

constexpr int kTileWaves = 4;

// Image of W indices of an operand, kStep r a stage, staged by four waves.
// CONTIG: memory [index][r], else [r][index].  PAIR: indices come in blocks
// of 32 from two places in turn (gate and up weights).
template <int W, bool CONTIG, bool PAIR>
struct Operand {
    static constexpr int kBytes = W * kStep * 2;
    static constexpr int kLoads = kBytes / 1024 / kTileWaves;   // of 1 KiB, per wave and stage
    static constexpr int kPieces = CONTIG ? kStep / 8 : W / 8;  // 16-byte pieces of an image row
    static constexpr int kRowsLoad = 64 / kPieces;              // image rows a load covers
    static constexpr bool kSwap = !CONTIG && W == 256;          // a wave's loads lie 8 r apart
    static_assert((CONTIG || !PAIR) && (CONTIG || W == 64 || W == 128 || W == 256), "the permutations below");
    const char *base[PAIR ? 2 : 1];
    int pitch, n;            // bytes of a memory row, indices inside
    int off[kSwap ? 2 : 1];  // this lane's offset in its wave's even loads, and odd ones
    int piece;               // CONTIG: its first r within the stage

    // Where piece c of image row i is kept.  The 64 lanes of a read fall on
    // 16 rows (CONTIG: 16 indices at one piece; else r = 0..3, 8..11, 16..19,
    // 24..27 at two neighbouring pieces); LDS has 256 bytes of banks.
    static __device__ __forceinline__ int place_of(int c, int i)
    {
        return CONTIG ? c ^ (i / 2 % 8)
                      : W == 64 ? c ^ (i / 2 % 2 * 2 + i / 8 % 2 * 4) : c ^ (i % 4 * 2 + i / 8 % 2 * 8);
    }

    // Index 0 and r = 0 at p (PAIR: up weights at p2), `pitch_` elements a
    // memory row, n_ indices inside.
    __device__ __forceinline__ void init(const uint16_t *p, const uint16_t *p2, int pitch_, int n_)
    {
        pitch = pitch_ * 2;
        n = n_;
        const int w = threadIdx.x / kWave, lane = lane_id();
        const int i = w * kRowsLoad + lane / kPieces;
        const int c = place_of(lane % kPieces, i);
        base[0] = reinterpret_cast<const char *>(p);
        if (PAIR)
            base[PAIR] = reinterpret_cast<const char *>(p2);
        piece = c * 8;
        off[0] = i * pitch + c * 16;
        if (kSwap)
            off[kSwap] = i * pitch + place_of(lane % kPieces, i + 8) * 16;
    }

    // Starts this wave's j-th load of r0 .. r0 + kStep - 1 into `image`; the
    // image's indices start at `first`.
    __device__ __forceinline__ void fetch(MOE_LDS char *__restrict__ image, int r0, int R, int j,
                                          int first = 0) const
    {
        const int load = static_cast<int>(uniform(threadIdx.x / kWave)) + j * kTileWaves;
        MOE_LDS void *to = (MOE_LDS void *)(image + load * 1024);
        // memory rows after those of the wave's first load; PAIR: four loads
        // cover a block of 32 indices, all gate or all up
        const int rows = PAIR ? j / 2 * 32 : j * kTileWaves * kRowsLoad;
        const char *src = base[PAIR ? j % 2 : 0];
        if (CONTIG) {
            // pieces past R are outside, whatever row is added
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                row_rsrc(const_cast<char *>(src) + static_cast<int64_t>(r0) * 2, max(0, n * pitch - r0 * 2)),
                to, 16, (r0 + piece < R ? off[0] : kOutside) + (first + rows) * pitch, 0, 0, 0);
        } else {
            const int live = min(kStep, R - r0);  // <= 0 past the end: nothing is read
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                row_rsrc(const_cast<char *>(src) + static_cast<int64_t>(r0) * pitch,
                         live > 0 ? (live - 1) * pitch + n * 2 : 0),
                to, 16, off[kSwap ? j % 2 : 0] + rows * pitch + first * 2, 0, 0, 0);
        }
    }

    // The fragment of indices i0 .. i0 + 15 (i0 a multiple of 16) and r = s ..
    // s + 31: lane l gets index l%16 and r = 8 (l/16) .. + 7.
    static __device__ __forceinline__ bf16x8 frag(const MOE_LDS char *__restrict__ image, int i0, int s)
    {
        const int lane = lane_id();
        if constexpr (CONTIG) {
            const int place = lane % 16 * (kStep * 2) + place_of(s / 8 + lane / 16, lane % 16) * 16;
            return *reinterpret_cast<const MOE_LDS bf16x8 *>(image + i0 * (kStep * 2) + place);
        } else {
            // lane l of 16 points at r = l/4, indices 4 (l%4) .. of the 4 x 16
            // block it is to get column l of; i0 adds 2 pieces a block of 16
            // under the same permutation, which is the same again 4 r later
            const int r = s + lane / 16 * 8 + lane % 16 / 4, i = lane % 4 * 4;
            const int place = r * (2 * W) + place_of(i / 8, r) * 16 + i % 8 * 2;
            const MOE_LDS char *p = image + (place ^ (i0 * 2));
            const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((MOE_LDS bf16x4 *)(p));
            const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((MOE_LDS bf16x4 *)(p + 4 * 2 * W));
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
};

// Wave w has the columns' half w%2 and, of every block of 64 rows, the 32 from
// 32 (w/2), so that a short tile's rows are shared evenly.
// THIN: tiles of at most 64 rows only, in half the LDS and registers, so that
// two workgroups share a CU.
template <int COLS, bool P_CONTIG, bool Q_CONTIG, bool GATED, bool THIN = false>
struct Tile {
    static constexpr int kCols = COLS;
    static constexpr int kBlocks = THIN ? 1 : 4;  // of 64 rows
    static constexpr int kFrags = kCols / 32;   // blocks of 16 columns of a wave
    typedef Operand<kCols, P_CONTIG, GATED> P;
    typedef Operand<64, Q_CONTIG, false> Q;  // an image for each block of 64 rows
    static constexpr int kStageBytes = P::kBytes + kBlocks * Q::kBytes;
    static constexpr int kThinBytes = P::kBytes + (THIN ? 1 : 2) * Q::kBytes;  // of a stage of at most 128 rows
    // two whole stages or three thin ones; the results pass through what the
    // first stages of the next tile leave free
    static constexpr int kOutBytes = 4096, kWhole = 2 * kStageBytes + kTileWaves * kOutBytes;
    static constexpr int kLdsBytes = !THIN && kWhole > 3 * kThinBytes ? kWhole : 3 * kThinBytes;
    static_assert(kLdsBytes >= 2 * kThinBytes + kTileWaves * kOutBytes, "thin stages and results");
    __device__ __forceinline__ MOE_LDS char *out_place(MOE_LDS char *lds) const
    {
        return lds + kLdsBytes - (kTileWaves - wave()) * kOutBytes;
    }
    P p;
    Q q;
    int R;
    f32x4 acc[kFrags][kBlocks][2];
    float sum[2][2];  // SUMS: this lane's parts of the sums of Q over r, of row blocks 2 (w%2), + 1

    __device__ __forceinline__ int wave() const { return static_cast<int>(uniform(threadIdx.x / kWave)); }
    __device__ __forceinline__ int col0() const { return wave() % 2 * (kCols / 2); }
    __device__ __forceinline__ int row0(int block) const { return block * 64 + wave() / 2 * 32; }

    __device__ __forceinline__ void clear()
    {
        sum[0][0] = sum[0][1] = sum[1][0] = sum[1][1] = 0.0f;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int c = 0; c < kFrags; ++c)
                acc[c][b][0] = acc[c][b][1] = f32x4{};
    }

    // Waits until at most LEFT of this wave's loads are in flight and its LDS
    // reads are done, then for the other waves.  Nothing moves across.
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

    typedef bf16x8 Slice[2][2];  // 32 indices (two of 16), 64 r (two of 32)
    struct Frags {
        bf16x8 p[kFrags][2];
        Slice q[2];
    };
    __device__ __forceinline__ void read_p(Frags &f, int c, int s, const MOE_LDS char *__restrict__ stage) const
    {
        f.p[c][s] = P::frag(stage, col0() + c * 16, 32 * s);
    }
    __device__ __forceinline__ void read_q(Slice &q, int b, int h, int s, const MOE_LDS char *__restrict__ stage) const
    {
        q[h][s] = Q::frag(stage + P::kBytes + b * Q::kBytes, wave() / 2 * 32 + h * 16, 32 * s);
    }
    __device__ __forceinline__ void load_p(MOE_LDS char *__restrict__ stage, int r0, int j) const
    {
        p.fetch(stage, r0, R, j);
    }
    __device__ __forceinline__ void load_q(MOE_LDS char *__restrict__ stage, int r0, int b, int j) const
    {
        q.fetch(stage + P::kBytes + b * Q::kBytes, r0, R, j, 64 * b);
    }

    // Multiplies row block b, half s of the stage; after each column block's
    // products, beside(c) issues what is to run beside the next ones.
    template <typename F>
    __device__ __forceinline__ void group(const Frags &f, const Slice &q, int b, int s, F beside)
    {
#pragma unroll
        for (int c = 0; c < kFrags; ++c) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (c == 0 && h == 0)  // two wait states behind whatever vector instruction wrote an operand
                    asm("s_nop 1\nv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc[c][b][h]) : "v"(f.p[c][s]), "v"(q[h][s]));
                else
                    asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc[c][b][h]) : "v"(f.p[c][s]), "v"(q[h][s]));
            __builtin_amdgcn_sched_barrier(0);
            beside(c);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    template <bool SUMS>
    __device__ __forceinline__ void add_up(const Slice &q, int b)
    {
        if (SUMS && wave() % 2 == b / 2)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v[8];
                unpack8(__builtin_bit_cast(u32x4, q[i / 2][i % 2]), v);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    sum[b % 2][i / 2] += v[j];
            }
    }

    // The loads that a tile's first steps expect to be in flight.
    __device__ __forceinline__ void start(MOE_LDS char *lds) const
    {
#pragma unroll
        for (int j = 0; j < P::kLoads; ++j)
            load_p(lds, 0, j);
        load_pair(lds, 0, 0);
        load_pair(lds, 0, 1);
        load_pair(lds, 0, 2);
#pragma unroll
        for (int j = 0; j < P::kLoads; ++j)
            load_p(lds + kStageBytes, kStep, j);
        load_pair(lds, 0, 3);
        load_pair(lds + kStageBytes, kStep, 0);
        load_pair(lds + kStageBytes, kStep, 1);
    }
    __device__ __forceinline__ void load_pair(MOE_LDS char *__restrict__ stage, int r0, int b) const
    {
#pragma unroll
        for (int j = 0; j < Q::kLoads; ++j)
            load_q(stage, r0, b, j);
    }

    // Stage k, at offset `cur` of LDS, in four phases, one for each block of
    // 64 rows; its P and first Q block are in f.  Each phase multiplies what
    // the phase before it read, and an image is refilled (for stage k + 2, Q
    // block 3 and the end of block 2: k + 1) as soon as a join has shown that
    // every wave has read it: one to one and a half stages ahead of its use,
    // two loads for every 16 MFMAs.  Issued together the loads stall their
    // waves (8192 x 8192, r 7168: 750 us instead of 735, and with zeros, at the
    // full clock, 634 instead of 576).  `rd` and `wr` are the same LDS, apart
    // for the compiler, which would else wait for every load before a read.
    template <bool SUMS>
    __device__ __forceinline__ void step(Frags &f, const MOE_LDS char *__restrict__ rd,
                                         MOE_LDS char *__restrict__ wr, int cur, int nxt, int r0)
    {
        // loads go behind the second half of a group's columns, fragments behind
        // the first ones
        constexpr int H = kFrags / 2, NP = P::kLoads / 4;
        auto p_share = [&](int c, int i) {
            if (c >= H && (c - H) % (H / NP) == 0)
                load_p(wr + cur, r0 + 2 * kStep, i * NP + (c - H) / (H / NP));
        };
        auto q_pair = [&](int c, int to, int r, int b) {
            if (c >= H && (c - H) % (H / 2) == 0)
                load_q(wr + to, r, b, (c - H) / (H / 2));
        };
        group(f, f.q[0], 0, 0, [&](int c) { q_pair(c, nxt, r0 + kStep, 2); });
        join<P::kLoads + 8>();  // Q blocks 1 and 2 of this stage are here; all P and Q block 0 were read
        add_up<SUMS>(f.q[0], 0);
        group(f, f.q[0], 0, 1, [&](int c) {
            if (c < 4)
                read_q(f.q[1], 1, c % 2, c / 2, rd + cur);
            p_share(c, 0);
        });
        group(f, f.q[1], 1, 0, [&](int c) {
            if (c == 1 || c == 3)
                read_q(f.q[0], 2, c / 2, 0, rd + cur);
            p_share(c, 1);
        });
        add_up<SUMS>(f.q[1], 1);
        group(f, f.q[1], 1, 1, [&](int c) {
            if (c == 1 || c == 3)
                read_q(f.q[0], 2, c / 2, 1, rd + cur);
            p_share(c, 2);
        });
        group(f, f.q[0], 2, 0, [&](int c) { p_share(c, 3); });
        join<P::kLoads + 4>();  // Q block 3 of this stage, P and Q block 0 of the next are here; blocks 1 and 2 were read
        add_up<SUMS>(f.q[0], 2);
        group(f, f.q[0], 2, 1, [&](int c) {
            if (c < 4)
                read_q(f.q[1], 3, c % 2, c / 2, rd + cur);
            q_pair(c, nxt, r0 + kStep, 3);
        });
        add_up<SUMS>(f.q[1], 3);
        group(f, f.q[1], 3, 0, [&](int c) {
            if (c < 4)
                read_q(f.q[0], 0, c % 2, c / 2, rd + nxt);
            read_p(f, c, 0, rd + nxt);
            q_pair(c, cur, r0 + 2 * kStep, 0);
        });
        group(f, f.q[1], 3, 1, [&](int c) {
            read_p(f, c, 1, rd + nxt);
            q_pair(c, cur, r0 + 2 * kStep, 1);
        });
    }

    // The product of a tile whose start() is under way.  (Memory operations
    // issued since only make the joins wait for more than they need.)
    template <bool SUMS>
    __device__ __forceinline__ void run(MOE_LDS char *lds)
    {
        int cur = 0, nxt = kStageBytes;
        Frags f;
        join<P::kLoads + 10>();  // P and Q block 0 of the first stage
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            read_q(f.q[0], 0, 0, s, lds);
            read_q(f.q[0], 0, 1, s, lds);
#pragma unroll
            for (int c = 0; c < kFrags; ++c)
                read_p(f, c, s, lds);
        }
#pragma unroll 1
        for (int r0 = 0; r0 < R; r0 += kStep) {
            step<SUMS>(f, lds, lds, cur, nxt, r0);
            const int t = cur;
            cur = nxt;
            nxt = t;
        }
        settle();
    }

    // A tile of at most NB blocks of 64 rows: three stages, whole stages in
    // flight.
    __device__ __forceinline__ void load_thin(MOE_LDS char *__restrict__ stage, int r0, int nb) const
    {
#pragma unroll
        for (int j = 0; j < P::kLoads; ++j)
            load_p(stage, r0, j);
#pragma unroll
        for (int b = 0; b < 2; ++b)
            if (b < nb)
                load_pair(stage, r0, b);
    }
    __device__ __forceinline__ void start_thin(MOE_LDS char *lds, int nb) const
    {
        load_thin(lds, 0, nb);
        load_thin(lds + kThinBytes, kStep, nb);
    }
    // Stage k at offset `cur`; its first half's fragments are in f.  The second
    // half's are read, and stage k + 2 is loaded over k - 1, beside the first
    // half's products; the next stage's first half beside the second's.
    template <int NB, bool SUMS>
    __device__ __forceinline__ void step_thin(Frags &f, const MOE_LDS char *__restrict__ rd,
                                              MOE_LDS char *__restrict__ wr, int cur, int nxt, int into, int r0)
    {
        constexpr int NP = P::kLoads, NL = NP + NB * Q::kLoads;  // loads of a stage
        constexpr int NG = NB * kFrags;                          // places beside products
#pragma unroll
        for (int b = 0; b < NB; ++b)
            group(f, f.q[b], b, 0, [&](int c) {
                const int at = b * kFrags + c;
                if (at < kFrags)
                    read_p(f, at, 1, rd + cur);
                if (at < 2 * NB)
                    read_q(f.q[at / 2], at / 2, at % 2, 1, rd + cur);
#pragma unroll
                for (int i = at * NL / NG; i < (at + 1) * NL / NG; ++i)
                    if (i < NP)
                        load_p(wr + into, r0 + 2 * kStep, i);
                    else
                        load_q(wr + into, r0 + 2 * kStep, (i - NP) / Q::kLoads, (i - NP) % Q::kLoads);
            });
        join<NL>();  // the next stage is here; this one was read
#pragma unroll
        for (int b = 0; b < NB; ++b)
            add_up<SUMS>(f.q[b], b);
#pragma unroll
        for (int b = 0; b < NB; ++b)
            group(f, f.q[b], b, 1, [&](int c) {
                const int at = b * kFrags + c;
                if (at < kFrags)
                    read_p(f, at, 0, rd + nxt);
                if (at < 2 * NB)
                    read_q(f.q[at / 2], at / 2, at % 2, 0, rd + nxt);
            });
    }
    template <int NB, bool SUMS>
    __device__ __forceinline__ void run_thin(MOE_LDS char *lds)
    {
        int cur = 0, nxt = kThinBytes, into = 2 * kThinBytes;
        Frags f;
        join<P::kLoads + NB * Q::kLoads>();  // the first stage
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i)
            read_q(f.q[i / 2], i / 2, i % 2, 0, lds);
#pragma unroll
        for (int c = 0; c < kFrags; ++c)
            read_p(f, c, 0, lds);
#pragma unroll 1
        for (int r0 = 0; r0 < R; r0 += kStep) {
            step_thin<NB, SUMS>(f, lds, lds, cur, nxt, into, r0);
            const int t = cur;
            cur = nxt;
            nxt = into;
            into = t;
        }
        settle();
    }

    // The same for a tile of `rows` rows (start_rows: its first loads).
    __device__ __forceinline__ void start_rows(int rows, MOE_LDS char *lds) const
    {
        if (THIN || rows <= 64)
            start_thin(lds, 1);
        else if (rows <= 128)
            start_thin(lds, 2);
        else
            start(lds);
    }
    template <bool SUMS>
    __device__ __forceinline__ void run_rows(int rows, MOE_LDS char *lds)
    {
        if constexpr (THIN) {
            run_thin<1, SUMS>(lds);
        } else {
            if (rows > 128)
                run<SUMS>(lds);
            else if (rows > 64)
                run_thin<2, SUMS>(lds);
            else
                run_thin<1, SUMS>(lds);
        }
    }

    // The last products written, all loads and reads done, in all waves.
    static __device__ __forceinline__ void settle()
    {
        asm volatile("s_nop 15\ns_nop 15" ::: "memory");  // MFMA results, before they are read
        join<0>();
    }

    // (written out, so that the accumulators stay in the AGPRs up to here)
    static __device__ __forceinline__ f32x4 read_acc(const f32x4 &a)
    {
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x;
            asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(x) : "a"(a[i]));
            v[i] = x;
        }
        return v;
    }

    // Calls f(row, v) for each 16 of this wave's rows of the tile, from `row`
    // on: v[c] has of row + lane%16 the columns col0() + 16 c + 4 (lane/16) ..
    // + 3.  Rows from `rows` on may be among them.  The accumulators are picked
    // by a switch, so that the code behind them is there once.
    template <typename F>
    __device__ __forceinline__ void finish(int rows, F &f) const
    {
#pragma unroll 1
        for (int i = 0; i < 2 * kBlocks && row0(i / 2) + i % 2 * 16 < rows; ++i) {
            f32x4 v[kFrags];
#define MOE_PICK(I)                                                                            \
    case I:                                                                                    \
        _Pragma("unroll") for (int c = 0; c < kFrags; ++c) v[c] = read_acc(acc[c][I / 2][I % 2]); \
        break
            switch (i) {
                MOE_PICK(0);
                MOE_PICK(1);
                MOE_PICK(2);
                MOE_PICK(3);
                MOE_PICK(4);
                MOE_PICK(5);
                MOE_PICK(6);
                MOE_PICK(7);
            }
#undef MOE_PICK
            // (past the last rows the next ones are again these: loads ahead of them are not used)
            const int next = min(i + 1, 2 * kBlocks - 1);
            f(row0(i / 2) + i % 2 * 16, row0(next / 2) + next % 2 * 16, v);
        }
    }
};

}  // namespace moe
