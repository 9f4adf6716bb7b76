// The tiles of a product over the experts' runs, as lists for its workgroups.
#pragma once

#include "expert_rows.hpp"
#include "launch.hpp"

namespace moe {

constexpr int kStep = 64;  // r of a stage of bf16 operands
enum Op { kForward, kDx, kDw };

namespace {

constexpr float kCutAbove = 1.7f;  // (TileList)

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
template <Op OP, int COLS, typename Args>
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
        if constexpr (OP == kDw) {
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
            if constexpr (OP == kDw) {
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

}  // namespace
}  // namespace moe
