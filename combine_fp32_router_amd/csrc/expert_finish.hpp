// How the results of the experts' products leave: 16 rows of a wave's columns at a
// time, as whole lines.
#pragma once

#include "expert_rows.hpp"

namespace moe {

typedef float f32x4 __attribute__((ext_vector_type(4)));
#define MOE_LDS __attribute__((address_space(3)))
constexpr int kOutside = static_cast<int>(0x80000000u);  // an offset past every descriptor

namespace {

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
    static __device__ __forceinline__ int half(int c, int lane = lane_id())
    {
        return lane % 16 * 256 + ((c * 2 + lane / 32) ^ (lane % 16)) * 16 + lane / 16 % 2 * 8;
    }
    static __device__ __forceinline__ int whole(int c, int lane = lane_id())
    {
        return lane % 16 * 256 + ((c * 4 + lane / 16) ^ (lane % 16)) * 16;
    }
    // row layout: piece lane%P of row (64 / P) j + lane/P
    template <int P>
    static __device__ __forceinline__ int piece(int j, int lane = lane_id())
    {
        const int row = 64 / P * j + lane / P;
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

}  // namespace
}  // namespace moe
