// E4M3 codes with one fp32 scale for a block of values: scale = max|v| / 448,
// code = E4M3(v / scale), the payload's rule (a block of zeros: scale 0, codes
// 0).  The largest size is taken over the values' bits, where a NaN is above an
// infinity: a block that holds either gets it as its scale, and whoever
// multiplies by that reads NaN.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace moe {

__device__ __forceinline__ uint32_t size_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Largest of a 16-lane row, in every lane of it.
__device__ __forceinline__ uint32_t row_umax(uint32_t v)
{
    v = umax(v, dpp32<0xB1>(v));
    v = umax(v, dpp32<0x4E>(v));
    v = umax(v, dpp32<0x141>(v));
    return umax(v, dpp32<0x140>(v));
}

// A subnormal scale is rounded up, so that no quotient is above 448 by more than
// its last bit (the conversion makes NaN of what rounds past 448).
__device__ __forceinline__ float scale_of(uint32_t top)
{
    const float s = __uint_as_float(top) / 448.0f;
    return __float_as_uint(s) < 0x00800000u && top ? __uint_as_float(__float_as_uint(s) + 1u) : s;
}

// Codes of values over one scale.  The quotients come from the scale's reciprocal
// with one step of correction, q + (v - q s) / s, which is the correctly rounded
// quotient but where v - q s is subnormal: three instructions a value where the
// division takes ten (which cost 13 us a tile of the products' gradients).  Where a
// wave has a scale whose reciprocal might not be finite, it divides.
struct Coder {
    float scale, inverse;
    bool divide;  // in any lane of the wave
    __device__ __forceinline__ explicit Coder(float s) : scale(s), inverse(1.0f / s), divide(__any(s < 1e-37f)) {}

    __device__ __forceinline__ float over(float v) const
    {
        const float q = v * inverse;
        return fmaf(fmaf(-q, scale, v), inverse, q);
    }
    // Four codes, the first in the lowest byte.
    __device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) const
    {
        if (__builtin_expect(divide, false)) {
            const uint32_t w = pack(a / scale, b / scale, c / scale, d / scale);
            return scale == 0.0f ? 0u : w;
        }
        return pack(over(a), over(b), over(c), over(d));
    }
    __device__ __forceinline__ u32x2 codes8(const float (&f)[8]) const
    {
        return u32x2{codes4(f[0], f[1], f[2], f[3]), codes4(f[4], f[5], f[6], f[7])};
    }
    static __device__ __forceinline__ uint32_t pack(float a, float b, float c, float d)
    {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
        return static_cast<uint32_t>(w);
    }
};

}  // namespace moe
