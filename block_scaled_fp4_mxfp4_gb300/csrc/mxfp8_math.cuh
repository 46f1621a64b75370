// MXFP8 encoding shared by the kernels that write it: E4M3 values with one
// E8M0 scale per 32. Header: device-side only.
#pragma once

#include <stdint.h>

namespace mxfp4 {

// E8M0 byte of a block whose largest magnitude has fp32 bits `amax_bits` (sign
// cleared): the smallest e >= -127 with amax <= 448 * 2^e = 1.75 * 2^(8 + e). For
// amax = 1.m * 2^(E - 127) that is e = E - 135, one more where 1.m > 1.75. A
// power of two at which the block's maximum lands in (224, 448] leaves nothing
// to saturate, and a maximum at the border between two scales is exact on
// either side of it. Infinities and NaN give 0xFF.
__device__ __forceinline__ uint32_t mxfp8_scale_byte(uint32_t amax_bits)
{
    const uint32_t E = amax_bits >> 23;
    if (E == 255) return 255;
    const uint32_t b = E + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
    return b > 8 ? b - 8 : 0;
}

// 2^-e of a scale byte b = e + 127 (exact; b <= 247 for finite blocks).
__device__ __forceinline__ float mxfp8_scale_inverse(uint32_t b)
{
    return __uint_as_float((254u - (b < 254u ? b : 253u)) << 23);
}

// E4M3 bytes of four values, the first in the low byte (ties to even).
__device__ __forceinline__ uint32_t e4m3x4_rn(float x0, float x1, float x2, float x3)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
    return r;
}

}  // namespace mxfp4
