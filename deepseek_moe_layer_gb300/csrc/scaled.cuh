// scaled.cuh -- device helpers of the block-scaled 8-bit path: the power-of-two scale of a
// block of 128 and the conversion to e4m3 codes.
#pragma once

#include "common.cuh"

namespace moe {

// The smallest power of two s >= 2^-126 with amax / s <= 448, and 1 / s; 1 for amax = 0.
// amax finite, >= 0.  448 = 1.75 * 2^8: the exponent field of s is amax's less 8, one more
// when amax's mantissa exceeds 1.75.
MOE_DEV void block_scale(float amax, float& s, float& inv) {
    const uint32_t u = __float_as_uint(amax);
    int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u);
    if (e < 1) e = 1;
    if (u == 0u) e = 127;
    s = __uint_as_float((uint32_t)e << 23);
    inv = __uint_as_float((uint32_t)(254 - e) << 23);
}

// Four fp32 -> four e4m3 codes, the first in the low byte; each within +-448 or NaN.
MOE_DEV uint32_t cvt_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

}  // namespace moe
