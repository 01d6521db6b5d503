// Warp-wide matrix products of two-byte operands with binary32 sums, and the
// conversions that feed them.
#pragma once

#include <stdint.h>

#include "ar_device.cuh"

namespace ar {

// d (16 x 8) += a (16 x 16) * b (16 x 8).  A lane holds of a: rows lane / 4 and
// that + 8, columns 2 * (lane % 4) + {0, 1} (words 0, 1) and 8 more (words 2, 3);
// of b: the same rows of k in column lane / 4; of d: rows lane / 4 (0, 1) and that
// + 8 (2, 3), columns 2 * (lane % 4) + {0, 1}.
template <int DT>
__device__ __forceinline__ void mma16(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    if (DT == AR_BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four E4M3 codes to binary16, exactly: elements 0, 1 and 2, 3.
__device__ __forceinline__ void from_e4m3x4(uint32_t q, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(q));
}

// Two binary32 values to a word of two binary16 numbers, a in the low half.
__device__ __forceinline__ uint32_t half2_of(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// What is left of a and b once half2_of(a, b) is taken away; an infinity leaves nothing.
__device__ __forceinline__ uint32_t rest_of(uint32_t taken, float a, float b) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&taken));
    return half2_of(isinf(f.x) ? 0.0f : a - f.x, isinf(f.y) ? 0.0f : b - f.y);
}

// The power of two that brings magnitudes up to `top` below 2^15, and its inverse
// (both exact; infinities and NaN stay what they are).
__device__ __forceinline__ void half_range(float top, float &scale, float &inverse) {
    const uint32_t e = __float_as_uint(top) >> 23;           // top >= 0
    const uint32_t up = e < 14u ? 254u : 268u - e;           // biased exponent of the scale
    scale = __uint_as_float(up << 23);
    inverse = up == 254u ? 0x1p-127f : __uint_as_float((254u - up) << 23);
}

}  // namespace ar
