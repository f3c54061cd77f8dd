// mx4.cuh -- 4-bit rows: e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives), two to a byte, the first in the low half, with one power-of-two
// scale per 32 channels, held as the byte exponent + 127.
//
// A block's exponent is that of its largest magnitude less 2 (so that it lands in
// [4, 8) and at most its values over 6 are cut), at least -127.  A block that
// holds an infinity or a NaN gets the scale byte 255, which stands for NaN, and
// codes 0: all of it reads back as NaN.
#pragma once

#include <stdint.h>

#include "numeric.cuh"

namespace moe {

constexpr int kMx4Block = 32;

// The scale byte of a block from the bits of its largest magnitude (as integers,
// so that a NaN is the largest of all).
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t amax_bits) {
    const int e = (int)(amax_bits >> 23);   // biased; 0 for subnormals, whose exponent is under the least
    return e == 255 ? 255u : (uint32_t)max(e - 2, 0);
}

// 2^-(byte - 127), for the quantisation: exact, as is its product with a value,
// unless that product is so small that its code is 0 anyway.  0 for byte 255.
__device__ __forceinline__ float mx4_inverse(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0u : (254u - byte) << 23);
}

// 2^(byte - 127); the least is subnormal; NaN for 255.
__device__ __forceinline__ float mx4_scale(uint32_t byte) {
    return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7fc00000u : byte << 23);
}

// Eight values times `inverse` to their codes, to the nearest, ties to the even
// code, 6 where it would be more.  inverse 0 (a block with an infinity or a NaN)
// gives codes 0.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float *v, float inverse) {
    uint32_t codes;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(codes)
        : "f"(v[0] * inverse), "f"(v[1] * inverse), "f"(v[2] * inverse), "f"(v[3] * inverse), "f"(v[4] * inverse),
          "f"(v[5] * inverse), "f"(v[6] * inverse), "f"(v[7] * inverse));
    return inverse == 0.0f ? 0u : codes;
}

// Eight codes to four pairs of half precision (exact).
__device__ __forceinline__ void unpack_e2m1x8(uint32_t codes, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

}  // namespace moe
