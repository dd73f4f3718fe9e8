// q8.cuh -- rows of a paged cache in 8 bits: e4m3 codes and one scale byte e, elements code * 2^(e - 127).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

namespace attn {
namespace q8 {

// 2^(e - 127): a float whose exponent field is e; 0 is the subnormal 2^-127, 255 a NaN.
__device__ __forceinline__ float pow2(uint32_t e) {
    return __uint_as_float((e << 23) | (((e + 1) & 0xffu) <= 1u ? 0x400000u : 0u));
}

// The same for e from -22 to 254, where it may be one of the least subnormals.
__device__ __forceinline__ float pow2_low(int e) { return __uint_as_float(e > 0 ? (uint32_t)e << 23 : 0x400000u >> -e); }

// A factor of logits, within the normal floats (0 times it is 0, -inf times it -inf); a NaN stays one.  A query row's power of two
// and a key's meet before the sum of their products does: either alone may take it out of fp32, with logits of ordinary size.
__device__ __forceinline__ float factor(float x) {
    asm("min.NaN.f32 %0, %0, %1;\n\tmax.NaN.f32 %0, %0, %2;" : "+f"(x) : "f"(3.402823466e38f), "f"(1.17549435e-38f));
    return x;
}

// The scale byte of a row whose largest finite magnitude is m: the least e >= 0 with m <= 448 * 2^(e - 127).
// With m = 1.f * 2^(x - 127) and 448 = 1.75 * 2^8 that is x - 8, one more where 1.f > 1.75.
__device__ __forceinline__ uint32_t scale_byte(float m) {
    const uint32_t u = __float_as_uint(m);
    return (uint32_t)max((int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
}
// 2^(127 - e) for such a byte (at most 247).
__device__ __forceinline__ float inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// Codes of four floats within 448, nearest, ties to even.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// The lower and the upper two of four codes as fp16, where every code is exact.
__device__ __forceinline__ void decode4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace q8
}  // namespace attn
