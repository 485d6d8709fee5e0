// The 8-bit cache's number format: e4m3 values with one power-of-two scale per row.
//
// A row is one token's D keys (or values) of one kv head.  With a the row's largest
// magnitude (before the rotation, for keys),
//     e = max(floor(log2 a) - 7, -64)   (0 for a row of zeros),   held = e4m3(x * 2^-e),
// kept as the byte e + 127.  |x * 2^-e| < 2^8 for the row itself and < 2^8.5 = 362 after
// a rotation (a pair's larger member grows by at most sqrt 2), below e4m3's 448: a
// row does not saturate (up to 1.9375 * 2^127, where the value itself leaves fp32's range).  The scale is a power of two, so a held value has four significant
// bits and is exact in bf16 and fp16, and the scale follows from the bf16 input bits
// alone: two kernels (or a kernel and a reference) cannot disagree about it.  e4m3 floats, so
// a scale that is not the tightest one loses no precision in its normal range, 2^-6..448
// (values below 2^-14 of the row's largest are held with fewer bits).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rlt {

constexpr int kExpBias = 127;
constexpr int kExpFloor = -64;

// The biased scale exponent of a row whose largest magnitude has these bf16 bits (sign
// dropped); infinities and NaN count as 2^128.
__host__ __device__ __forceinline__ int row_exponent(uint32_t amax_bits)
{
    const int e = (int)(amax_bits >> 7) - 127 - 7;
    return amax_bits == 0u ? kExpBias : (e < kExpFloor ? kExpFloor : e) + kExpBias;
}

// 2^(byte - 127) and its inverse, for bytes row_exponent makes (63..248).
__device__ __forceinline__ float exp_scale(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float exp_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Two fp32 values to e4m3, nearest even, past 448 clamped: lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 values (the low 16 bits of w) to fp16, exactly.
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t w)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
    return r;
}

__device__ __forceinline__ float2 f32x2_of_f16(uint32_t h)
{
    float lo, hi;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
    return make_float2(lo, hi);
}

}  // namespace rlt
