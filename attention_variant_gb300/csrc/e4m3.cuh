// e4m3.cuh -- values to e4m3 codes and back, and the scales that codes take.
#pragma once

#include <cuda_fp16.h>
#include <cstdint>

namespace fl {
namespace {

constexpr uint32_t kLeastScale = (127u - 100u) << 23; // 2^-100

// The smallest power of two, from 2^-100 on, 448 times which is at least a; both as
// bits of a float.
__device__ __forceinline__ uint32_t scale_bits(uint32_t a)
{
    const uint32_t e = (a + 0x1fffffu) >> 23; // 448 = 1.75 * 2^8
    return e > (kLeastScale >> 23) + 8u ? (e - 8u) << 23 : kLeastScale;
}

// Two values to codes, the first in the low byte (past 448: 448; NaN stays NaN).
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two codes (the low bytes of c) to values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
    return h;
}
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t c, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c)
{
    const uint32_t h = e4m3x2_to_f16x2(c);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// A code's value times a scale (up to 28 bits) in 24, rounded to odd: rounded again to
// fewer, it comes out as if rounded once.
__device__ __forceinline__ float times_to_odd(float c, float s)
{
    const float p = __fmul_rz(c, s);
    return fmaf(c, s, -p) == 0.f ? p : __uint_as_float(__float_as_uint(p) | 1u);
}

} // namespace
} // namespace fl
