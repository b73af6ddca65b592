// Conversions between 16-bit values and e4m3 codes with power-of-two scales, of
// the paged cache's append and the activation checkpoints.
#pragma once

#include <cstdint>

#include "paged_params.h"

namespace attn {

// Four floats to four e4m3 codes (round to nearest even, beyond +-448 to
// +-448, NaN stays NaN), the first in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

__device__ __forceinline__ float2 from_e4m3x2(uint32_t w) {
    uint32_t h;
    float2 f;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

template <bool BF16>
__device__ __forceinline__ float2 widen(uint32_t w) {
    float2 f;
    if (BF16) {
        f.x = __uint_as_float(w << 16);
        f.y = __uint_as_float(w & 0xffff0000u);
    } else {
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
            : "=f"(f.x), "=f"(f.y)
            : "r"(w));
    }
    return f;
}

// The smallest 2^e >= 2^kMinScaleExp with a <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ float block_scale(float a) {
    const uint32_t bits = __float_as_uint(a);
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(e, paged::kMinScaleExp);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

}  // namespace attn
