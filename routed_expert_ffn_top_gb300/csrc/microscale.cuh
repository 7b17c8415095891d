// microscale.cuh -- the 4-bit block format's arithmetic (microscale.cu describes it).
#pragma once

#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {

// Scale byte of a block from the bits of its largest magnitude: the exponent field less 2,
// at least 0 (2^-127); 255 (a NaN block) when the block holds an infinity or a NaN.
__device__ __forceinline__ uint32_t microscale_byte(uint32_t top) {
    const uint32_t e = top >> 23;
    return e == 255u ? 255u : (e <= 2u ? 0u : e - 2u);
}

// 2^-X of a scale byte below 253 (the largest a finite block has is 252); 1 for 255.
__device__ __forceinline__ float microscale_inverse(uint32_t byte) {
    return byte == 255u ? 1.0f : __uint_as_float((254u - byte) << 23);
}

// 2^X of a scale byte.
__device__ __forceinline__ float microscale_value(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7fffffffu : (byte == 0u ? 0x00400000u : byte << 23));
}

// Eight floats to eight codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t fp4x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// One float to its code.
__device__ __forceinline__ uint32_t fp4(float v) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\t"
        "cvt.u32.u8 %0, b;\n\t}"
        : "=r"(r)
        : "f"(v), "f"(0.0f));
    return r;
}

}  // namespace moe
