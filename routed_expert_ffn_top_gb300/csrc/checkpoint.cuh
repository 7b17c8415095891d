// checkpoint.cuh -- the 8-bit block format's arithmetic (checkpoint.cu describes it).
#pragma once

#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {

// Pairs of floats in one register pair: one instruction for both, each rounded as by itself.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Scale byte of a block from the bits of its largest magnitude: X + 127 with X the smallest power
// with max <= Q 2^X, at least -127; 255 (a NaN block) when the block holds an infinity or a NaN.
// Q = 448 = 1.75 2^8 or 127 = 1.984375 2^6: a mantissa above Q's carries into the exponent field.
template <bool kInt8>
__device__ __forceinline__ uint32_t eight_byte(uint32_t top) {
    constexpr uint32_t carry = kInt8 ? 0x7fffffu - 0x7e0000u : 0x7fffffu - 0x600000u, less = kInt8 ? 6u : 8u;
    const uint32_t e = (top + carry) >> 23;
    return top >= 0x7f800000u ? 255u : (e <= less ? 0u : e - less);
}

// 2^-X of a finite block's scale byte (249 at most); 0 for 255, which makes finite values code 0.
__device__ __forceinline__ float eight_inverse(uint32_t byte) {
    return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// 2^X of a scale byte, a NaN for 255.
__device__ __forceinline__ float eight_scale(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7fffffffu : (byte == 0u ? 0x00400000u : byte << 23));
}

// Four values, within the codes' range, to their codes, the first in the lowest byte.
template <bool kInt8>
__device__ __forceinline__ uint32_t eight_pack(float a, float b, float c, float d) {
    if constexpr (kInt8) {
        // x + 1.5 2^23 is rounded to an integer, ties to even, whose low byte is the code
        constexpr float magic = 12582912.0f;
        const uint32_t ab = __byte_perm(__float_as_uint(a + magic), __float_as_uint(b + magic), 0x0040);
        const uint32_t cd = __byte_perm(__float_as_uint(c + magic), __float_as_uint(d + magic), 0x0040);
        return __byte_perm(ab, cd, 0x5410);
    } else {
        uint32_t r;
        asm("{\n\t.reg .b16 l, h;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
            "mov.b32 %0, {l, h};\n\t}"
            : "=r"(r)
            : "f"(a), "f"(b), "f"(c), "f"(d));
        return r;
    }
}

// Four codes to their values, before the scale (exact), as two pairs.
template <bool kInt8>
__device__ __forceinline__ void eight_unpack(uint32_t code, uint64_t &a, uint64_t &b) {
    if constexpr (kInt8) {
        // a byte with 128 added as the low mantissa bits of 2^23
        const uint32_t u = code ^ 0x80808080u;
        const uint64_t less = f2(-8388736.0f, -8388736.0f);
        a = f2_add(f2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540)), __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7541))), less);
        b = f2_add(f2(__uint_as_float(__byte_perm(u, 0x4b000000u, 0x7542)), __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7543))), less);
    } else {
        uint32_t l, h;
        asm("{\n\t.reg .b16 a, b;\n\t"
            "mov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(l), "=r"(h)
            : "r"(code));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&l));
        const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        a = f2(f.x, f.y), b = f2(g.x, g.y);
    }
}

// Sixteen values times 2^-X to codes; a NaN block's are 0.
template <bool kInt8>
__device__ __forceinline__ uint4 eight_codes(const float (&v)[16], uint32_t byte) {
    const float s = eight_inverse(byte);
    const uint64_t inv = f2(s, s);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b, c, d;
        f2_split(f2_mul(f2(v[4 * i], v[4 * i + 1]), inv), a, b);
        f2_split(f2_mul(f2(v[4 * i + 2], v[4 * i + 3]), inv), c, d);
        o[i] = eight_pack<kInt8>(a, b, c, d);
    }
    return byte == 255u ? uint4{0, 0, 0, 0} : uint4{o[0], o[1], o[2], o[3]};
}

// Sixteen codes to their values, in pairs.
template <bool kInt8>
__device__ __forceinline__ void eight_values(const uint4 &code, uint32_t byte, uint64_t (&v)[8]) {
    const float x = eight_scale(byte);
    const uint64_t s = f2(x, x);
    const uint32_t c[4] = {code.x, code.y, code.z, code.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint64_t a, b;
        eight_unpack<kInt8>(c[i], a, b);
        v[2 * i] = f2_mul(a, s), v[2 * i + 1] = f2_mul(b, s);
    }
}
template <bool kInt8>
__device__ __forceinline__ void eight_values(const uint4 &code, uint32_t byte, float (&v)[16]) {
    uint64_t w[8];
    eight_values<kInt8>(code, byte, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) f2_split(w[i], v[2 * i], v[2 * i + 1]);
}

}  // namespace moe
