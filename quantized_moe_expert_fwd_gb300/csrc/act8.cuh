// act8.cuh -- rows kept in 8 bits, on the device: blocks of 32 consecutive
// elements of a row, each with e4m3 codes and one scale byte b, 2^(b - 127).
//
// The scale is the smallest power of two (at least 2^-126) that a block's
// largest magnitude does not exceed 448 times, so that no element saturates
// and each is off by at most half a step of e4m3: 2^-4 of itself, or 2^-10 of
// the scale.  255 marks a block that held an infinity or a NaN: all its codes
// are NaN.  Byte 0, which no block gets, reads as zeros.
#pragma once

#include "common.cuh"

namespace strata {

constexpr int kAct8Block = 32;

// The scale byte of a block whose largest magnitude has this fp32 pattern:
// 448 = 1.75 2^8, so a mantissa above 1.75 (0x600000) carries into the exponent.
__device__ __forceinline__ uint32_t act8_byte(uint32_t amax) {
    if (amax >= 0x7f800000u) return 255u;
    const int b = int((amax + 0x1fffffu) >> 23) - 8;
    return uint32_t(b > 1 ? b : 1);
}
// 2^(127 - b) and 2^(b - 127), both normal for every byte that act8_byte gives.
__device__ __forceinline__ float act8_inverse(uint32_t b) {
    return __uint_as_float((254u - b) << 23);
}
__device__ __forceinline__ float act8_scale(uint32_t b) { return __uint_as_float(b << 23); }

// Four values as codes (the first in the low byte), scaled by inv.
__device__ __forceinline__ uint32_t act8_codes(float a, float b, float c, float d, float inv) {
    uint32_t r;
    asm("{ .reg .b16 lo, hi;\n"
        "  cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
        "  cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
        "  mov.b32 %0, {lo, hi}; }"
        : "=r"(r)
        : "f"(a * inv), "f"(b * inv), "f"(c * inv), "f"(d * inv));
    return r;
}
constexpr uint32_t kAct8Nan = 0x7f7f7f7fu;

// Four codes as values (exact but where the product is below 2^-126).
__device__ __forceinline__ void act8_values(uint32_t codes, float scale, float* v) {
    uint32_t lo, hi;
    asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2;\n"
        "  cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
        : "=r"(lo), "=r"(hi)
        : "r"(codes));
    const uint64_t s = pk(scale, scale);
    const float2 a = upk(mul2(pk(f16_to_f32(uint16_t(lo)), f16_to_f32(uint16_t(lo >> 16))), s));
    const float2 b = upk(mul2(pk(f16_to_f32(uint16_t(hi)), f16_to_f32(uint16_t(hi >> 16))), s));
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
}

}  // namespace strata
