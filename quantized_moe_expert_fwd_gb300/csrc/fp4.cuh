// fp4.cuh -- the 4-bit block formats on the device.
//
// A row is cut into blocks of V consecutive elements (MX: 32, NV: 16), each
// with one scale byte: MX a power of two (ue8m0, 2^(byte - 127), 255 = NaN),
// NV an e4m3 value.  Elements are e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives), two a byte, the first in the low half.
//
// Scales lie in tiles of 512 bytes, 128 rows by 4 consecutive scales of a
// row: row r of the tile at bytes (r % 32) * 16 + (r / 32) * 4, which is the
// order the tensor cores' scale factors take in tensor memory (32 lanes by 4
// words), so a tile moves there without any shuffling.  Tiles of a row block
// follow each other along the row; a group's rows start at a block of their
// own.
#pragma once

#include "common.cuh"

namespace strata {

// Scale words of a row.
__host__ __device__ constexpr int fp4_words(int cols, int fmt) {
    return (cols + (fmt == 0 ? 127 : 63)) / (fmt == 0 ? 128 : 64);
}

// Byte offset of row `r`'s scale word `w` within a group's row block `b`.
__device__ __forceinline__ size_t fp4_scale_at(size_t block, int words, int r, int w) {
    return (block * words + w) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

__device__ __forceinline__ float ue8m0_to_f32(uint32_t b) {
    if (b == 255u) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(b == 0u ? 0x00400000u : b << 23);
}
__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
    uint32_t h2;
    asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.f16x2.e4m3x2 %0, t; }" : "=r"(h2) : "r"(b));
    return f16_to_f32(uint16_t(h2 & 0xffffu));
}
template <int FMT>
__device__ __forceinline__ float fp4_scale_f32(uint32_t b) {
    return FMT == 0 ? ue8m0_to_f32(b) : e4m3_to_f32(b);
}

// Two e2m1 (one byte) as two fp16, exactly; the first element in the low half.
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t byte) {
    uint32_t r;
    asm("{ .reg .b8 b; cvt.u8.u32 b, %1; cvt.rn.f16x2.e2m1x2 %0, b; }" : "=r"(r) : "r"(byte));
    return r;
}

}  // namespace strata
