// swiglu.cuh -- SwiGLU and its gradient in the epilogue of a grouped product.
//
// With p = W x (rows 2i of W gate, 2i + 1 up), g = p[2i], u = p[2i + 1]:
//   h = g s u,  s = 1 / (1 + e^-g)
// and, with dh the gradient by h,
//   du = dh g s,   dg = dh u (s + g s (1 - s)).
// Both are taken from e = e^-|g|, which never passes 1 (1 + e^-g leaves fp32 at
// g = -88.7): with r = 1 / (1 + e), s is r or e r, and s (1 - s) = r (e r), so
// that nothing cancels.  e is the square of 2^(-|g| / (2 ln 2)), which is normal
// where e is not.  The outputs have 16 bits: the approximate exponential (2
// steps of 2^-23, twice) and reciprocal (1 step) and the argument's rounding
// leave s within 7 + 1.2 |g| steps of 2^-23, next to roundings of 2^-9 or 2^-12.
// Two columns at a time in packed fp32 (with the fast exponential and quotient,
// column by column: 2048-token prompt of 256 experts 190 us forward and 117 back,
// so 183 and 114).
#pragma once

#include "act8.cuh"
#include "grouped.cuh"
#include "grouped.h"

namespace strata {

struct Silu2 {
    uint64_t s, st;                          // sigmoid(g) and sigmoid(g) (1 - sigmoid(g))
};
__device__ __forceinline__ Silu2 silu2(float g0, float g1) {
    constexpr float kHalfLog2e = 0.7213475204444817f;
    float h0, h1, r0, r1;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h0) : "f"(-fabsf(g0) * kHalfLog2e));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h1) : "f"(-fabsf(g1) * kHalfLog2e));
    const uint64_t e = mul2(pk(h0, h1), pk(h0, h1));
    const float2 d = upk(add2(e, pk(1.0f, 1.0f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(d.y));
    const uint64_t r = pk(r0, r1), er = mul2(e, r);
    const float2 x = upk(er);
    return Silu2{pk(g0 < 0.0f ? x.x : r0, g1 < 0.0f ? x.y : r1), mul2(r, er)};
}
// h of two columns.
__device__ __forceinline__ float2 swiglu2(float g0, float u0, float g1, float u1) {
    return upk(mul2(mul2(pk(g0, g1), silu2(g0, g1).s), pk(u0, u1)));
}
__device__ __forceinline__ float swiglu(float g, float u) { return swiglu2(g, u, g, u).x; }
struct SwigluGrads2 {
    float2 dg, du, h;
};
__device__ __forceinline__ SwigluGrads2 swiglu_grads2(const float* g, const float* u, const float* dh) {
    const Silu2 f = silu2(g[0], g[1]);
    const uint64_t gg = pk(g[0], g[1]), uu = pk(u[0], u[1]), dd = pk(dh[0], dh[1]), a = mul2(gg, f.s);
    return SwigluGrads2{upk(mul2(mul2(dd, uu), ffma2(gg, f.st, f.s))), upk(mul2(dd, a)), upk(mul2(a, uu))};
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, int bf16) {
    uint32_t r;
    if (bf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float unpack16(uint32_t half, int bf16) {
    return bf16 ? __uint_as_float(half << 16) : f16_to_f32(uint16_t(half));
}

// What the forward epilogue writes: h, and p where it is kept (in the operands'
// type, or with scales in 8 bits).
struct SwigluKeep {
    void* h;
    void* p;
    uint8_t* scales;
    int I, bf16;
};
// What the backward epilogue reads and writes.
struct SwigluBack {
    const void* p;
    const uint8_t* scales;
    void* dp;
    void* h;                                 // or NULL
    int I, bf16;
};

// On the tensor cores (g: the product's sizes and operands).
cudaError_t launch_swiglu_tc(const GmmArgs& g, const SwigluKeep& k, cudaStream_t s);
cudaError_t launch_swiglu_back_tc(const GmmArgs& g, const SwigluBack& k, cudaStream_t s);

__device__ __forceinline__ void store_u16(void* p, size_t at, uint32_t v) {
    static_cast<uint16_t*>(p)[at] = uint16_t(v);
}

// Four columns of p of one row, c (a multiple of 4) on.  Whole warps call it;
// eight neighbouring lanes hold 32 columns of one row.  live: the row exists
// (columns past the width are left out here).
__device__ __forceinline__ void swiglu_quad(const SwigluKeep& k, size_t row, int c, const float* v,
                                            bool live) {
    const int cols = 2 * k.I;
    live = live && c < cols;
    const bool both = c + 2 < cols;
    if (k.p != nullptr && k.scales != nullptr) {             // the width is a multiple of 32
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
        if (!live) m = 0;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t b = act8_byte(m);
        if (live) {
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(k.p) + row * cols + c) =
                b == 255u ? kAct8Nan : act8_codes(v[0], v[1], v[2], v[3], act8_inverse(b));
            if (c % kAct8Block == 0) k.scales[row * (cols / kAct8Block) + c / kAct8Block] = uint8_t(b);
        }
    }
    if (!live) return;
    if (k.p != nullptr && k.scales == nullptr) {
        const size_t at = row * cols + c;
        const uint32_t a = pack16(v[0], v[1], k.bf16), b = pack16(v[2], v[3], k.bf16);
        store_u16(k.p, at, a);
        store_u16(k.p, at + 1, a >> 16);
        if (both) {
            store_u16(k.p, at + 2, b);
            store_u16(k.p, at + 3, b >> 16);
        }
    }
    const float2 o = swiglu2(v[0], v[1], v[2], v[3]);
    const uint32_t h = pack16(o.x, o.y, k.bf16);
    const size_t at = row * k.I + c / 2;
    store_u16(k.h, at, h);
    if (both) store_u16(k.h, at + 1, h >> 16);
}

// Four columns of dh of one row, c (a multiple of 4) on.
__device__ __forceinline__ void swiglu_back_quad(const SwigluBack& k, size_t row, int c,
                                                 const float* v, bool live) {
    if (!live) return;
    const int n = min(4, k.I - c);
    const size_t at = row * 2 * k.I + 2 * c;
    float g[4] = {}, u[4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j >= n) break;
        if (k.scales != nullptr) {                            // I is a multiple of 16
            const uint32_t w = static_cast<const uint16_t*>(k.p)[at / 2 + j];
            float q[4];
            act8_values(w, act8_scale(k.scales[(at + 2 * j) / kAct8Block]), q);
            g[j] = q[0];
            u[j] = q[1];
        } else {
            g[j] = unpack16(static_cast<const uint16_t*>(k.p)[at + 2 * j], k.bf16);
            u[j] = unpack16(static_cast<const uint16_t*>(k.p)[at + 2 * j + 1], k.bf16);
        }
    }
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        const SwigluGrads2 d = swiglu_grads2(g + j, u + j, v + j);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (j + i >= n) break;
            const uint32_t w = pack16(i ? d.dg.y : d.dg.x, i ? d.du.y : d.du.x, k.bf16);
            store_u16(k.dp, at + 2 * (j + i), w);
            store_u16(k.dp, at + 2 * (j + i) + 1, w >> 16);
            if (k.h != nullptr) store_u16(k.h, row * k.I + c + j + i, pack16(i ? d.h.y : d.h.x, 0.0f, k.bf16));
        }
    }
}

}  // namespace strata
