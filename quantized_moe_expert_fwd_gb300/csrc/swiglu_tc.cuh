// swiglu_tc.cuh -- the epilogues of the tensor-core kernel for SwiGLU and its
// gradient.  A lane has a row; gate and up are neighbouring columns, so
// everything stays in its registers, a block of 32 kept in 8 bits too.
#pragma once

#include "grouped_tc_kernel.cuh"
#include "swiglu.cuh"

namespace strata {

// 32 bytes of each of a warp's rows: one sector a lane where they are aligned.
__device__ __forceinline__ void put32(uint8_t* p, bool wide, const uint32_t (&w)[8]) {
    if (wide) {
        gt_st8(p, w);
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
__device__ __forceinline__ void get32(const uint8_t* p, bool wide, uint32_t (&w)[8]) {
    if (wide) {
        asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                       "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
        const uint4 b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
}

struct SwigluPiece {
    SwigluKeep k;
    int vec_h, vec_p;                        // bytes that every row is aligned to: 32, 16, 0
    template <int CH>
    __device__ __forceinline__ void ahead(size_t, bool, int) const {}
    __device__ __forceinline__ void quad(size_t row, int c, const float* v, bool live) const {
        swiglu_quad(k, row, c, v, live);
    }
    __device__ __forceinline__ void piece(size_t row0, int rows, int c, const float* v,
                                          uint32_t* stage) const {
        const int cols = 2 * k.I, nv = cols - c, lane = threadIdx.x & 31;
        if (rows <= 0 || nv <= 0) return;
        if (k.p != nullptr && k.scales == nullptr)
            gt_store<false, 32>(k.p, row0 * cols + c, cols, rows, v, nv, vec_p, k.bf16, stage);
        if (k.scales != nullptr && lane < rows) {            // whole blocks
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 32; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
            const uint32_t b = act8_byte(m);
            const float inv = act8_inverse(b);
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j] = b == 255u ? kAct8Nan : act8_codes(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3], inv);
            put32(static_cast<uint8_t*>(k.p) + (row0 + lane) * cols + c, vec_p == 32, w);
            k.scales[(row0 + lane) * (cols / kAct8Block) + c / kAct8Block] = uint8_t(b);
        }
        // rows that do not exist may hold anything: the slow paths of their
        // quotients are not taken
        float h[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) h[j] = lane < rows ? swiglu(v[2 * j], v[2 * j + 1]) : 0.0f;
        gt_store<false, 16>(k.h, row0 * k.I + c / 2, k.I, rows, h, nv / 2, vec_h, k.bf16, stage);
    }
};

struct SwigluBackPiece {
    SwigluBack k;
    int vec_p, vec_dp, vec_h;
    // The lines of p that a lane will read, into the L2 while the products run.
    template <int CH>
    __device__ __forceinline__ void ahead(size_t row, bool live, int c0) const {
        const int bytes = k.scales != nullptr ? 2 : 4;       // of a column
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (live && c0 + c * 32 < k.I)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t*>(k.p) +
                                                              (row * k.I + c0 + c * 32) * bytes));
    }
    __device__ __forceinline__ void quad(size_t row, int c, const float* v, bool live) const {
        swiglu_back_quad(k, row, c, v, live);
    }
    // Sixteen columns at a time: 32 values of p.
    __device__ __forceinline__ void piece(size_t row0, int rows, int c, const float* v,
                                          uint32_t* stage) const {
        const int lane = threadIdx.x & 31;
        if (rows <= 0) return;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int c1 = c + 16 * half, nv = k.I - c1;     // nv is a multiple of 8
            if (nv <= 0) return;
            float d[32], h[16];
            const size_t at = (row0 + lane) * 2 * k.I + 2 * c1;
            if (lane < rows) {
                if (k.scales != nullptr) {                   // whole blocks
                    uint32_t w[8];
                    get32(static_cast<const uint8_t*>(k.p) + at, vec_p == 32, w);
                    const float s = act8_scale(__ldg(k.scales + at / kAct8Block));
#pragma unroll
                    for (int j = 0; j < 8; ++j) act8_values(w[j], s, d + 4 * j);
                } else {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t w[8] = {};
                        if (8 * q < nv)
                            get32(static_cast<const uint8_t*>(k.p) + (at + 16 * q) * 2, vec_p == 32, w);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            d[16 * q + 2 * j] = unpack16(w[j] & 0xffffu, k.bf16);
                            d[16 * q + 2 * j + 1] = unpack16(w[j] >> 16, k.bf16);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const SwigluGrads g = swiglu_grads(d[2 * j], d[2 * j + 1], v[16 * half + j]);
                    d[2 * j] = g.dg;
                    d[2 * j + 1] = g.du;
                    h[j] = g.h;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) d[2 * j] = d[2 * j + 1] = h[j] = 0.0f;
            }
            gt_store<false, 32>(k.dp, row0 * 2 * k.I + 2 * c1, size_t(2) * k.I, rows, d, 2 * nv, vec_dp,
                                k.bf16, stage);
            if (k.h != nullptr)
                gt_store<false, 16>(k.h, row0 * k.I + c1, k.I, rows, h, nv, vec_h, k.bf16, stage);
        }
    }
};

}  // namespace strata
