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

// gt_store of values that are packed already: 2 WORDS columns (nv of them
// exist, a multiple of 8) of a warp's rows.
template <int WORDS>
__device__ __forceinline__ void put_rows(void* out, size_t at, size_t pitch, int rows, const uint32_t (&w)[WORDS],
                                         int nv, int vec, uint32_t* stage) {
    const int lane = threadIdx.x & 31;
    uint16_t* p = static_cast<uint16_t*>(out) + at;
    if (vec == 32) {
        if (lane < rows) gt_store_words(reinterpret_cast<uint8_t*>(p + lane * pitch), w, nv * 2);
        return;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < WORDS; ++j) stage[lane * 17 + j] = w[j];
    __syncwarp();
    gt_store_staged<WORDS>(reinterpret_cast<uint8_t*>(p), pitch * 2, rows, stage, nv * 2);
}

// BF16: the operands' type, or fp16.
template <bool BF16>
struct SwigluPiece {
    SwigluKeep k;
    int vec_h, vec_p;                        // bytes that every row is aligned to: 32, 16, 0
    static constexpr int kStep = 32;
    __device__ __forceinline__ int ahead(size_t, bool, int, int) const { return 0; }
    __device__ __forceinline__ void quad(size_t row, int c, const float* v, bool live) const {
        swiglu_quad(k, row, c, v, live);
    }
    __device__ __forceinline__ void take(int, size_t row0, int rows, int c, int, const float* v,
                                         uint32_t* stage) const {
        const int cols = 2 * k.I, nv = cols - c, lane = threadIdx.x & 31;
        if (rows <= 0 || nv <= 0) return;
        if (k.p != nullptr && k.scales == nullptr)
            gt_store<false, 32>(k.p, row0 * cols + c, cols, rows, v, nv, vec_p, BF16, stage);
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
        float h[16];
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            const float2 o = swiglu2(v[2 * j], v[2 * j + 1], v[2 * j + 2], v[2 * j + 3]);
            h[j] = o.x;
            h[j + 1] = o.y;
        }
        gt_store<false, 16>(k.h, row0 * k.I + c / 2, k.I, rows, h, nv / 2, vec_h, BF16, stage);
    }
};

template <bool BF16>
struct SwigluBackPiece {
    SwigluBack k;
    int vec_p, vec_dp, vec_h;
    // Sixteen columns' part of p, read while what is before it is worked on (one
    // after the other, 8192 rows of 4096 columns, a dense block: 156 us; DENSE).
    struct Ahead {
        uint32_t lo[8], hi[8];
        float scale;
    };
    __device__ __forceinline__ void read(Ahead& a, size_t row, bool live, int c) const {
        if (!live || c >= k.I) return;
        const size_t at = row * 2 * k.I + 2 * c;
        const uint8_t* p = static_cast<const uint8_t*>(k.p);
        if (k.scales != nullptr) {                           // whole blocks
            get32(p + at, vec_p == 32, a.lo);
            a.scale = act8_scale(__ldg(k.scales + at / kAct8Block));
        } else {
            get32(p + at * 2, vec_p == 32, a.lo);
            if (c + 8 < k.I) get32(p + (at + 16) * 2, vec_p == 32, a.hi);
        }
    }
    // The first of them, and the others' lines into the L2, while the products run.
    __device__ __forceinline__ Ahead ahead(size_t row, bool live, int c0, int end) const {
        Ahead a{};
        read(a, row, live, c0);
        const int bytes = k.scales != nullptr ? 2 : 4;       // of a column
        for (int c = c0; c < end; c += 128 / bytes)
            if (live)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t*>(k.p) +
                                                              (row * k.I + c) * bytes));
        return a;
    }
    __device__ __forceinline__ void quad(size_t row, int c, const float* v, bool live) const {
        swiglu_back_quad(k, row, c, v, live);
    }
    static constexpr int kStep = 16;
    __device__ __forceinline__ void take(Ahead& a, size_t row0, int rows, int c, int end, const float* v,
                                         uint32_t* stage) const {
        const int lane = threadIdx.x & 31, nv = k.I - c;     // nv is a multiple of 8
        if (rows <= 0 || nv <= 0) return;
        const Ahead now = a;
        if (c + 16 < end) read(a, row0 + lane, lane < rows, c + 16);
        float g[16], u[16];
        if (k.scales != nullptr) {
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                float q[4];
                act8_values(now.lo[j / 2], now.scale, q);
                g[j] = q[0];
                u[j] = q[1];
                g[j + 1] = q[2];
                u[j + 1] = q[3];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const uint32_t w = j < 8 ? now.lo[j & 7] : now.hi[j & 7];
                g[j] = unpack16(w & 0xffffu, BF16);
                u[j] = BF16 ? bf16_hi(w) : unpack16(w >> 16, BF16);
            }
        }
        uint32_t d[16], h[8];
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            const SwigluGrads2 o = swiglu_grads2(g + j, u + j, v + j);
            d[j] = pack16(o.dg.x, o.du.x, BF16);
            d[j + 1] = pack16(o.dg.y, o.du.y, BF16);
            h[j / 2] = pack16(o.h.x, o.h.y, BF16);
        }
        put_rows<16>(k.dp, row0 * 2 * k.I + 2 * c, size_t(2) * k.I, rows, d, 2 * nv, vec_dp, stage);
        if (k.h != nullptr) put_rows<8>(k.h, row0 * k.I + c, k.I, rows, h, nv, vec_h, stage);
    }
};

}  // namespace strata
