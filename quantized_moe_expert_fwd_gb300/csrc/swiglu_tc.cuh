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

// BF16: the operands' type, or fp16.
template <bool BF16>
struct SwigluPiece {
    SwigluKeep k;
    int vec_h, vec_p;                        // bytes that every row is aligned to: 32, 16, 0
    static constexpr uint32_t kWarpStaging = kGtStoreWords * 4;
    // reads nothing
    __device__ __forceinline__ int ahead(size_t, int, int, int, uint32_t*) const { return 0; }
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

// The gradient reads as much as it writes, 10 bytes a column and row.  A lane a
// row, 32 bytes at a time, both took two shared-memory cycles a lane and access
// and bound the kernel (8192 rows, 2048 to 4096 columns: 125 us, now 112, against
// 72 of the plain product, which moves a fifth of the bytes).  So 32 columns of
// the warp's 32 rows go through its staging, 128 bytes a row: p comes there by
// asynchronous copies of neighbouring 16 bytes, the next columns' while these
// are worked on; a lane reads its row's and leaves dp in its place; and 8 lanes
// store a row's line.  h follows the same way.  16-byte pieces are spread over
// the banks by the row.  (Of the 112: stores 28, reads 12, arithmetic 3; dp by
// TMA from the same place gains 1.)
template <bool BF16>
struct SwigluBackPiece {
    SwigluBack k;
    static constexpr uint32_t kBuffer = 32 * 128, kWarpStaging = 2 * kBuffer;
    struct Ahead {
        int buf;                             // the buffer that holds the next columns
        uint32_t scales;                     // and their two scale bytes (of the lane's row)
    };
    static __device__ __forceinline__ uint32_t place(int r, int chunk) {
        return uint32_t(r) * 128 + uint32_t((chunk ^ (r & 7)) * 16);
    }
    // Starts the copies of p's columns c .. of rows row0 ..
    __device__ __forceinline__ void fetch(Ahead& a, size_t row0, int rows, int c, uint32_t* stage) const {
        const int lane = threadIdx.x & 31, n = min(32, k.I - c);
        const uint32_t to = smem_u32(stage) + a.buf * kBuffer;
        const bool small = k.scales != nullptr;              // 64 bytes a row, else 128
        const int per = small ? 4 : 8, have = small ? n / 8 : n / 4;
        const size_t pitch = size_t(2) * k.I * (small ? 1 : 2);
        const uint8_t* p = static_cast<const uint8_t*>(k.p) + row0 * pitch + size_t(c) * (small ? 2 : 4);
        const int q = lane & (per - 1);
        if (q < have)
            for (int r = lane / per; r < rows; r += 32 / per)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + place(r, q)),
                             "l"(p + r * pitch + q * 16)
                             : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (small && lane < rows) {
            const uint8_t* s = k.scales + (row0 + lane) * (2 * k.I / kAct8Block) + 2 * c / kAct8Block;
            a.scales = __ldg(s) | (n > 16 ? uint32_t(__ldg(s + 1)) << 8 : 0u);
        }
    }
    __device__ __forceinline__ Ahead ahead(size_t row0, int rows, int c0, int end, uint32_t* stage) const {
        Ahead a{};
        if (rows > 0 && c0 < end) fetch(a, row0, rows, c0, stage);
        return a;
    }
    __device__ __forceinline__ void quad(size_t row, int c, const float* v, bool live) const {
        swiglu_back_quad(k, row, c, v, live);
    }
    // `chunks` pieces of 16 bytes a row, out of a buffer into rows of `pitch` bytes.
    template <int PER>
    static __device__ __forceinline__ void put(uint8_t* out, size_t pitch, int rows, int chunks,
                                               const uint8_t* buf) {
        const int lane = threadIdx.x & 31, q = lane % PER;
        __syncwarp();
        if (q < chunks) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int r = i * (32 / PER) + lane / PER;
                if (r < rows)
                    *reinterpret_cast<uint4*>(out + r * pitch + q * 16) =
                        *reinterpret_cast<const uint4*>(buf + place(r, q));
            }
        }
        __syncwarp();
    }
    __device__ __forceinline__ void take(Ahead& a, size_t row0, int rows, int c, int end, const float* v,
                                         uint32_t* stage) const {
        const int lane = threadIdx.x & 31, nv = min(32, k.I - c);            // a multiple of 8
        if (rows <= 0 || nv <= 0) return;
        uint8_t* buf = reinterpret_cast<uint8_t*>(stage) + a.buf * kBuffer;
        const uint32_t scales = a.scales;
        a.buf ^= 1;
        if (c + 32 < end) {
            fetch(a, row0, rows, c + 32, stage);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncwarp();
        // what does not exist is worked on like the rest and not stored
        uint4 small[4];
        if (k.scales != nullptr) {
#pragma unroll
            for (int q = 0; q < 4; ++q) small[q] = *reinterpret_cast<const uint4*>(buf + place(lane, q));
        }
        uint32_t h[16];
#pragma unroll
        for (int q = 0; q < 8; ++q) {                        // four columns
            float g[4], u[4];
            if (k.scales != nullptr) {
                const float s = act8_scale((scales >> (q < 4 ? 0 : 8)) & 0xffu);
                const uint4& w = small[q / 2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float t[4];
                    act8_values(q & 1 ? (j ? w.w : w.z) : (j ? w.y : w.x), s, t);
                    g[2 * j] = t[0];
                    u[2 * j] = t[1];
                    g[2 * j + 1] = t[2];
                    u[2 * j + 1] = t[3];
                }
            } else {
                const uint4 w = *reinterpret_cast<const uint4*>(buf + place(lane, q));
                const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    g[j] = unpack16(x[j] & 0xffffu, BF16);
                    u[j] = BF16 ? bf16_hi(x[j]) : unpack16(x[j] >> 16, BF16);
                }
            }
            const SwigluGrads2 o = swiglu_grads2(g, u, v + 4 * q), p = swiglu_grads2(g + 2, u + 2, v + 4 * q + 2);
            *reinterpret_cast<uint4*>(buf + place(lane, q)) =
                make_uint4(pack16(o.dg.x, o.du.x, BF16), pack16(o.dg.y, o.du.y, BF16),
                           pack16(p.dg.x, p.du.x, BF16), pack16(p.dg.y, p.du.y, BF16));
            h[2 * q] = pack16(o.h.x, o.h.y, BF16);
            h[2 * q + 1] = pack16(p.h.x, p.h.y, BF16);
        }
        put<8>(static_cast<uint8_t*>(k.dp) + (row0 * 2 * k.I + 2 * c) * 2, size_t(4) * k.I, rows, nv / 4, buf);
        if (k.h == nullptr) return;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(buf + place(lane, q)) =
                make_uint4(h[4 * q], h[4 * q + 1], h[4 * q + 2], h[4 * q + 3]);
        put<4>(static_cast<uint8_t*>(k.h) + (row0 * k.I + c) * 2, size_t(2) * k.I, rows, nv / 8, buf);
    }
};

}  // namespace strata
