// fp4.cu -- the 4-bit block formats: rows quantised to e2m1 blocks with a
// scale byte each, and back to values.
#include <type_traits>

#include "fp4.cuh"
#include "grouped.cuh"
#include "grouped.h"

namespace strata {

size_t fp4_scale_bytes(int fmt, int64_t rows, int64_t cols, int64_t groups, bool ragged) {
    const int64_t blocks = ragged ? rows / 128 + (groups < rows ? groups : rows)
                                  : groups * ((rows / groups + 127) / 128);
    return size_t(blocks) * size_t(fp4_words(int(cols), fmt)) * 512;
}

namespace {

constexpr int kQThreads = 256;

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&v)[16]) {
    constexpr int n = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 16; i += n) {
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(p + i));
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 4) {
                v[i + j] = __uint_as_float(ws[j]);
            } else if constexpr (std::is_same<T, __half>::value) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&ws[j]));
                v[i + 2 * j] = f.x;
                v[i + 2 * j + 1] = f.y;
            } else {
                v[i + 2 * j] = bf16_lo(ws[j]);
                v[i + 2 * j + 1] = bf16_hi(ws[j]);
            }
        }
    }
}

// Eight values, already divided by the block's scale, as e2m1: rounded to
// nearest, ties to the even code, saturated at 6.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float* y) {
    uint32_t r;
    asm("{ .reg .b8 b0, b1, b2, b3;\n"
        "  cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        "  cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        "  cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        "  cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        "  mov.b32 %0, {b0, b1, b2, b3}; }"
        : "=r"(r)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return r;
}

// A thread quantises 16 elements of one row: an NV block, or half an MX
// block (its amax shared with the neighbour lane).  Units of a row are padded
// to a multiple of 8, so the 4 (NV) or 8 (MX) lanes that make one scale word
// are an aligned group of lanes; the padding's scales are zero.
//
// Every rounding decision is that of exact arithmetic:
//  - MX: dividing by a power of two is exact.
//  - NV scale: amax / 6 in fp32 lands on a border between two e4m3 values
//    only when it is one (a border times 6 has at most 7 bits, and floats
//    next to it stay apart after the division).
//  - NV elements of 16-bit inputs: the quotient by an e4m3 scale, if not on a
//    border between two e2m1 values, is at least 2^-11 of it away, so the
//    product with the scale's reciprocal (relative error below 2^-22) is
//    first rounded to 16 bits: that restores the exact ties and moves no
//    value across a border.
//  - NV elements of fp32 inputs: compared with the seven borders times the
//    scale, which have at most 7 bits.
template <int FMT, typename T>
__global__ void __launch_bounds__(kQThreads) k_fp4_quantize(Fp4QuantArgs a) {
    __shared__ GroupTable t;
    build_groups(t, a.offsets, a.n_groups, a.rows, 128, a.err);
    const int units = a.cols / 16, padded = (units + 7) & ~7;
    const int words = fp4_words(a.cols, FMT);
    const long long total = (long long)a.rows * padded;
    const float down = ldexpf(1.0f, -a.scale_exp);
    const T* x = static_cast<const T*>(a.x);
    for (long long i = (long long)blockIdx.x * kQThreads + threadIdx.x; i - (threadIdx.x & 31) < total;
         i += (long long)gridDim.x * kQThreads) {
        const int row = int(i / padded), u = int(i % padded);
        const int e = row < a.rows ? group_of_row(t, a.n_groups, row) : -1;
        int src = row;
        if (e >= 0 && a.perm != nullptr) {
            src = a.perm[row];
            src = src < 0 ? -1 : src / a.top_k;
        }
        // a source row out of range reads as zeros and is reported
        const bool bad = e >= 0 && (src < 0 || src >= a.x_rows);
        latch_warp(a.err, STRATA_EBADROUTE, __ballot_sync(0xffffffffu, bad));
        const bool live = e >= 0 && u < units;
        float v[16];
        if (live && !bad) {
            load16(x + size_t(src) * a.cols + u * 16, v);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0.0f;
        }
        // amax of the magnitudes as bit patterns: infinities and NaNs order
        // above every finite value, so they reach the scale
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
        if (FMT == 0) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        const bool finite = amax < 0x7f800000u;
        uint32_t sbyte;
        uint32_t q[2] = {0u, 0u};
        if (FMT == 0) {
            // floor(log2 amax) - 2, at least -127: elements of the top binade
            // reach 4 .. 6 (above 6 they saturate)
            int ex = -127;
            if (amax >= 0x00800000u) ex = max(int(amax >> 23) - 127 - 2, -127);
            sbyte = !finite ? 255u : (amax == 0u ? 0u : uint32_t(ex + 127));
            const float inv = __uint_as_float(uint32_t(127 - ex) << 23);     // 2^-ex
            if (finite && amax != 0u) {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] *= inv;
                q[0] = cvt_e2m1x8(v);
                q[1] = cvt_e2m1x8(v + 8);
            }
        } else {
            const float want = __uint_as_float(amax) * down / 6.0f;
            uint16_t s2;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s2) : "f"(0.0f), "f"(want));
            sbyte = finite ? uint32_t(s2 & 0xffu) : 0x7fu;
            const float s = e4m3_to_f32(sbyte);
            if (finite && sbyte != 0u) {
                if constexpr (sizeof(T) == 4) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float m = fabsf(v[j]) * down;
                        uint32_t code = uint32_t(m > 0.25f * s) + uint32_t(m >= 0.75f * s) +
                                        uint32_t(m > 1.25f * s) + uint32_t(m >= 1.75f * s) +
                                        uint32_t(m > 2.5f * s) + uint32_t(m >= 3.5f * s) +
                                        uint32_t(m > 5.0f * s);
                        code |= __float_as_uint(v[j]) >> 31 << 3;
                        q[j >> 3] |= code << (4 * (j & 7));
                    }
                } else {
                    const float inv = down / s;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        v[j] = __uint_as_float((__float_as_uint(v[j] * inv) + 0x80u) & 0xffffff00u);
                    q[0] = cvt_e2m1x8(v);
                    q[1] = cvt_e2m1x8(v + 8);
                }
            }
        }
        // the scale word: 4 bytes from 4 (NV) or every other of 8 (MX) lanes
        uint32_t word = 0;
        const int lane = threadIdx.x & 31, first = FMT == 0 ? lane & ~7 : lane & ~3;
        const uint32_t mine = e >= 0 && u < units ? sbyte : 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            word |= __shfl_sync(0xffffffffu, mine, first + (FMT == 0 ? 2 * k : k)) << (8 * k);
        const int w = u >> (FMT == 0 ? 3 : 2);
        if (e >= 0 && lane == first && w < words) {
            const int r = row - t.row[e];
            *reinterpret_cast<uint32_t*>(
                a.scales + fp4_scale_at(size_t(t.pre[e]) + (r >> 7), words, r, w)) = word;
        }
        if (live)
            *reinterpret_cast<uint2*>(a.q + size_t(row) * (a.cols / 2) + u * 8) =
                make_uint2(q[0], q[1]);
    }
}

template <int FMT, typename T>
__global__ void __launch_bounds__(kQThreads) k_fp4_dequantize(Fp4DequantArgs a) {
    __shared__ GroupTable t;
    build_groups(t, a.offsets, a.n_groups, a.rows, 128, a.err);
    const int units = a.cols / 16, words = fp4_words(a.cols, FMT);
    const long long total = (long long)a.rows * units;
    const float up = ldexpf(1.0f, a.scale_exp);
    T* out = static_cast<T*>(a.out);
    for (long long i = (long long)blockIdx.x * kQThreads + threadIdx.x; i < total;
         i += (long long)gridDim.x * kQThreads) {
        const int row = int(i / units), u = int(i % units);
        const int e = group_of_row(t, a.n_groups, row);
        if (e < 0) continue;
        const int r = row - t.row[e], sc = u / (FMT == 0 ? 2 : 1);
        const uint32_t sb =
            a.scales[fp4_scale_at(size_t(t.pre[e]) + (r >> 7), words, r, sc >> 2) + (sc & 3)];
        const float s = fp4_scale_f32<FMT>(sb);
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(a.q + size_t(row) * (a.cols / 2) + u * 8));
        T* o = out + size_t(row) * a.cols + u * 16;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t h2 = e2m1x2_to_f16x2(((j < 4 ? q.x : q.y) >> (8 * (j & 3))) & 0xffu);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            // value times scale is exact (6 bits); the power of two is applied
            // last, so it rounds only outside fp32's normal range
            o[2 * j] = from_f32<T>(f.x * s * up);
            o[2 * j + 1] = from_f32<T>(f.y * s * up);
        }
    }
}

int flat_grid(long long items, int threads) {
    const long long want = (items + threads - 1) / threads, most = (long long)device_info().sms * 8;
    return int(want < most ? want : most);
}

}  // namespace

cudaError_t launch_fp4_quantize(const Fp4QuantArgs& a, cudaStream_t s) {
    const int grid = flat_grid((long long)a.rows * ((a.cols / 16 + 7) & ~7), kQThreads);
    auto go = [&](auto fmt) {
        constexpr int F = decltype(fmt)::value;
        if (a.dtype == STRATA_BF16) k_fp4_quantize<F, __nv_bfloat16><<<grid, kQThreads, 0, s>>>(a);
        else if (a.dtype == STRATA_F16) k_fp4_quantize<F, __half><<<grid, kQThreads, 0, s>>>(a);
        else k_fp4_quantize<F, float><<<grid, kQThreads, 0, s>>>(a);
    };
    if (a.fmt == STRATA_FP4_MX) go(std::integral_constant<int, 0>{});
    else go(std::integral_constant<int, 1>{});
    return cudaGetLastError();
}

cudaError_t launch_fp4_dequantize(const Fp4DequantArgs& a, cudaStream_t s) {
    const int grid = flat_grid((long long)a.rows * (a.cols / 16), kQThreads);
    auto go = [&](auto fmt) {
        constexpr int F = decltype(fmt)::value;
        if (a.out_dtype == STRATA_BF16)
            k_fp4_dequantize<F, __nv_bfloat16><<<grid, kQThreads, 0, s>>>(a);
        else if (a.out_dtype == STRATA_F16) k_fp4_dequantize<F, __half><<<grid, kQThreads, 0, s>>>(a);
        else k_fp4_dequantize<F, float><<<grid, kQThreads, 0, s>>>(a);
    };
    if (a.fmt == STRATA_FP4_MX) go(std::integral_constant<int, 0>{});
    else go(std::integral_constant<int, 1>{});
    return cudaGetLastError();
}

}  // namespace strata
