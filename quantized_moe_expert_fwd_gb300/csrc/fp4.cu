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

// Where row `r` lies: its group's rows [first, end) and first row block, or
// first = -1 for a row of no group (end = the next row that may have one).
// Computed by a whole warp straight from the offsets: a warp works on
// consecutive rows, so it looks a group up about once, and no table has to be
// built by the CTA before the first row is read.
struct RowGroup {
    int first, end, block;
};
__device__ __forceinline__ RowGroup row_group(const int32_t* offsets, int E, int rows, int r,
                                              uint32_t* err) {
    if (offsets == nullptr) {
        const int n = rows / E, e = r / n;
        return RowGroup{e * n, (e + 1) * n, e * ((n + 127) / 128)};
    }
    int block = 0, first = -1, end = -1;
    bool bad = false;
    for (int e = int(threadIdx.x & 31); e < E; e += 32) {
        const int a = __ldg(offsets + e), b = __ldg(offsets + e + 1);
        bad |= a < 0 || b < a || b > rows;
        if (b <= r) {
            block += (b - a + 127) / 128;
        } else if (a <= r) {
            first = a;
            end = b;
        }
    }
    if (__any_sync(0xffffffffu, bad)) {
        if ((threadIdx.x & 31) == 0) latch(err, STRATA_EBADROUTE);
        return RowGroup{-1, rows, 0};
    }
    block = __reduce_add_sync(0xffffffffu, block);
    first = __reduce_max_sync(0xffffffffu, first);
    end = __reduce_max_sync(0xffffffffu, end);
    if (first < 0) {
        const int o0 = __ldg(offsets);
        return RowGroup{-1, r < o0 ? o0 : rows, 0};
    }
    return RowGroup{first, end, block};
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

// The sixteen elements at p as raw words (8 of a 16-bit type, 16 of fp32).
template <typename T>
struct Raw16 {
    uint32_t w[sizeof(T) * 4];
};
template <typename T>
__device__ __forceinline__ Raw16<T> load_raw(const T* p) {
    Raw16<T> r;
#pragma unroll
    for (int i = 0; i < int(sizeof(T)); ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
        r.w[4 * i] = v.x;
        r.w[4 * i + 1] = v.y;
        r.w[4 * i + 2] = v.z;
        r.w[4 * i + 3] = v.w;
    }
    return r;
}
// Their largest magnitude as an fp32 bit pattern: magnitudes order like
// integers, infinities and NaNs above every finite value.
template <typename T>
__device__ __forceinline__ uint32_t raw_amax(const Raw16<T>& r) {
    uint32_t m = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 16; ++i) m = max(m, r.w[i] & 0x7fffffffu);
        return m;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __vmaxu2(m, r.w[i] & 0x7fff7fffu);
        m = max(m & 0xffffu, m >> 16);
        if constexpr (std::is_same<T, __half>::value)
            return __float_as_uint(f16_to_f32(uint16_t(m)));
        else
            return m << 16;
    }
}
template <typename T>
__device__ __forceinline__ void raw_f32(const Raw16<T>& r, float (&v)[16]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        if constexpr (sizeof(T) == 4) v[j] = __uint_as_float(r.w[j]);
        else if constexpr (std::is_same<T, __half>::value)
            v[j] = f16_to_f32(uint16_t(r.w[j >> 1] >> (16 * (j & 1))));
        else v[j] = (j & 1) ? bf16_hi(r.w[j >> 1]) : bf16_lo(r.w[j >> 1]);
    }
}

// Sixteen elements to their codes and scale byte: an NV block, or half an MX
// block (amax: the whole block's).
//
// Every rounding decision is that of exact arithmetic:
//  - MX: dividing by a power of two is exact.
//  - NV scale: amax / 6 in fp32 lands on a border between two e4m3 values
//    only when it is one (a border times 6 has at most 7 bits, and floats
//    next to it stay apart after the division).
//  - NV elements of 16-bit inputs: the quotient x / s is either a border t
//    between two e2m1 values or at least 2^-11 of it away, and x times the
//    reciprocal of s rounded up, rounded toward zero, is exactly t in the
//    first case (all 8 mantissas of s by all 7 borders) and within 2^-22 of
//    the quotient in the second.
//  - NV elements of fp32 inputs can be closer: they are compared with the
//    seven borders times s, which have at most 7 bits.
template <int FMT, typename T>
__device__ __forceinline__ uint32_t quantize16(const Raw16<T>& raw, uint32_t amax, float down,
                                               uint2& q) {
    const bool finite = amax < 0x7f800000u;
    q = make_uint2(0u, 0u);
    float v[16];
    if (FMT == 0) {
        // floor(log2 amax) - 2, at least -127: elements of the top binade
        // reach 4 .. 6 (above 6 they saturate)
        const int ex = max(int(amax >> 23) - 129, -127);
        const float inv = __uint_as_float(uint32_t(127 - ex) << 23);         // 2^-ex
        if (!finite) return 255u;
        if (amax == 0u) return 0u;
        raw_f32(raw, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= inv;
        q = make_uint2(cvt_e2m1x8(v), cvt_e2m1x8(v + 8));
        return uint32_t(ex + 127);
    }
    const float want = __uint_as_float(amax) * down / 6.0f;
    uint16_t s2;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s2) : "f"(0.0f), "f"(want));
    const uint32_t sbyte = uint32_t(s2 & 0xffu);
    if (!finite) return 0x7fu;
    if (sbyte == 0u) return 0u;
    const float s = e4m3_to_f32(sbyte);
    raw_f32(raw, v);
    if constexpr (sizeof(T) == 4) {
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float m = fabsf(v[j]) * down;
            uint32_t code = uint32_t(m > 0.25f * s) + uint32_t(m >= 0.75f * s) +
                            uint32_t(m > 1.25f * s) + uint32_t(m >= 1.75f * s) +
                            uint32_t(m > 2.5f * s) + uint32_t(m >= 3.5f * s) +
                            uint32_t(m > 5.0f * s);
            code |= __float_as_uint(v[j]) >> 31 << 3;
            w[j >> 3] |= code << (4 * (j & 7));
        }
        q = make_uint2(w[0], w[1]);
    } else {
        const float inv = __fdiv_ru(down, s);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __fmul_rz(v[j], inv);
        q = make_uint2(cvt_e2m1x8(v), cvt_e2m1x8(v + 8));
    }
    return sbyte;
}

// A warp works through consecutive rows, a lane 16 elements (a unit) at a
// time: 512 columns of a row a step, gridDim.y steps side by side.  The 4
// (NV) or 8 (MX) lanes of a scale word write it as one; units past the row's
// end contribute the zeros of its last word.
//
// Bound by instructions: about 100 a unit, near 4 for each two elements;
// memory moves 2.6 bytes an element.
template <int FMT, typename T>
__global__ void __launch_bounds__(kQThreads) k_fp4_quantize(Fp4QuantArgs a, int rows_per_warp) {
    pdl_launch();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int units = a.cols / 16, words = fp4_words(a.cols, FMT);
    const float down = ldexpf(1.0f, -a.scale_exp);
    const T* x = static_cast<const T*>(a.x);
    int row = int(blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5)) * rows_per_warp;
    const int last = min(row + rows_per_warp, a.rows);
    RowGroup g{-1, -1, 0};
    while (row < last) {
        if (row >= g.end) g = row_group(a.offsets, a.n_groups, a.rows, row, a.err);
        if (g.first < 0) {
            row = g.end;
            continue;
        }
        int src = row;
        if (a.perm != nullptr) {
            const int p = __ldg(a.perm + row);
            src = p < 0 ? -1 : p / a.top_k;
        }
        // a source row out of range reads as zeros and is reported
        const bool bad = src < 0 || src >= a.x_rows;
        if (bad && lane == 0) latch(a.err, STRATA_EBADROUTE);
        const int r = row - g.first;
        const size_t block = size_t(g.block) + (r >> 7);
        for (int u = int(blockIdx.y) * 32 + lane; u - lane < units; u += 32 * int(gridDim.y)) {
            const bool live = u < units;
            Raw16<T> raw = {};
            if (live && !bad) raw = load_raw(x + size_t(src) * a.cols + u * 16);
            uint32_t amax = raw_amax(raw);
            if (FMT == 0) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            uint2 q;
            uint32_t word = quantize16<FMT>(raw, amax, down, q);
            // gather the word's 4 bytes: two exchanges among its lanes
            if (FMT == 0) {
                word |= __shfl_down_sync(0xffffffffu, word, 2) << 8;
                word |= __shfl_down_sync(0xffffffffu, word, 4) << 16;
            } else {
                word |= __shfl_down_sync(0xffffffffu, word, 1) << 8;
                word |= __shfl_down_sync(0xffffffffu, word, 2) << 16;
            }
            const int w = u >> (FMT == 0 ? 3 : 2);
            if ((lane & (FMT == 0 ? 7 : 3)) == 0 && w < words)
                *reinterpret_cast<uint32_t*>(a.scales + fp4_scale_at(block, words, r, w)) = word;
            if (live)
                *reinterpret_cast<uint2*>(a.q + size_t(row) * (a.cols / 2) + u * 8) = q;
        }
        ++row;
    }
}

template <int FMT, typename T>
__global__ void __launch_bounds__(kQThreads) k_fp4_dequantize(Fp4DequantArgs a, int rows_per_warp) {
    pdl_launch();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int units = a.cols / 16, words = fp4_words(a.cols, FMT);
    const float up = ldexpf(1.0f, a.scale_exp);
    T* out = static_cast<T*>(a.out);
    int row = int(blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5)) * rows_per_warp;
    const int last = min(row + rows_per_warp, a.rows);
    RowGroup g{-1, -1, 0};
    while (row < last) {
        if (row >= g.end) g = row_group(a.offsets, a.n_groups, a.rows, row, a.err);
        if (g.first < 0) {
            row = g.end;
            continue;
        }
        const int r = row - g.first;
        const size_t block = size_t(g.block) + (r >> 7);
        for (int u = int(blockIdx.y) * 32 + lane; u < units; u += 32 * int(gridDim.y)) {
            const int sc = FMT == 0 ? u >> 1 : u;
            const float s = fp4_scale_f32<FMT>(
                __ldg(a.scales + fp4_scale_at(block, words, r, sc >> 2) + (sc & 3)));
            const uint2 q =
                __ldg(reinterpret_cast<const uint2*>(a.q + size_t(row) * (a.cols / 2) + u * 8));
            uint32_t w[sizeof(T) * 4];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t h2 = e2m1x2_to_f16x2(((j < 4 ? q.x : q.y) >> (8 * (j & 3))) & 0xffu);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                // value times scale is exact (6 bits); the power of two is
                // applied last, so it rounds only outside fp32's normal range
                const float v0 = f.x * s * up, v1 = f.y * s * up;
                if constexpr (sizeof(T) == 4) {
                    w[2 * j] = __float_as_uint(v0);
                    w[2 * j + 1] = __float_as_uint(v1);
                } else if constexpr (std::is_same<T, __half>::value) {
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v1), "f"(v0));
                } else {
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v1), "f"(v0));
                }
            }
            uint4* o = reinterpret_cast<uint4*>(out + size_t(row) * a.cols + u * 16);
#pragma unroll
            for (int j = 0; j < int(sizeof(T)); ++j)
                o[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        }
        ++row;
    }
}

// Rows in runs over all the warps the GPU holds; with fewer rows than that, a
// row's 512-column steps go to warps of their own.
struct RowGrid {
    dim3 grid;
    int rows_per_warp;
};
RowGrid row_grid(int rows, int units) {
    const int warps = device_info().sms * 64, per_cta = kQThreads / 32;
    RowGrid g;
    g.rows_per_warp = (rows + warps - 1) / warps;
    const int runs = (rows + g.rows_per_warp - 1) / g.rows_per_warp;
    const int steps = (units + 31) / 32, room = warps / runs;
    g.grid = dim3((runs + per_cta - 1) / per_cta, steps < room ? steps : (room > 0 ? room : 1));
    return g;
}

template <typename... P, typename... A>
cudaError_t launch_rows(void (*kernel)(P...), dim3 grid, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kQThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int FMT>
cudaError_t quantize(const Fp4QuantArgs& a, cudaStream_t s) {
    const RowGrid g = row_grid(a.rows, a.cols / 16);
    if (a.dtype == STRATA_BF16)
        return launch_rows(k_fp4_quantize<FMT, __nv_bfloat16>, g.grid, s, a, g.rows_per_warp);
    if (a.dtype == STRATA_F16)
        return launch_rows(k_fp4_quantize<FMT, __half>, g.grid, s, a, g.rows_per_warp);
    return launch_rows(k_fp4_quantize<FMT, float>, g.grid, s, a, g.rows_per_warp);
}

template <int FMT>
cudaError_t dequantize(const Fp4DequantArgs& a, cudaStream_t s) {
    const RowGrid g = row_grid(a.rows, a.cols / 16);
    if (a.out_dtype == STRATA_BF16)
        return launch_rows(k_fp4_dequantize<FMT, __nv_bfloat16>, g.grid, s, a, g.rows_per_warp);
    if (a.out_dtype == STRATA_F16)
        return launch_rows(k_fp4_dequantize<FMT, __half>, g.grid, s, a, g.rows_per_warp);
    return launch_rows(k_fp4_dequantize<FMT, float>, g.grid, s, a, g.rows_per_warp);
}

}  // namespace

cudaError_t launch_fp4_quantize(const Fp4QuantArgs& a, cudaStream_t s) {
    return a.fmt == STRATA_FP4_MX ? quantize<0>(a, s) : quantize<1>(a, s);
}

cudaError_t launch_fp4_dequantize(const Fp4DequantArgs& a, cudaStream_t s) {
    return a.fmt == STRATA_FP4_MX ? dequantize<0>(a, s) : dequantize<1>(a, s);
}

}  // namespace strata
