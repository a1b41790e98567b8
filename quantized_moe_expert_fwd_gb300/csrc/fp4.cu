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
constexpr int kQAhead = 2;               // steps whose loads a warp has in flight

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

// Eight words at once where the address is a multiple of 32 bytes (`wide`): a
// lane then takes a whole sector, and a warp's 32 lanes one request.
__device__ __forceinline__ void load8(const void* p, bool wide, uint32_t* w) {
    if (wide) {
        asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                       "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    } else {
        const uint4 a = __ldg(static_cast<const uint4*>(p)), b = __ldg(static_cast<const uint4*>(p) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
}
__device__ __forceinline__ void store8(void* p, bool wide, const uint32_t* w) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// The sixteen elements at p as raw words (8 of a 16-bit type, 16 of fp32).
template <typename T>
struct Raw16 {
    uint32_t w[sizeof(T) * 4];
};
template <typename T>
__device__ __forceinline__ Raw16<T> load_raw(const T* p, bool wide) {
    Raw16<T> r;
#pragma unroll
    for (int i = 0; i < int(sizeof(T)); i += 2)
        load8(reinterpret_cast<const uint8_t*>(p) + 16 * i, wide, r.w + 4 * i);
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
//  - NV, 16-bit inputs: a quotient amax / 6 (x / s) either is a border between
//    two e4m3 (e2m1) values, or is at least 2^-11 of it away.  The product with
//    the reciprocal rounded up, rounded toward zero, is exactly the border in
//    the first case -- for all 126 borders of e4m3, and for all 8 mantissas of
//    s by all 7 borders of e2m1 -- and within 2^-22 of the quotient in the
//    second.  (Two IEEE divisions a unit were a third of its instructions.)
//  - NV, fp32 inputs can be closer: amax / 6 rounded to fp32 is a border only
//    when it is one (6 times a border has at most 7 bits, and floats next to
//    it stay apart after the division); elements are compared with the seven
//    borders times s, which have at most 7 bits.
// recip[m]: 8 / (8 + m) rounded up, for the mantissa m of s.
constexpr float kSixthUp = 0x1.555556p-3f;
__device__ __forceinline__ float recip_up(int m) { return __fdiv_ru(8.0f, float(8 + m)); }

template <int FMT, typename T>
__device__ __forceinline__ uint32_t quantize16(const Raw16<T>& raw, uint32_t amax, float down,
                                               int scale_exp, const float* recip, uint2& q) {
    const bool finite = amax < 0x7f800000u;
    float v[16];
    // blocks without a finite scale above zero are computed along and replaced
    // at the end: no branch
    if (FMT == 0) {
        // floor(log2 amax) - 2, at least -127: elements of the top binade
        // reach 4 .. 6 (above 6 they saturate)
        const int ex = max(int(amax >> 23) - 129, -127);
        const float inv = __uint_as_float(uint32_t(127 - ex) << 23);         // 2^-ex
        raw_f32(raw, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= inv;
        const bool codes = finite && amax != 0u;
        q = make_uint2(codes ? cvt_e2m1x8(v) : 0u, codes ? cvt_e2m1x8(v + 8) : 0u);
        return !finite ? 255u : codes ? uint32_t(ex + 127) : 0u;
    }
    const float top = __uint_as_float(amax) * down;
    const float want = sizeof(T) == 4 ? top / 6.0f : __fmul_rz(top, kSixthUp);
    uint16_t s2;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s2) : "f"(0.0f), "f"(want));
    const uint32_t sbyte = uint32_t(s2 & 0xffu);
    const bool codes = finite && sbyte != 0u;
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
        q = make_uint2(codes ? w[0] : 0u, codes ? w[1] : 0u);
    } else {
        // the exponent of s and the tensor's power of two come off as integers
        const int e = int(__float_as_uint(s) >> 23) - 127 + scale_exp;
        const float inv = __uint_as_float(
            __float_as_uint(recip[__float_as_uint(s) >> 20 & 7u]) - (uint32_t(e) << 23));
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __fmul_rz(v[j], inv);
        q = make_uint2(codes ? cvt_e2m1x8(v) : 0u, codes ? cvt_e2m1x8(v + 8) : 0u);
    }
    return finite ? sbyte : 0x7fu;
}

// The rows cut into steps of 512 columns (a lane 16 of them, a unit), a run of
// consecutive steps a warp: all warps the GPU holds get the same number to
// within one, and a row's group is looked up about once a run.
struct Steps {
    int row, step, left;                 // the next step and the number that remain
    __device__ __forceinline__ void skip(int to, int steps) {
        const long long n = (long long)(to - row) * steps - step;
        left = n < left ? left - int(n) : 0;
        row = to;
        step = 0;
    }
};
// each, more: all warps take `each` steps, the first `more` one more.  (Worked
// out by the host: the 64-bit divisions were a sixth of the instructions.)
__device__ __forceinline__ Steps warp_steps(int steps, int each, int more) {
    const int w = int(blockIdx.x) * (kQThreads / 32) + int(threadIdx.x >> 5);
    const long long lo = (long long)w * each + min(w, more);
    const int left = each + (w < more ? 1 : 0);
    if (lo < (1ll << 31)) {
        const uint32_t l = uint32_t(lo), r = l / uint32_t(steps);
        return Steps{int(r), int(l - r * uint32_t(steps)), left};
    }
    return Steps{int(lo / steps), int(lo % steps), left};
}

// 2^e for a small e.
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }

// The 4 (NV) or 8 (MX) lanes of a scale word write it as one; units past the
// row's end contribute the zeros of its last word.
//
// 16384 rows of 2048 in bf16: gathered from 2048 rows 15.0 us (MX) and 15.6
// (NV), read from memory 15.3 and 16.2 (12.7 us of bytes; 19 and 20.5 with one
// step's loads in flight).  Bound by instructions: about 170 for a warp's 512 elements.
template <int FMT, typename T>
__global__ void __launch_bounds__(kQThreads, 4) k_fp4_quantize(Fp4QuantArgs a, int wide, int each, int more) {
    __shared__ float recip[8];
    if (threadIdx.x < 8) recip[threadIdx.x] = recip_up(threadIdx.x);
    __syncthreads();
    pdl_launch();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int units = a.cols / 16, words = fp4_words(a.cols, FMT), steps = (units + 31) / 32;
    const float down = pow2f(-a.scale_exp);
    const T* x = static_cast<const T*>(a.x);
    Steps s = warp_steps(steps, each, more);
    RowGroup g{-1, -1, 0, -1};
    while (s.left > 0) {
        const int row = s.row;
        if (row >= g.end) g = row_group(a.offsets, a.n_groups, a.rows, row, a.err);
        if (g.first < 0) {
            // on to the next row that may have a group
            s.skip(g.end, steps);
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
        const T* xr = x + size_t(bad ? 0 : src) * a.cols;
        uint8_t* qr = a.q + size_t(row) * (a.cols / 2);
        uint8_t* sr = a.scales + fp4_scale_at(size_t(g.block) + (r >> 7), words, r, 0);
        const int end = min(steps, s.step + s.left);
        s.left -= end - s.step;
        for (int u0 = s.step * 32 + lane; u0 < end * 32; u0 += 32 * kQAhead) {
            Raw16<T> raws[kQAhead];
#pragma unroll
            for (int k = 0; k < kQAhead; ++k) {
                const int u = u0 + 32 * k;
                raws[k] = Raw16<T>{};
                if (u < min(units, end * 32) && !bad) raws[k] = load_raw(xr + u * 16, wide != 0);
            }
#pragma unroll
            for (int k = 0; k < kQAhead; ++k) {
                const int u = u0 + 32 * k;
                if (u - lane >= end * 32) break;
                const Raw16<T>& raw = raws[k];
                uint32_t amax = raw_amax(raw);
                if (FMT == 0) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                uint2 q;
                uint32_t word = quantize16<FMT>(raw, amax, down, a.scale_exp, recip, q);
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
                    *reinterpret_cast<uint32_t*>(sr + size_t(w) * 512) = word;
                if (u < units) *reinterpret_cast<uint2*>(qr + u * 8) = q;
            }
        }
        s.step = 0;
        ++s.row;
    }
}

template <int FMT, typename T>
__global__ void __launch_bounds__(kQThreads, 6) k_fp4_dequantize(Fp4DequantArgs a, int wide, int each, int more) {
    pdl_launch();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int units = a.cols / 16, words = fp4_words(a.cols, FMT), steps = (units + 31) / 32;
    const float up = pow2f(a.scale_exp);
    T* out = static_cast<T*>(a.out);
    Steps s = warp_steps(steps, each, more);
    RowGroup g{-1, -1, 0, -1};
    while (s.left > 0) {
        const int row = s.row;
        if (row >= g.end) g = row_group(a.offsets, a.n_groups, a.rows, row, a.err);
        if (g.first < 0) {
            s.skip(g.end, steps);
            continue;
        }
        const int r = row - g.first;
        const uint8_t* qr = a.q + size_t(row) * (a.cols / 2);
        const uint8_t* sr = a.scales + fp4_scale_at(size_t(g.block) + (r >> 7), words, r, 0);
        const int end = min(steps, s.step + s.left);
        s.left -= end - s.step;
        for (int u = s.step * 32 + lane; u < min(end * 32, units); u += 32) {
            const int sc = FMT == 0 ? u >> 1 : u;
            const float f32s = fp4_scale_f32<FMT>(__ldg(sr + size_t(sc >> 2) * 512 + (sc & 3)));
            const uint2 q = __ldg(reinterpret_cast<const uint2*>(qr + u * 8));
            uint32_t w[sizeof(T) * 4];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t h2 = e2m1x2_to_f16x2(((j < 4 ? q.x : q.y) >> (8 * (j & 3))) & 0xffu);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                // value times scale is exact (6 bits); the power of two is
                // applied last, so it rounds only outside fp32's normal range
                const float v0 = f.x * f32s * up, v1 = f.y * f32s * up;
                if constexpr (sizeof(T) == 4) {
                    w[2 * j] = __float_as_uint(v0);
                    w[2 * j + 1] = __float_as_uint(v1);
                } else if constexpr (std::is_same<T, __half>::value) {
                    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v1), "f"(v0));
                } else {
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(v1), "f"(v0));
                }
            }
            uint8_t* o = reinterpret_cast<uint8_t*>(out + size_t(row) * a.cols + u * 16);
#pragma unroll
            for (int j = 0; j < int(sizeof(T)); j += 2) store8(o + 16 * j, wide != 0, w + 4 * j);
        }
        s.step = 0;
        ++s.row;
    }
}

// per_sm: the CTAs of the kernel that a SM holds.
template <typename... P, typename A>
cudaError_t launch_steps(void (*kernel)(P...), int per_sm, cudaStream_t s, const A& args,
                         const void* wide_base) {
    const long long steps = (long long)args.rows * ((args.cols / 16 + 31) / 32);
    const long long want = (steps + kQThreads / 32 - 1) / (kQThreads / 32);
    const int most = device_info().sms * per_sm;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(want < most ? int(want) : most);
    cfg.blockDim = dim3(kQThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const long long warps = (long long)cfg.gridDim.x * (kQThreads / 32);
    // rows are multiples of 64 bytes, so the base decides for all of them
    return cudaLaunchKernelEx(&cfg, kernel, args,
                              int((reinterpret_cast<uintptr_t>(wide_base) & 31u) == 0),
                              int(steps / warps), int(steps % warps));
}

template <int FMT>
cudaError_t quantize(const Fp4QuantArgs& a, cudaStream_t s) {
    if (a.dtype == STRATA_BF16)
        return launch_steps(k_fp4_quantize<FMT, __nv_bfloat16>, 4, s, a, a.x);
    if (a.dtype == STRATA_F16) return launch_steps(k_fp4_quantize<FMT, __half>, 4, s, a, a.x);
    return launch_steps(k_fp4_quantize<FMT, float>, 4, s, a, a.x);
}

template <int FMT>
cudaError_t dequantize(const Fp4DequantArgs& a, cudaStream_t s) {
    if (a.out_dtype == STRATA_BF16)
        return launch_steps(k_fp4_dequantize<FMT, __nv_bfloat16>, 6, s, a, a.out);
    if (a.out_dtype == STRATA_F16)
        return launch_steps(k_fp4_dequantize<FMT, __half>, 6, s, a, a.out);
    return launch_steps(k_fp4_dequantize<FMT, float>, 6, s, a, a.out);
}

}  // namespace

cudaError_t launch_fp4_quantize(const Fp4QuantArgs& a, cudaStream_t s) {
    return a.fmt == STRATA_FP4_MX ? quantize<0>(a, s) : quantize<1>(a, s);
}

cudaError_t launch_fp4_dequantize(const Fp4DequantArgs& a, cudaStream_t s) {
    return a.fmt == STRATA_FP4_MX ? dequantize<0>(a, s) : dequantize<1>(a, s);
}

}  // namespace strata
