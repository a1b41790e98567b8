// rows.cuh -- a few consecutive elements of a row as one memory access, and
// the launch of kernels whose threads lie along rows.
#pragma once

#include <type_traits>

#include "grouped.cuh"

namespace strata {

// V elements of T (16-bit types, fp32), up to 32 bytes, as raw words.
template <typename T, int V>
struct Raw {
    static constexpr int kBytes = int(sizeof(T)) * V;
    static constexpr int kWords = (kBytes + 3) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ float get(int j) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
        else {
            const uint32_t h = w[j >> 1] >> (16 * (j & 1));
            if constexpr (std::is_same<T, __half>::value) return f16_to_f32(uint16_t(h));
            else return __uint_as_float(h << 16);
        }
    }
};

// `wide`: the address is a multiple of 32 bytes (only asked where V elements
// have that many); otherwise of their size, or of 16 bytes.  NC: nobody writes
// there while the kernel runs.
template <bool NC = true, int WORDS>
__device__ __forceinline__ void ld_words(const void* p, bool wide, uint32_t (&w)[WORDS]) {
    if constexpr (WORDS == 1) {
        const uint32_t* q = static_cast<const uint32_t*>(p);
        w[0] = NC ? __ldg(q) : *q;
    } else if constexpr (WORDS == 2) {
        const uint2* q = static_cast<const uint2*>(p);
        const uint2 v = NC ? __ldg(q) : *q;
        w[0] = v.x;
        w[1] = v.y;
    } else if constexpr (WORDS == 4) {
        const uint4* q = static_cast<const uint4*>(p);
        const uint4 v = NC ? __ldg(q) : *q;
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
        static_assert(WORDS == 8, "words of an access");
        if (wide) {
            if (NC)
                asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                               "=r"(w[6]), "=r"(w[7])
                             : "l"(p));
            else
                asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                               "=r"(w[6]), "=r"(w[7])
                             : "l"(p)
                             : "memory");
        } else {
            const uint4* q = static_cast<const uint4*>(p);
            const uint4 a = NC ? __ldg(q) : q[0], b = NC ? __ldg(q + 1) : q[1];
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
            w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
        }
    }
}
template <int WORDS>
__device__ __forceinline__ void st_words(void* p, bool wide, const uint32_t (&w)[WORDS]) {
    if constexpr (WORDS == 1) *static_cast<uint32_t*>(p) = w[0];
    else if constexpr (WORDS == 2) *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (WORDS == 4) *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else {
        static_assert(WORDS == 8, "words of an access");
        if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]),
                         "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
        } else {
            static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}
template <typename T, int V, bool NC = true>
__device__ __forceinline__ Raw<T, V> ld_row(const T* p, bool wide = false) {
    Raw<T, V> r;
    if constexpr (Raw<T, V>::kBytes == 2) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
        r.w[0] = NC ? __ldg(q) : *q;
    } else {
        ld_words<NC>(p, wide, r.w);
    }
    return r;
}
// One rounding, to nearest even, into T.
template <typename T, int V>
__device__ __forceinline__ void st_row(T* p, const float (&v)[V], bool wide = false) {
    Raw<T, V> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < V; ++j) r.w[j] = __float_as_uint(v[j]);
    } else if constexpr (V == 1) {
        *p = from_f32<T>(v[0]);
        return;
    } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            if constexpr (std::is_same<T, __half>::value)
                asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r.w[j]) : "f"(v[2 * j + 1]), "f"(v[2 * j]));
            else
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.w[j]) : "f"(v[2 * j + 1]), "f"(v[2 * j]));
        }
    }
    st_words(p, wide, r.w);
}

inline bool aligned32(const void* p, size_t pitch) {
    return ((reinterpret_cast<uintptr_t>(p) | pitch) & 31u) == 0;
}

// Starts behind the grids before it as soon as those have no block left to
// start (programmatic dependent launch): the kernel has to call pdl_wait()
// before it touches memory.
template <typename... P, typename... A>
cudaError_t row_launch(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t s, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace strata
