// norm.cuh -- the RMS norms before and after a block, its gate and the scales
// of residual and branch, forward (norm.cu) and backward (norm_bwd.cu).
//   n  = f s0 wpost          s0 = 1 / sqrt(mean f^2 + eps)   (or n = f)
//   r' = alpha r + beta gate n
//   x  = r' s1 wpre          s1 = 1 / sqrt(mean r'^2 + eps)
// Backward, from dx and the gradient dr' of r' by other paths, with
// D = dr' + s1 (dx wpre - r' s1^2 mean(dx wpre r')) the whole gradient by r':
//   dr = alpha D,  dgate = beta sum(D n),  dn = beta gate D
//   df = s0 (dn wpost - f s0^2 mean(dn wpost f))             (or df = dn)
//   dwpre = sum over the rows of dx r' s1,  dwpost = sum of dn f s0
// x is of r' as it is stored, so that the backward pass sees what the forward
// pass did.
//
// Both are bound by memory: every tensor moves once.  W warps have a row in
// their registers, 8 C columns a thread: fours of neighbouring ones where rows
// are whole numbers of 4 columns (VEC).  Neighbouring lanes have neighbouring
// fours, so that an access of a warp covers whole sectors in fp32 and in 16
// bits.  Other rows: strided columns forward (16384 rows of 1031 columns 55 us;
// aligned fours with the rows' ends one by one 81), the fours that the row lies
// in backward.  Longer rows take a kernel that reads them once a pass.
#pragma once

#include "grouped.h"
#include "rows.cuh"

namespace strata {

// A warp's sums: one access.
template <int N>
struct __align__(N == 1 ? 4 : 16) NormSums {
    float v[N == 1 ? 1 : (N + 3) / 4 * 4];
};

// A thread's place among the W warps of a row, and their sums.
template <int W, int C, bool VEC>
struct NormRow {
    static constexpr int kThreads = W * 32, kBlock = kThreads > 256 ? kThreads : 256;
    static constexpr int kGroups = kBlock / kThreads;
    int group, id;                           // row of the block, thread of the row
    __device__ __forceinline__ NormRow() : group(int(threadIdx.x) / kThreads), id(int(threadIdx.x) % kThreads) {}
    __device__ __forceinline__ int column(int c, int j) const {
        return VEC ? ((2 * c + j / 4) * kThreads + id) * 4 + j % 4 : (c * 8 + j) * kThreads + id;
    }
    // Eight columns; zeros past the row's end.
    template <bool NC, typename T>
    __device__ __forceinline__ Raw<T, 8> load(const T* row, int c, int H) const {
        Raw<T, 8> r{};
        if constexpr (VEC) {
            constexpr int N = Raw<T, 4>::kWords;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (column(c, 4 * h) >= H) continue;
                const Raw<T, 4> p = ld_row<T, 4, NC>(row + column(c, 4 * h));
#pragma unroll
                for (int i = 0; i < N; ++i) r.w[h * N + i] = p.w[i];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (column(c, j) >= H) continue;
                const Raw<T, 1> e = ld_row<T, 1, NC>(row + column(c, j));
                if constexpr (sizeof(T) == 4) r.w[j] = e.w[0];
                else r.w[j >> 1] |= e.w[0] << (16 * (j & 1));
            }
        }
        return r;
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, int c, int H, const float (&v)[8]) const {
        if constexpr (VEC) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (column(c, 4 * h) < H)
                    st_row<T, 4>(row + column(c, 4 * h), reinterpret_cast<const float(&)[4]>(v[4 * h]));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (column(c, j) < H) row[column(c, j)] = from_f32<T>(v[j]);
        }
    }
    // N sums over the row's threads, in all of them; buf is used by
    // every other call (a thread past the barrier of the next has read this one's).
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N], NormSums<N> (*buf)[kGroups][W]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
        if constexpr (W > 1) {
            if ((id & 31) == 0) {
#pragma unroll
                for (int i = 0; i < N; ++i) (*buf)[group][id >> 5].v[i] = v[i];
            }
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kThreads) : "memory");
            NormSums<N> s = (*buf)[group][0];
#pragma unroll
            for (int k = 1; k < W; ++k) {
                const NormSums<N> o = (*buf)[group][k];
#pragma unroll
                for (int i = 0; i < N; ++i) s.v[i] += o.v[i];
            }
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = s.v[i];
        }
    }
};

// ------------------------------------------------- rows of any length
constexpr int kNmThreads = 256;

// The sum over a CTA, in all its threads; buf: a float a warp, free again
// after the next barrier.
__device__ __forceinline__ float cta_sum(float v, float* buf) {
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < int(blockDim.x) >> 5; ++i) s += buf[i];
    return s;
}

// A thread's sum of f(c) over its columns of a row, in pieces of 64.
template <typename F>
__device__ __forceinline__ float column_sum(int H, F f) {
    float sum = 0.0f;
    for (int c0 = threadIdx.x; c0 < H; c0 += 64 * kNmThreads) {
        float part = 0.0f;
        for (int c = c0; c < min(H, c0 + 64 * kNmThreads); c += kNmThreads) part += f(c);
        sum += part;
    }
    return sum;
}

}  // namespace strata
