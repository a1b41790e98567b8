// act8.cu -- rows to 8 bits and back.
#include <type_traits>

#include "act8.cuh"
#include "grouped.cuh"
#include "grouped.h"

namespace strata {

namespace {

constexpr int kA8Threads = 256;

// A lane takes 8 elements, four lanes a block of 32.
template <typename T>
__device__ __forceinline__ void a8_load(const T* p, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p));
        const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
        const T* e = reinterpret_cast<const T*>(&a);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = to_f32(e[j]);
    }
}

template <typename T>
__global__ void __launch_bounds__(kA8Threads) k_act8_save(const T* x, size_t units, uint8_t* q,
                                                          uint8_t* scales) {
    const size_t step = size_t(gridDim.x) * kA8Threads;
    // units is a multiple of 4: the lanes of a block stay together
    for (size_t i = size_t(blockIdx.x) * kA8Threads + threadIdx.x; i < units; i += step) {
        float v[8];
        a8_load(x + i * 8, v);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
        const uint32_t group = 0xfu << (threadIdx.x & 28);
        m = max(m, __shfl_xor_sync(group, m, 1));
        m = max(m, __shfl_xor_sync(group, m, 2));
        const uint32_t b = act8_byte(m);
        const float inv = act8_inverse(b);
        uint2 w = make_uint2(act8_codes(v[0], v[1], v[2], v[3], inv), act8_codes(v[4], v[5], v[6], v[7], inv));
        if (b == 255u) w = make_uint2(kAct8Nan, kAct8Nan);
        *reinterpret_cast<uint2*>(q + i * 8) = w;
        if (i % 4 == 0) scales[i / 4] = uint8_t(b);
    }
}

// A value that fp16 cannot hold reads as its largest.
template <typename T>
__device__ __forceinline__ float a8_fit(float v) {
    if constexpr (sizeof(T) == 2 && !std::is_same<T, __nv_bfloat16>::value)
        if (fabsf(v) > 65504.0f) return copysignf(65504.0f, v);       // (not a NaN)
    return v;
}

// Destination row r from source row perm[r] / top_k (perm NULL: r).
template <typename T>
__global__ void __launch_bounds__(kA8Threads) k_act8_load(Act8LoadArgs a) {
    const int per = a.cols / 8;                       // units of a row
    const size_t units = size_t(a.rows) * per, step = size_t(gridDim.x) * kA8Threads;
    T* out = static_cast<T*>(a.out);
    for (size_t i = size_t(blockIdx.x) * kA8Threads + threadIdx.x; i < units; i += step) {
        const size_t r = i / per;
        const int c = int(i % per);
        long long src = (long long)r;
        if (a.perm != nullptr) {
            const int p = __ldg(a.perm + r);
            src = p < 0 ? -1 : p / a.top_k;
        }
        float v[8] = {};
        if (src < 0 || src >= a.q_rows) {
            if (c == 0) latch(a.err, STRATA_EBADROUTE);
        } else {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(a.q + size_t(src) * a.cols) + c);
            const float s = act8_scale(__ldg(a.scales + size_t(src) * (a.cols / kAct8Block) + c / 4));
            act8_values(w.x, s, v);
            act8_values(w.y, s, v + 4);
        }
        T o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = from_f32<T>(a8_fit<T>(v[j]));
#pragma unroll
        for (int j = 0; j < int(sizeof(T)) / 2; ++j)
            reinterpret_cast<uint4*>(out + i * 8)[j] = reinterpret_cast<const uint4*>(o)[j];
    }
}

int a8_grid(size_t units) {
    const size_t want = (units + kA8Threads - 1) / kA8Threads, most = size_t(device_info().sms) * 8;
    return int(want < most ? want : most);
}

template <typename T>
cudaError_t run_save(const Act8SaveArgs& a, cudaStream_t s) {
    const size_t units = size_t(a.rows) * a.cols / 8;
    k_act8_save<T><<<a8_grid(units), kA8Threads, 0, s>>>(static_cast<const T*>(a.x), units, a.q, a.scales);
    return cudaGetLastError();
}
template <typename T>
cudaError_t run_load(const Act8LoadArgs& a, cudaStream_t s) {
    k_act8_load<T><<<a8_grid(size_t(a.rows) * a.cols / 8), kA8Threads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_act8_save(const Act8SaveArgs& a, cudaStream_t s) {
    return a.dtype == STRATA_BF16  ? run_save<__nv_bfloat16>(a, s)
           : a.dtype == STRATA_F16 ? run_save<__half>(a, s)
                                   : run_save<float>(a, s);
}
cudaError_t launch_act8_load(const Act8LoadArgs& a, cudaStream_t s) {
    return a.out_dtype == STRATA_BF16  ? run_load<__nv_bfloat16>(a, s)
           : a.out_dtype == STRATA_F16 ? run_load<__half>(a, s)
                                       : run_load<float>(a, s);
}

}  // namespace strata
