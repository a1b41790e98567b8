// slots.cu -- a token's slots weighted into its row, and the gradients of
// that: its row's gradient spread over its slots, the weights' as dot products.
//   combine  out[t] = sum_k w[t][k] y[slot(t, k)]
//   spread   dy[slot(t, k)] = w[t][k] dout[t],  dw[t][k] = <dout[t], y[slot(t, k)]>
#include "grouped.cuh"
#include "grouped.h"

namespace strata {

namespace {

constexpr int kSlThreads = 128;

// The slots of a token; -1 for one outside [0, M).
__device__ __forceinline__ int slot_of(const SlotsArgs& a, size_t t, int k) {
    const int s = __ldg(a.inv + t * a.top_k + k);
    return s < 0 || s >= a.M ? -1 : s;
}

template <typename T, typename TO>
__global__ void __launch_bounds__(kSlThreads) k_slots_combine(SlotsArgs a) {
    const size_t t = blockIdx.x;
    const T* y = static_cast<const T*>(a.y);
    TO* out = static_cast<TO*>(a.out);
    for (int c = threadIdx.x; c < a.H; c += kSlThreads) {
        float sum = 0.0f;
        for (int k = 0; k < a.top_k; ++k) {
            const int s = slot_of(a, t, k);
            if (s < 0) {
                if (c == 0) latch(a.err, STRATA_EBADROUTE);
                continue;
            }
            const float w = a.weights ? __ldg(a.weights + t * a.top_k + k) : 1.0f;
            sum = fmaf(w, to_f32(y[size_t(s) * a.H + c]), sum);
        }
        out[t * a.H + c] = from_f32<TO>(sum);
    }
}

template <typename T>
__global__ void __launch_bounds__(kSlThreads) k_slots_spread(SlotsArgs a) {
    __shared__ float part[kSlThreads / 32];
    const size_t t = blockIdx.x;
    const T* dout = static_cast<const T*>(a.dout) + t * a.H;
    for (int k = 0; k < a.top_k; ++k) {
        const int s = slot_of(a, t, k);
        if (s < 0 && threadIdx.x == 0) latch(a.err, STRATA_EBADROUTE);
        const float w = a.weights ? __ldg(a.weights + t * a.top_k + k) : 1.0f;
        float dot = 0.0f;
        if (s >= 0)
            for (int c = threadIdx.x; c < a.H; c += kSlThreads) {
                const float d = to_f32(dout[c]);
                const size_t at = size_t(s) * a.H + c;
                if (a.dy) static_cast<T*>(a.dy)[at] = from_f32<T>(w * d);
                if (a.dweights) dot = fmaf(d, to_f32(static_cast<const T*>(a.y)[at]), dot);
            }
        if (a.dweights) {
            dot = warp_sum(dot);
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
            __syncthreads();
            if (threadIdx.x == 0) {
                for (int i = 1; i < kSlThreads / 32; ++i) dot += part[i];
                a.dweights[t * a.top_k + k] = dot;
            }
            __syncthreads();
        }
    }
}

}  // namespace

cudaError_t launch_slots_combine(const SlotsArgs& a, cudaStream_t s) {
    if (a.dtype == STRATA_BF16) {
        if (a.out_dtype == STRATA_F32) k_slots_combine<__nv_bfloat16, float><<<a.T, kSlThreads, 0, s>>>(a);
        else k_slots_combine<__nv_bfloat16, __nv_bfloat16><<<a.T, kSlThreads, 0, s>>>(a);
    } else {
        if (a.out_dtype == STRATA_F32) k_slots_combine<__half, float><<<a.T, kSlThreads, 0, s>>>(a);
        else k_slots_combine<__half, __half><<<a.T, kSlThreads, 0, s>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_slots_spread(const SlotsArgs& a, cudaStream_t s) {
    if (a.dtype == STRATA_BF16) k_slots_spread<__nv_bfloat16><<<a.T, kSlThreads, 0, s>>>(a);
    else k_slots_spread<__half><<<a.T, kSlThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace strata
