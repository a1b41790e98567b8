// act8.cu -- rows to 8 bits and back.  Bound by memory: 3.03 bytes an element
// each way in 16 bits.  A lane takes 16 elements (an access of 16 bytes of
// codes, of 32 in 16 bits), two lanes a block of 32.  Loads of several pieces a
// lane at once cost more by their registers than they hid: 65536 rows of 2048
// read back 66 us with four, 61 with two, 54 with one; 8 elements a lane 72.
#include "act8.cuh"
#include "grouped.h"
#include "rows.cuh"

namespace strata {

namespace {

constexpr int kA8Threads = 256;

template <typename T>
struct Raw16 {                               // 16 elements
    static constexpr int kParts = int(sizeof(T)) / 2;
    Raw<T, 16 / kParts> r[kParts];
    __device__ __forceinline__ float get(int j) const { return r[j / (16 / kParts)].get(j % (16 / kParts)); }
};
template <typename T>
__device__ __forceinline__ Raw16<T> ld16(const T* p, bool wide) {
    Raw16<T> v;
#pragma unroll
    for (int i = 0; i < Raw16<T>::kParts; ++i) ld_words(p + i * (16 / Raw16<T>::kParts), wide, v.r[i].w);
    return v;
}

template <typename T>
__global__ void __launch_bounds__(kA8Threads) k_act8_save(const T* x, size_t units, uint8_t* q,
                                                          uint8_t* scales, bool wide) {
    pdl_launch();
    pdl_wait();
    const size_t step = size_t(gridDim.x) * kA8Threads;
    // units (of 16 elements) is even: the two lanes of a block stay together
    for (size_t i = size_t(blockIdx.x) * kA8Threads + threadIdx.x; i < units; i += step) {
        const Raw16<T> v = ld16(x + i * 16, wide);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max(m, __float_as_uint(v.get(j)) & 0x7fffffffu);
        m = max(m, __shfl_xor_sync(0x3u << (threadIdx.x & 30), m, 1));
        const uint32_t b = act8_byte(m);
        const float inv = act8_inverse(b);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = b == 255u
                       ? kAct8Nan
                       : act8_codes(v.get(4 * j), v.get(4 * j + 1), v.get(4 * j + 2), v.get(4 * j + 3), inv);
        st_words(q + i * 16, false, w);
        if (i % 2 == 0) scales[i / 2] = uint8_t(b);
    }
}

// A value that fp16 cannot hold reads as its largest.
template <typename T>
__device__ __forceinline__ float a8_fit(float v) {
    if constexpr (std::is_same<T, __half>::value)
        if (fabsf(v) > 65504.0f) return copysignf(65504.0f, v);       // (not a NaN)
    return v;
}

// Block (bx, by): bx lanes along a row, by rows at a time.  Destination row r
// from source row perm[r] / top_k (perm NULL: r).
template <typename T>
__global__ void __launch_bounds__(kA8Threads) k_act8_load(Act8LoadArgs a, bool wide) {
    pdl_launch();
    pdl_wait();
    const int c = int(blockIdx.y * blockDim.x + threadIdx.x) * 16;
    if (c >= a.cols) return;
    const size_t step = size_t(gridDim.x) * blockDim.y;
    T* out = static_cast<T*>(a.out) + c;
    for (size_t r = size_t(blockIdx.x) * blockDim.y + threadIdx.y; r < size_t(a.rows); r += step) {
        int src = int(r);
        if (a.perm != nullptr) {
            const int p = __ldg(a.perm + r);
            src = p < 0 ? -1 : p / a.top_k;
        }
        float v[16] = {};
        if (src >= 0 && src < a.q_rows) {
            uint32_t w[4];
            ld_words(a.q + size_t(src) * a.cols + c, false, w);
            const float s = act8_scale(__ldg(a.scales + size_t(src) * (a.cols / kAct8Block) + c / kAct8Block));
#pragma unroll
            for (int j = 0; j < 4; ++j) act8_values(w[j], s, v + 4 * j);
        } else if (c == 0) {
            latch(a.err, STRATA_EBADROUTE);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = a8_fit<T>(v[j]);
        T* o = out + r * a.cols;
        if constexpr (sizeof(T) == 4) {
            st_row<T, 8>(o, reinterpret_cast<const float(&)[8]>(v[0]), wide);
            st_row<T, 8>(o + 8, reinterpret_cast<const float(&)[8]>(v[8]), wide);
        } else {
            st_row<T, 16>(o, v, wide);
        }
    }
}

template <typename T>
cudaError_t run_save(const Act8SaveArgs& a, cudaStream_t s) {
    const size_t units = size_t(a.rows) * a.cols / 16;
    const size_t want = (units + kA8Threads - 1) / kA8Threads, most = size_t(device_info().sms) * 16;
    return row_launch(k_act8_save<T>, dim3(unsigned(want < most ? want : most)), dim3(kA8Threads), s,
                      static_cast<const T*>(a.x), units, a.q, a.scales, aligned32(a.x, 0));
}
template <typename T>
cudaError_t run_load(const Act8LoadArgs& a, cudaStream_t s) {
    const int units = a.cols / 16;
    int bx = 2;
    while (bx < units && bx < kA8Threads) bx *= 2;
    const int by = kA8Threads / bx, pieces = (units + bx - 1) / bx;
    const int want = (a.rows + by - 1) / by, most = (device_info().sms * 32 + pieces - 1) / pieces;
    return row_launch(k_act8_load<T>, dim3(want < most ? want : most, pieces), dim3(bx, by), s, a,
                      aligned32(a.out, size_t(a.cols) * sizeof(T)));
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
