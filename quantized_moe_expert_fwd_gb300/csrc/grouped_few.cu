// grouped_few.cu -- the forward products for a handful of rows (the kernel is in
// grouped_few.cuh) or of columns.
#include "grouped_few.cuh"

namespace strata {

namespace {

constexpr int kNarrowCols = kNarrowColsMax;

// The sums as the output's type.
template <typename TO>
struct FewStore {
    TO* y;
    int N;
    __device__ __forceinline__ void operator()(size_t row, int n0, const float (&s)[kFewRows]) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < kFewRows; ++i)
            if (lane == i && n0 + i < N) y[row * N + n0 + i] = from_f32<TO>(s[i]);
    }
};
template <bool BF16, typename TO>
cudaError_t store_few(const GmmArgs& g, cudaStream_t s) {
    return run_few<BF16>(g, FewStore<TO>{static_cast<TO*>(g.out), g.N}, s);
}

// Few columns instead of few rows: a warp a row of x, every column's W row
// from the caches (the warps of a CTA work on neighbouring rows, so mostly on
// one expert's).  On the tensor cores a tile of any width takes every stage of
// the reduction.  Tensor cores and here, us, calls back to back: 2536 rows of
// 317 experts, 1816 wide, 1 column 24.2 4.4, 4 columns 24.3 6.6, 8 columns 24.0
// 9.3; 8000 rows of 4 experts, 4096 wide (in the L2), 21.7 9.3, 17.2 19.5, 16.4
// 33.1; 32000 such rows, 62.0 41.6, 46.0 58.2, 45.7 113.7.  Hence at most 4
// columns: 5 to 8 would gain only where the experts have few rows.
template <bool BF16, bool LONG, typename TO>
__global__ void __launch_bounds__(kFewThreads, 3) k_gmm_narrow(GmmArgs g) {
    pdl_launch();
    pdl_wait();
    const int lane = threadIdx.x & 31, pieces = g.K / 8;
    const int warps = int(gridDim.x) * (kFewThreads / 32);
    const int wi = int(blockIdx.x) * (kFewThreads / 32) + int(threadIdx.x >> 5);
    const uint4* w = static_cast<const uint4*>(g.b);
    TO* y = static_cast<TO*>(g.out);
    RowGroup gr{-1, -1, 0, -1};
    const int last = int((long long)g.M * (wi + 1) / warps);
    for (int row = int((long long)g.M * wi / warps); row < last; ++row) {
        if (row >= gr.end) gr = row_group(g.offsets, g.E, g.M, row, g.err);
        if (gr.first < 0) {
            row = gr.end - 1;
            continue;
        }
        const uint4* x = static_cast<const uint4*>(g.a) + size_t(row) * pieces;
        const uint4* we = w + size_t(gr.e) * g.N * pieces;
        float acc[kNarrowCols] = {}, aside[kNarrowCols] = {};
        for (int p0 = lane; p0 < pieces; p0 += 32 * kFewLoads) {
            if (LONG && p0 >= kFewChunk && p0 % kFewChunk == lane) {
#pragma unroll
                for (int n = 0; n < kNarrowCols; ++n) {
                    aside[n] += acc[n];
                    acc[n] = 0.0f;
                }
            }
            uint4 v[kFewLoads];
#pragma unroll
            for (int l = 0; l < kFewLoads; ++l)
                v[l] = p0 + 32 * l < pieces ? ldg_stream(x + p0 + 32 * l) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int n = 0; n < kNarrowCols; ++n) {
                if (n >= g.N) break;
#pragma unroll
                for (int l = 0; l < kFewLoads; ++l)
                    if (p0 + 32 * l < pieces)
                        acc[n] = dot8<BF16>(v[l], __ldg(we + size_t(n) * pieces + p0 + 32 * l), acc[n]);
            }
        }
#pragma unroll
        for (int n = 0; n < kNarrowCols; ++n) {
            if (n >= g.N) break;
            const float s = warp_sum(LONG ? aside[n] + acc[n] : acc[n]);
            if (lane == n) y[size_t(row) * g.N + n] = from_f32<TO>(s);
        }
    }
}

template <bool BF16, typename TO>
cudaError_t run_narrow(const GmmArgs& g, cudaStream_t s) {
    return few_long(g) ? few_launch(k_gmm_narrow<BF16, true, TO>, g.M, 3, s, g)
                       : few_launch(k_gmm_narrow<BF16, false, TO>, g.M, 3, s, g);
}

}  // namespace

cudaError_t launch_grouped_few(const GmmArgs& g, cudaStream_t s) {
    if (g.dtype == STRATA_BF16)
        return g.out_dtype == STRATA_F32 ? store_few<true, float>(g, s)
                                         : store_few<true, __nv_bfloat16>(g, s);
    return g.out_dtype == STRATA_F32 ? store_few<false, float>(g, s) : store_few<false, __half>(g, s);
}

cudaError_t launch_grouped_narrow(const GmmArgs& g, cudaStream_t s) {
    if (g.dtype == STRATA_BF16)
        return g.out_dtype == STRATA_F32 ? run_narrow<true, float>(g, s)
                                         : run_narrow<true, __nv_bfloat16>(g, s);
    return g.out_dtype == STRATA_F32 ? run_narrow<false, float>(g, s)
                                     : run_narrow<false, __half>(g, s);
}

}  // namespace strata
