// swiglu.cu -- the gated feed-forward block over grouped rows: gate and up
// products with SwiGLU, and the down product's input gradient with SwiGLU's
// gradient, each one kernel: the grouped products' own, with another epilogue
// (tensor cores; few rows forward; any width).  A pass over p in memory, or over
// dh, is what the epilogue saves: 2048-token prompt of 256 experts of 1024 x 2048
// (bf16, us) 186 forward with p kept where the plain product alone takes 182;
// 113 back where its product alone takes 94 (at the copy's rate 175 and 101).
#include "grouped_few.cuh"
#include "grouped_simt.cuh"
#include "swiglu.cuh"

namespace strata {

namespace {

struct KeepQuad {
    SwigluKeep k;
    __device__ __forceinline__ void operator()(size_t row, int c, const float* v, bool live) const {
        swiglu_quad(k, row, c, v, live);
    }
};
// Few rows: a warp has the sums of two pairs.  (8 rows of 8 such experts: 7.9 us
// against 11.5 on the tensor cores, the plain product 7.6.)
struct KeepFew {
    SwigluKeep k;
    __device__ __forceinline__ void operator()(size_t row, int n0, const float (&s)[kFewRows]) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < kFewRows; i += 2) {
            if (n0 + i >= 2 * k.I || lane != i) continue;
            store_u16(k.h, row * k.I + (n0 + i) / 2, pack16(swiglu(s[i], s[i + 1]), 0.0f, k.bf16));
            if (k.p == nullptr) continue;
            const uint32_t w = pack16(s[i], s[i + 1], k.bf16);
            store_u16(k.p, row * 2 * k.I + n0 + i, w);
            store_u16(k.p, row * 2 * k.I + n0 + i + 1, w >> 16);
        }
    }
};
struct BackQuad {
    SwigluBack k;
    __device__ __forceinline__ void operator()(size_t row, int c, const float* v, bool live) const {
        swiglu_back_quad(k, row, c, v, live);
    }
};

template <int MODE, typename EPI>
cudaError_t swiglu_simt(const GmmArgs& g, const EPI& epi, cudaStream_t s) {
    const int grid = device_info().sms * 4;
    if (g.dtype == STRATA_BF16) k_gmm_simt<MODE, __nv_bfloat16><<<grid, kSimtThreads, 0, s>>>(g, epi);
    else k_gmm_simt<MODE, __half><<<grid, kSimtThreads, 0, s>>>(g, epi);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_swiglu(const SwigluArgs& a, cudaStream_t s) {
    GmmArgs g{};
    g.a = a.x;
    g.b = a.w;
    g.offsets = a.offsets;
    g.err = a.err;
    g.M = a.M;
    g.K = a.K;
    g.N = 2 * a.I;
    g.E = a.E;
    g.dtype = a.dtype;
    const SwigluKeep k{a.h, a.p, a.scales, a.I, a.dtype == STRATA_BF16};
    // (8-bit blocks span the columns of several warps of the few-row kernel)
    if (g.M <= kFewRowsMax && g.K % 8 == 0 && a.scales == nullptr)
        return k.bf16 ? run_few<true>(g, KeepFew{k}, s) : run_few<false>(g, KeepFew{k}, s);
    if (grouped_tc_takes(kGmmFwd, g)) return launch_swiglu_tc(g, k, s);
    return swiglu_simt<kGmmFwd>(g, KeepQuad{k}, s);
}

cudaError_t launch_swiglu_bwd(const SwigluBwdArgs& a, cudaStream_t s) {
    GmmArgs g{};
    g.a = a.dy;
    g.b = a.w;
    g.offsets = a.offsets;
    g.err = a.err;
    g.M = a.M;
    g.K = a.I;
    g.N = a.N;
    g.E = a.E;
    g.dtype = a.dtype;
    const SwigluBack k{a.p, a.scales, a.dp, a.h, a.I, a.dtype == STRATA_BF16};
    if (grouped_tc_takes(kGmmDx, g)) return launch_swiglu_back_tc(g, k, s);
    return swiglu_simt<kGmmDx>(g, BackQuad{k}, s);
}

}  // namespace strata
