// swiglu_tc.cu -- SwiGLU on the tensor cores, forward.
#include "swiglu_tc.cuh"

namespace strata {

namespace {
template <bool BF16>
cudaError_t run(const GmmArgs& g, const SwigluKeep& k, cudaStream_t s) {
    const SwigluPiece<BF16> epi{k, gt_vec(k.h, size_t(k.I) * 2),
                                k.p == nullptr ? 0 : gt_vec(k.p, size_t(2) * k.I * (k.scales ? 1 : 2))};
    return gt_pick<kGmmFwd>(g, epi, s);
}
}  // namespace

cudaError_t launch_swiglu_tc(const GmmArgs& g, const SwigluKeep& k, cudaStream_t s) {
    return k.bf16 ? run<true>(g, k, s) : run<false>(g, k, s);
}

}  // namespace strata
