// swiglu_back_tc.cu -- SwiGLU's gradient on the tensor cores.
#include "swiglu_tc.cuh"

namespace strata {

namespace {
template <bool BF16>
cudaError_t run(const GmmArgs& g, const SwigluBack& k, cudaStream_t s) {
    const SwigluBackPiece<BF16> epi{k};
    return gt_pick<kGmmDx>(g, epi, s);
}
}  // namespace

cudaError_t launch_swiglu_back_tc(const GmmArgs& g, const SwigluBack& k, cudaStream_t s) {
    return k.bf16 ? run<true>(g, k, s) : run<false>(g, k, s);
}

}  // namespace strata
