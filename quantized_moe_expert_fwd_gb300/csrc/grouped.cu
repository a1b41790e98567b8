// grouped.cu -- matrix products grouped by expert over ragged row groups:
//   forward   y[s]  = W[e] x[s]
//   dx        dx[s] = W[e]^T dy[s]
//   dw        dW[e] = sum over the group's rows s of dy[s] x[s]^T
// for the rows s of group e (offsets), W [E][N][K].
#include "grouped_simt.cuh"

namespace strata {

namespace {

template <int MODE, typename TI, typename TO>
cudaError_t run_simt(const GmmArgs& g, cudaStream_t s) {
    const SimtStore<TO> store{static_cast<TO*>(g.out), MODE == kGmmFwd ? g.N : g.K};
    k_gmm_simt<MODE, TI><<<device_info().sms * 4, kSimtThreads, 0, s>>>(g, store);
    return cudaGetLastError();
}

template <int MODE>
cudaError_t pick_simt(const GmmArgs& g, cudaStream_t s) {
    if (g.dtype == STRATA_BF16)
        return g.out_dtype == STRATA_F32 ? run_simt<MODE, __nv_bfloat16, float>(g, s)
                                         : run_simt<MODE, __nv_bfloat16, __nv_bfloat16>(g, s);
    return g.out_dtype == STRATA_F32 ? run_simt<MODE, __half, float>(g, s)
                                     : run_simt<MODE, __half, __half>(g, s);
}

}  // namespace

cudaError_t launch_grouped_mm(GroupedMode mode, const GmmArgs& g, cudaStream_t s) {
    if (mode == kGmmFwd && g.K % 8 == 0) {
        if (g.M <= kFewRowsMax) return launch_grouped_few(g, s);
        if (g.N <= kNarrowColsMax) return launch_grouped_narrow(g, s);
    }
    if (grouped_tc_takes(mode, g)) return launch_grouped_tc(mode, g, s);
    switch (mode) {
        case kGmmFwd: return pick_simt<kGmmFwd>(g, s);
        case kGmmDx: return pick_simt<kGmmDx>(g, s);
        default: return pick_simt<kGmmDw>(g, s);
    }
}

}  // namespace strata
