// grouped_tc.cu -- the grouped products on the tensor cores: plain outputs.
#include "grouped_tc_kernel.cuh"

namespace strata {

// The tensor maps need rows of a multiple of 16 bytes.
bool grouped_tc_takes(GroupedMode mode, const GmmArgs& g) {
    return g.K % 8 == 0 && (mode == kGmmFwd || g.N % 8 == 0);
}

cudaError_t launch_grouped_tc(GroupedMode mode, const GmmArgs& g, cudaStream_t s) {
    switch (mode) {
        case kGmmFwd: return gt_pick<kGmmFwd>(g, GtPlain{}, s);
        case kGmmDx: return gt_pick<kGmmDx>(g, GtPlain{}, s);
        default: return gt_pick<kGmmDw>(g, GtPlain{}, s);
    }
}

}  // namespace strata
