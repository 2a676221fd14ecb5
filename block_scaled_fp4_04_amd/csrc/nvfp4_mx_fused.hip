// nvfp4_mx_fused.hip -- the MXFP4 product with bias, activation and residual
// (nvfp4_mx_product.h).  The grouped product's kernels have a source file of their
// own, so that the two compile side by side.
#include "nvfp4_mx_product.h"

namespace nvfp4 {

hipError_t launch_mx_fused(const MxGemmArgs& a, const MxEpilogueArgs& e, hipStream_t stream) {
    if (a.groups > 0) return launch_mx_fused_grouped(a, e, stream);
    Launch<EPI_ONE> l{a, {e}, stream, false, 0, hipSuccess};
    choose_single(l);
    return l.error;
}

bool mx_fused_fits(const MxGemmArgs& a) {
    if (a.groups > 0) return mx_fused_grouped_fits(a);
    Launch<EPI_ONE> l{a, {}, nullptr, true, 0, hipSuccess};
    choose_single(l);
    return l.items < ((int64_t)1 << 32);
}

}  // namespace nvfp4
