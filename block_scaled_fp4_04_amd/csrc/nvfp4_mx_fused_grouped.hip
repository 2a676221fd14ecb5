// nvfp4_mx_fused_grouped.hip -- the grouped MXFP4 product with bias, activation and
// residual (nvfp4_mx_product.h).
#include "nvfp4_mx_product.h"

namespace nvfp4 {

hipError_t launch_mx_fused_grouped(const MxGemmArgs& a, const MxEpilogueArgs& e, hipStream_t stream) {
    Launch<EPI_ONE> l{a, {e}, stream, false, 0, hipSuccess};
    choose_grouped(l);
    return l.error;
}

bool mx_fused_grouped_fits(const MxGemmArgs& a) {
    Launch<EPI_ONE> l{a, {}, nullptr, true, 0, hipSuccess};
    choose_grouped(l);
    return l.items < ((int64_t)1 << 32);
}

bool mx_fused_packs(const MxGemmArgs& a) {
    Launch<EPI_ONE> l{a, {}, nullptr, true, 0, hipSuccess};
    choose_grouped(l);
    return l.packs;
}

}  // namespace nvfp4
