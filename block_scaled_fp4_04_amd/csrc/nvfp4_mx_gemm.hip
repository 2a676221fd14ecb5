// nvfp4_mx_gemm.hip -- the MXFP4 product without an epilogue
// (nvfp4_mx_product.h).
#include "nvfp4_mx_product.h"

namespace nvfp4 {

hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t stream) {
    Launch<EPI_NONE> l{a, {}, stream, false, 0, hipSuccess};
    choose(l);
    return l.error;
}

bool mx_gemm_fits(const MxGemmArgs& a) {
    Launch<EPI_NONE> l{a, {}, nullptr, true, 0, hipSuccess};
    choose(l);
    return l.items < ((int64_t)1 << 32);
}

}  // namespace nvfp4
