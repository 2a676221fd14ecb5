// nvfp4_norm_f32.hip -- the norms on fp32 rows (nvfp4_norm_kernels.h).
#include "nvfp4_norm_kernels.h"

namespace nvfp4 {

hipError_t launch_norm_f32(const NormArgs& a, hipStream_t stream) { return run_norm<float, 4>(a, stream); }

}  // namespace nvfp4
