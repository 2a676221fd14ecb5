// nvfp4_norm_bf16.hip -- the norms on bfloat16 rows (nvfp4_norm_kernels.h).
#include "nvfp4_norm_kernels.h"

namespace nvfp4 {

hipError_t launch_norm_bf16(const NormArgs& a, hipStream_t stream) { return run_norm<uint16_t, 8>(a, stream); }

}  // namespace nvfp4
