// nvfp4_norm.hip -- launches of the norms around a block's residual and of
// their gradients (nvfp4_norm_kernels.h), and the last step of the gradients'
// sums over rows.
#include "nvfp4_norm_kernels.h"

namespace nvfp4 {
namespace {

// Adds the workgroups' sums: 64 columns to a workgroup, 16 waves that each take
// every sixteenth.
__global__ void __launch_bounds__(1024) norm_grad_sum_kernel(NormArgs a) {
    __shared__ float part[16][64];
    const int which = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float* const out = which == 0 ? a.dpre_weight : which == 1 ? a.dpost_weight
                     : a.gate_mode == kGateChannel ? static_cast<float*>(a.dgate) : nullptr;
    if (!out) return;
    const int col = blockIdx.x * 64 + lane, at = min(col, a.hidden - 1);
    float s = 0.0f;
#pragma unroll 16
    for (int k = wave; k < a.parts; k += 16) s += a.partials[((int64_t)k * 3 + which) * a.hidden + at];
    part[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || col >= a.hidden) return;
#pragma unroll
    for (int w = 1; w < 16; ++w) s += part[w][lane];
    out[col] = s;
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
    return a.bf16 ? launch_norm_bf16(a, stream) : launch_norm_f32(a, stream);
}

hipError_t launch_norm_grad(const NormArgs& a, hipStream_t stream) {
    if (a.rows > 0) {
        const hipError_t error = a.bf16 ? launch_norm_grad_bf16(a, stream) : launch_norm_grad_f32(a, stream);
        if (error != hipSuccess) return error;
    }
    if (a.partials || a.rows == 0)  // (no rows: the sums are zeros)
        hipLaunchKernelGGL(norm_grad_sum_kernel, dim3((unsigned)((a.hidden + 63) / 64), 3), dim3(1024), 0, stream, a);
    return hipGetLastError();
}

int norm_grad_parts(bool bf16, int64_t rows, int hidden) {
    return bf16 ? parts_of<8>(rows, hidden) : parts_of<4>(rows, hidden);
}

}  // namespace nvfp4
