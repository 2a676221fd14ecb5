// nvfp4_mx_quantize.hip -- gfx950 kernels that turn fp32 or bfloat16 rows
// into packed MXFP4 and back.
//
// Per block of 32 values x_i of a row (OCP Microscaling Formats v1.0):
//   e = max(0, floor(log2(max |x_i|)) - 2 + 127)   scale 2^(e - 127)
//   c_i = E2M1 value nearest to x_i / 2^(e - 127), ties to the even code,
//         at most 6 in magnitude
// and e = 255 (NaN), codes 0, for a block with an infinity or a NaN in it.
//
// A wave makes one fragment of the packed layout, 16 rows x 128 elements:
// lane l owns the whole block of row l % 16 at elements 32 * (l / 16), so
// the largest magnitude needs no exchange between lanes and the lanes' 16
// code bytes fill one contiguous 1 KB.  Bound by memory.
#include "nvfp4_mx_device.h"

#include <algorithm>

namespace nvfp4 {
namespace {

template <typename T>
__device__ __forceinline__ T mx_zero() { return T{}; }

template <typename T>
__global__ void __launch_bounds__(256) mx_quantize_kernel(MxQuantArgs a) {
    const int lane = threadIdx.x & 63;
    const int r16 = lane & 15, kg = lane >> 4;
    const int64_t frag = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);  // (group, row block, step)
    const int64_t total = a.groups * a.RB * a.C;
    if (frag >= total) return;
    const int64_t grb = frag / a.C;
    const int c = (int)(frag % a.C);
    const int64_t g = grb / a.RB;
    const int row = (int)(grb % a.RB) * kMxRows + r16;
    const int k = c * kMxStep + kg * kMxBlock;
    mx_u4 w = {0, 0, 0, 0};
    uint32_t byte = 0;
    if (row < a.rows && k < a.K) {
        const T* p = static_cast<const T*>(a.x) + g * a.group_stride + (int64_t)row * a.ld + k;
        byte = mx_quant_load(p, w);
    }
    *reinterpret_cast<mx_u4*>(a.codes + frag * kMxFrag + mx_code_at(r16, kg)) = w;
    const int Q = (a.C + 3) / 4;
    a.scales[(grb * Q + c / 4) * kMxScaleFrag + mx_scale_at(r16, kg) + (c & 3)] = (uint8_t)byte;
    // the last step also clears the scales of the steps that fill its word
    if (c == a.C - 1)
        for (int s = (c & 3) + 1; s < 4; ++s)
            a.scales[(grb * Q + c / 4) * kMxScaleFrag + mx_scale_at(r16, kg) + s] = 0;
}

template <typename T>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(MxQuantArgs a) {
    const int lane = threadIdx.x & 63;
    const int r16 = lane & 15, kg = lane >> 4;
    const int64_t frag = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t total = a.groups * a.RB * a.C;
    if (frag >= total) return;
    const int64_t grb = frag / a.C;
    const int c = (int)(frag % a.C);
    const int64_t g = grb / a.RB;
    const int row = (int)(grb % a.RB) * kMxRows + r16;
    const int k = c * kMxStep + kg * kMxBlock;
    if (row >= a.rows || k >= a.K) return;
    const mx_u4 w = *reinterpret_cast<const mx_u4*>(a.codes + frag * kMxFrag + mx_code_at(r16, kg));
    const int Q = (a.C + 3) / 4;
    const uint32_t byte = a.scales[(grb * Q + c / 4) * kMxScaleFrag + mx_scale_at(r16, kg) + (c & 3)];
    const float s = mx_scale(byte);
    T* p = static_cast<T*>(a.x) + g * a.group_stride + (int64_t)row * a.ld + k;
    // 8 codes of a word -> 8 values (a code times a power of two is exact in
    // either type, subnormals included)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 2) {
            mx_u4 o;
            o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 0));
            o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 1));
            o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 2));
            o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[j], s, 3));
            reinterpret_cast<mx_u4*>(p)[j] = o;
        } else {
            const mx_f2 o0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], s, 0);
            const mx_f2 o1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], s, 1);
            const mx_f2 o2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], s, 2);
            const mx_f2 o3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], s, 3);
            reinterpret_cast<mx_f4*>(p)[2 * j] = mx_f4{o0[0], o0[1], o1[0], o1[1]};
            reinterpret_cast<mx_f4*>(p)[2 * j + 1] = mx_f4{o2[0], o2[1], o3[0], o3[1]};
        }
    }
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantArgs& a, hipStream_t stream) {
    const int64_t frags = a.groups * a.RB * a.C;
    const dim3 grid((unsigned)((frags + 3) / 4));
    if (a.bf16)
        hipLaunchKernelGGL(mx_quantize_kernel<uint16_t>, grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL(mx_quantize_kernel<float>, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxQuantArgs& a, hipStream_t stream) {
    const int64_t frags = a.groups * a.RB * a.C;
    const dim3 grid((unsigned)((frags + 3) / 4));
    if (a.bf16)
        hipLaunchKernelGGL(mx_dequantize_kernel<uint16_t>, grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL(mx_dequantize_kernel<float>, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace nvfp4
