// nvfp4_mx_quantize.hip -- gfx950 kernels that turn fp32 or bfloat16 rows
// into packed MXFP4 and back.
//
// Per block of 32 values x_i of a row (OCP Microscaling Formats v1.0):
//   e = max(0, floor(log2(max |x_i|)) - 2 + 127)   scale 2^(e - 127)
//   c_i = E2M1 value nearest to x_i / 2^(e - 127), ties to the even code,
//         at most 6 in magnitude
// and e = 255 (NaN), codes 0, for a block with an infinity or a NaN in it.
//
// A wave makes one fragment of the packed layout, 16 rows x 128 elements.
// Bound by memory.
#include "nvfp4_mx_device.h"

#include <algorithm>

namespace nvfp4 {
namespace {

// Every load covers whole lines: 16 bytes a lane, side by side along the rows
// (with a lane loading its whole block, in pieces at a stride of 128 or 64
// bytes, 16381 x 8160 fp32 took 122 us, and 269 with non-temporal loads).  The
// 8 or 4 lanes of a block find its largest magnitude with lane permutes; the
// codes go through LDS, from where lane l stores bytes 16 l ... of the
// fragment.  NT: non-temporal loads, for inputs of more than kStreamBytes
// (105 us; 116 without; 16384 x 8192 bfloat16 54 and 59 us).
template <typename T, bool NT>
__global__ void __launch_bounds__(256) mx_quantize_kernel(MxQuantArgs a) {
    constexpr int E = 16 / (int)sizeof(T);     // elements of a load
    constexpr int LPB = kMxBlock / E;          // lanes to a block
    constexpr int LPR = kMxStep / E;           // lanes to a row
    constexpr int RPL = 64 / LPR;              // rows to a load
    constexpr int L = kMxRows / RPL;           // loads
    __shared__ __attribute__((aligned(16))) uint8_t lds[4][kMxFrag + 64];
    const int lane = threadIdx.x & 63;
    const int64_t frag = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);  // (group, row block, step)
    const int64_t total = a.groups * a.RB * a.C;
    if (frag >= total) return;
    const int64_t grb = frag / a.C;
    const int c = (int)(frag % a.C);
    const int row0 = (int)(grb % a.RB) * kMxRows + lane / LPR;
    const int k = c * kMxStep + lane % LPR * E, b = lane % LPR / LPB;
    const T* x = static_cast<const T*>(a.x) + grb / a.RB * a.group_stride + min(k, a.K - E);
    mx_u4 v[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {  // (rows and columns past the ends: others, unused)
        const mx_u4* p = reinterpret_cast<const mx_u4*>(x + (int64_t)min(row0 + i * RPL, a.rows - 1) * a.ld);
        if constexpr (NT)
            v[i] = __builtin_nontemporal_load(p);
        else
            v[i] = *p;
    }
    uint8_t* codes = lds[threadIdx.x >> 6];
    uint8_t* bytes = codes + kMxFrag;
#pragma unroll
    for (int i = 0; i < L; ++i) {
        if (row0 + i * RPL >= a.rows || k >= a.K) v[i] = mx_u4{0, 0, 0, 0};
        uint32_t top = mx_top<T>(v[i]);
        top = mx_block_top<LPB>(top);
        const uint32_t byte = mx_scale_byte(top);
        const uint32_t w = byte == 255u ? 0u : mx_codes<T, 0>(0, v[i], mx_scale(byte));
        const int r = i * RPL + lane / LPR;
        uint8_t* d = codes + mx_code_at(r, b) + lane % LPB * (E / 2);
        if constexpr (E == 8)
            *reinterpret_cast<uint32_t*>(d) = w;
        else
            *reinterpret_cast<uint16_t*>(d) = (uint16_t)w;
        if (lane % LPB == 0) bytes[r * 4 + b] = (uint8_t)byte;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    reinterpret_cast<mx_u4*>(a.codes + frag * kMxFrag)[lane] = reinterpret_cast<const mx_u4*>(codes)[lane];
    const int Q = (a.C + 3) / 4;
    uint8_t* s = a.scales + (grb * Q + c / 4) * kMxScaleFrag + lane * 4;  // of row lane / 4, block lane % 4
    s[c & 3] = bytes[lane];
    // the last step also clears the scales of the steps that fill its word
    if (c == a.C - 1)
        for (int t = (c & 3) + 1; t < 4; ++t) s[t] = 0;
}

// A wave takes one fragment here, too, but stores whole rows of it: the codes
// go through LDS, from where lane l picks those of the elements E l, E l + 1,
// ... of a few rows at a time (E = 16 bytes of output), so that every store
// covers whole lines (a lane storing its own block in pieces cost 180 us
// instead of 125 for 16381 x 8160 fp32).  NT: non-temporal stores.
template <typename T, bool NT>
__global__ void __launch_bounds__(256) mx_dequantize_kernel(MxQuantArgs a) {
    constexpr int E = 16 / (int)sizeof(T);     // elements of a store
    constexpr int LPR = kMxStep / E;           // lanes to a row
    constexpr int RPS = 64 / LPR;              // rows to a store
    __shared__ __attribute__((aligned(16))) uint8_t lds[4][kMxFrag + 64];
    const int lane = threadIdx.x & 63;
    const int64_t frag = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t total = a.groups * a.RB * a.C;
    if (frag >= total) return;
    uint8_t* codes = lds[threadIdx.x >> 6];
    uint8_t* bytes = codes + kMxFrag;
    const int64_t grb = frag / a.C;
    const int c = (int)(frag % a.C);
    const int64_t g = grb / a.RB;
    const int Q = (a.C + 3) / 4;
    reinterpret_cast<mx_u4*>(codes)[lane] = reinterpret_cast<const mx_u4*>(a.codes + frag * kMxFrag)[lane];
    bytes[lane] = a.scales[(grb * Q + c / 4) * kMxScaleFrag + lane * 4 + (c & 3)];  // of row lane / 4, block lane % 4
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int col = lane % LPR * E, k = c * kMxStep + col, b = col / kMxBlock;
#pragma unroll
    for (int r0 = 0; r0 < kMxRows; r0 += RPS) {
        const int r = r0 + lane / LPR;
        const int row = (int)(grb % a.RB) * kMxRows + r;
        const float s = mx_scale(bytes[r * 4 + b]);
        const uint8_t* p = codes + mx_code_at(r, b) + col % kMxBlock / 2;
        // (a code times a power of two is exact in either type, subnormals
        // included, up to the overflow to infinity at 2^128)
        mx_u4 o;
        if constexpr (sizeof(T) == 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
            o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
            o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
            o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
            o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
        } else {
            const uint32_t w = *reinterpret_cast<const uint16_t*>(p);
            const mx_f2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
            const mx_f2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
            o = __builtin_bit_cast(mx_u4, mx_f4{lo[0], lo[1], hi[0], hi[1]});
        }
        if (row >= a.rows || k >= a.K) continue;
        mx_u4* d = reinterpret_cast<mx_u4*>(static_cast<T*>(a.x) + g * a.group_stride + (int64_t)row * a.ld + k);
        if constexpr (NT)
            __builtin_nontemporal_store(o, d);
        else
            *d = o;
    }
}

template <typename T>
void run_quantize(const MxQuantArgs& a, hipStream_t stream) {
    const int64_t frags = a.groups * a.RB * a.C;
    const dim3 grid((unsigned)((frags + 3) / 4));
    if (a.groups * a.rows * (int64_t)a.K * (int64_t)sizeof(T) > kStreamBytes)
        hipLaunchKernelGGL((mx_quantize_kernel<T, true>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((mx_quantize_kernel<T, false>), grid, dim3(256), 0, stream, a);
}

template <typename T>
void run_dequantize(const MxQuantArgs& a, hipStream_t stream) {
    const int64_t frags = a.groups * a.RB * a.C;
    const dim3 grid((unsigned)((frags + 3) / 4));
    if (a.groups * a.rows * (int64_t)a.K * (int64_t)sizeof(T) > kStreamBytes)
        hipLaunchKernelGGL((mx_dequantize_kernel<T, true>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((mx_dequantize_kernel<T, false>), grid, dim3(256), 0, stream, a);
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantArgs& a, hipStream_t stream) {
    if (a.bf16)
        run_quantize<uint16_t>(a, stream);
    else
        run_quantize<float>(a, stream);
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const MxQuantArgs& a, hipStream_t stream) {
    if (a.bf16)
        run_dequantize<uint16_t>(a, stream);
    else
        run_dequantize<float>(a, stream);
    return hipGetLastError();
}

}  // namespace nvfp4
