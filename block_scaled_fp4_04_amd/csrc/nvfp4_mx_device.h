// nvfp4_mx_device.h -- device helpers of the MXFP4 kernels: the quantisation
// rule for one block and the scaled MFMAs.
//
// An MXFP4 block is 32 consecutive values of a row: E2M1 codes c_i and one
// E8M0 byte e, standing for c_i * 2^(e - 127) (OCP Microscaling Formats
// v1.0; e = 255: the whole block is NaN).  gfx950 multiplies such blocks as
// they are: each lane of a scaled MFMA brings the 32 codes of one block (16
// bytes) and that block's scale byte, which is why the packed layout keeps
// the 16 code bytes of a block together.
#pragma once
#include "nvfp4_mx_internal.h"

namespace nvfp4 {
namespace {

typedef int mx_v8i __attribute__((ext_vector_type(8)));
typedef float mx_f4 __attribute__((ext_vector_type(4)));
typedef float mx_f16 __attribute__((ext_vector_type(16)));
typedef float mx_f2 __attribute__((ext_vector_type(2)));
typedef __bf16 mx_b2 __attribute__((ext_vector_type(2)));
typedef unsigned int mx_u4 __attribute__((ext_vector_type(4)));

// The scale byte of a block whose largest magnitude has the fp32 bits
// `top`: floor(log2(top)) - 2 + 127 (2 = the exponent of the largest E2M1
// power of two, 4), at least 0; 255 if the block holds an infinity or a NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
    const uint32_t e = top >> 23;
    return e == 255u ? 255u : e < 2u ? 0u : e - 2u;
}

// The scale as the conversion instructions take it: the byte in the
// exponent field (they read nothing else of it, so byte 0 is 2^-127 and 255
// NaN; checked for every byte and every bfloat16 value).
__device__ __forceinline__ float mx_scale(uint32_t byte) {
    return __builtin_bit_cast(float, byte << 23);
}

// Two bfloat16 values of a word.  (By value: a bit cast of a vector's element
// in place takes the vector's first one.)
__device__ __forceinline__ mx_b2 mx_pair(uint32_t w) { return __builtin_bit_cast(mx_b2, w); }

// The largest magnitude, as fp32 bits, of 16 bytes of values: 4 fp32, or 8
// bfloat16 (element 2i in the low half of word i).  Magnitudes order like
// their bits, so two bfloat16 are compared at once with the packed 16-bit
// maximum.
template <typename T>
__device__ __forceinline__ uint32_t mx_top(const mx_u4& v) {
    if constexpr (sizeof(T) == 2) {
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        u16x2 m = {0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[j] & 0x7FFF7FFFu));
        return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
    } else {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, v[j] & 0x7FFFFFFFu);
        return top;
    }
}
// The codes of the same values under scale s: a word from bfloat16 ones, half
// HALF of word c from fp32 ones.  The conversion divides by the scale exactly
// (a power of two), rounds to the nearest E2M1 value, ties to the even code,
// and saturates at 6; from bfloat16 it equals the one from fp32.
template <typename T, int HALF>
__device__ __forceinline__ uint32_t mx_codes(uint32_t c, const mx_u4& v, float s) {
    if constexpr (sizeof(T) == 2) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, mx_pair(v[0]), s, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, mx_pair(v[1]), s, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, mx_pair(v[2]), s, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, mx_pair(v[3]), s, 3);
    } else {
        const mx_f4 f = __builtin_bit_cast(mx_f4, v);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[0], f[1], s, 2 * HALF);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, f[2], f[3], s, 2 * HALF + 1);
    }
    return c;
}

// A whole block in one lane: the 32 values at p (16-byte aligned) -> 16 bytes
// of codes and the scale byte.
template <typename T>
__device__ __forceinline__ uint32_t mx_quant_load(const T* p, mx_u4& w) {
    constexpr int L = kMxBlock * (int)sizeof(T) / 16, PER = L / 4;  // loads; of them, to a word of codes
    mx_u4 v[L];
#pragma unroll
    for (int i = 0; i < L; ++i) v[i] = reinterpret_cast<const mx_u4*>(p)[i];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < L; ++i) top = max(top, mx_top<T>(v[i]));
    const uint32_t byte = mx_scale_byte(top);
    const float s = mx_scale(byte);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t c = mx_codes<T, 0>(0, v[PER * j], s);
        if constexpr (PER == 2) c = mx_codes<T, 1>(c, v[PER * j + 1], s);
        w[j] = byte == 255u ? 0u : c;
    }
    return byte;
}

__device__ __forceinline__ mx_v8i mx_operand(const mx_u4& w) {
    return mx_v8i{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
}

// acc += A (16 rows) . B (16 rows)^T over 128 elements.  Lane l brings row
// l % 16, elements 32 * (l / 16) ...; its scale is byte S of the word.
// Result: lane l holds row l % 16 of the second operand and rows
// 4 * (l / 16) .. + 3 of the first.
template <int S>
__device__ __forceinline__ mx_f4 mx_mfma16(const mx_u4& a, uint32_t sa, const mx_u4& b, uint32_t sb,
                                           mx_f4 acc) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(a), mx_operand(b), acc, 4, 4, S,
                                                            (int)sa, S, (int)sb);
}
// The same for 32 x 32 rows over 64 elements: lane l brings row l % 32,
// elements 32 * (l / 32) ...; result: row l % 32 of the second operand, rows
// 8 * (v / 4) + 4 * (l / 32) + v % 4 of the first.
template <int S>
__device__ __forceinline__ mx_f16 mx_mfma32(const mx_u4& a, uint32_t sa, const mx_u4& b, uint32_t sb,
                                            mx_f16 acc) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(a), mx_operand(b), acc, 4, 4, S,
                                                           (int)sa, S, (int)sb);
}

__device__ __forceinline__ uint16_t mx_to_bf16(float x) {
    return __builtin_bit_cast(uint16_t, (__bf16)x);
}

}  // namespace
}  // namespace nvfp4
