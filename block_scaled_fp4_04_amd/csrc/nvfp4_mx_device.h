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

#include <type_traits>

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
// The largest of `top` over the LPB lanes (4 or 8, side by side) of a block.
template <int CTRL>
__device__ __forceinline__ uint32_t mx_dpp(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xF, 0xF, true);
}
template <int LPB>
__device__ __forceinline__ uint32_t mx_block_top(uint32_t top) {
    top = max(top, mx_dpp<0xB1>(top));   // lane ^ 1
    top = max(top, mx_dpp<0x4E>(top));   // lane ^ 2
    if constexpr (LPB == 8) top = max(top, mx_dpp<0x141>(top));  // 7 - lane, of 8
    return top;
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

// A whole block in one lane: its 32 values as they lie in memory (16-byte
// aligned) and, of those, 16 bytes of codes and the scale byte.
template <typename T>
struct MxRaw {
    static constexpr int L = kMxBlock * (int)sizeof(T) / 16;
    mx_u4 v[L];
};
template <typename T>
__device__ __forceinline__ MxRaw<T> mx_raw_load(const T* p) {
    MxRaw<T> r;
#pragma unroll
    for (int i = 0; i < r.L; ++i) r.v[i] = reinterpret_cast<const mx_u4*>(p)[i];
    return r;
}
template <typename T>
__device__ __forceinline__ uint32_t mx_quant_block(const MxRaw<T>& r, mx_u4& w) {
    constexpr int PER = MxRaw<T>::L / 4;  // loads to a word of codes
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < r.L; ++i) top = max(top, mx_top<T>(r.v[i]));
    const uint32_t byte = mx_scale_byte(top);
    const float s = mx_scale(byte);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t c = mx_codes<T, 0>(0, r.v[PER * j], s);
        if constexpr (PER == 2) c = mx_codes<T, 1>(c, r.v[PER * j + 1], s);
        w[j] = byte == 255u ? 0u : c;
    }
    return byte;
}
template <typename T>
__device__ __forceinline__ uint32_t mx_quant_load(const T* p, mx_u4& w) {
    return mx_quant_block(mx_raw_load(p), w);
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
// Keeps the matrix instructions that made x out of a branch that alone uses
// it: the compiler moves them there, but they work on every lane of the wave
// whoever takes the branch.  (A lane permute, here of each lane to itself, is
// not moved.)
__device__ __forceinline__ mx_f4 mx_pin(mx_f4 x) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        const float f = x[v];  // (by value, as mx_pair)
        x[v] = __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, f), 0xE4, 0xF, 0xF, true));
    }
    return x;
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
// The low or high bfloat16 of a word.
__device__ __forceinline__ float mx_widen(uint32_t w, int high) {
    return __builtin_bit_cast(float, high ? w & 0xFFFF0000u : w << 16);
}

// Activations (kMxAct*, uniform), in fp32:
//   silu       z / (1 + exp(-z))
//   gelu       z (1 + erf(z / sqrt 2)) / 2
//   gelu_tanh  z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2, which is
//              z / (1 + exp(-2 sqrt(2 / pi) (z + 0.044715 z^3)))
// The exponential is the hardware's power of two of a product rounded to fp32,
// the quotient a product with the hardware's reciprocal: each is off by an
// ulp or two, and by |z| 2^-24 of the exponential for the rounded product.
// gelu is z Phi(z).  Phi(-a) of a >= 0 is the exponential of -a^2 / 2 times a
// polynomial in 1 / (1 + p a), fitted by its relative error so that gelu keeps its
// digits where Phi is small: from 0 on with an error of 3.4e-7 for bfloat16
// results; from 1.25 on with 1.8e-7 for fp32 ones, and below that Phi is 0.5 + z times
// a polynomial in z^2 (1e-8).  With the roundings, relative errors of at most 7.5e-7
// and 1.3e-7 (z > -0.5) or 6e-7 for |z| up to 2, and of 1.7e-6 at -5 and 8e-6 at -12,
// mostly the square's.  A wave has the epilogue to itself: 1237 x 2056 x 6112 with
// bias, gelu and residual 21.8 us in fp32 (24.8 with the library's erfc, 19.5 without
// gelu) and 20.1 in bfloat16.
constexpr int kMxActGeluFine = -1;  // (a form of kMxActGelu)
__device__ __forceinline__ float mx_logistic(float z) {  // 1 / (1 + exp(-z))
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z));
}
// c + x * (c1 + x * (c2 + ...))
__device__ __forceinline__ float mx_poly(float, float c) { return c; }
template <typename... C>
__device__ __forceinline__ float mx_poly(float x, float c, C... more) { return c + x * mx_poly(x, more...); }
template <int ACT>
__device__ __forceinline__ float mx_act(float z) {
    if constexpr (ACT == kMxActRelu) return z < 0.0f ? 0.0f : z;
    if constexpr (ACT == kMxActSilu) return z * mx_logistic(z);
    if constexpr (ACT == kMxActGelu || ACT == kMxActGeluFine) {
        constexpr bool FINE = ACT == kMxActGeluFine;
        const float a = __builtin_fabsf(z), t = __builtin_amdgcn_rcpf(1.0f + (FINE ? 0.51f : 0.26f) * a);
        const float poly = FINE ? mx_poly(t, 9.08206948e-06f, 0.203170561f, 0.20727439f, 0.123785575f, 0.15231941f,
                                          -0.31529205f, 0.130706478f)
                                : mx_poly(t, 3.61269065e-05f, 0.102933339f, 0.111002466f, 0.0601200644f, 0.192377761f,
                                          -0.135641261f, 0.246433442f, -0.0772621069f);
        const float tail = poly * __builtin_amdgcn_exp2f(-0.72134752f * a * a);  // Phi(-a)
        float phi = z < 0.0f ? tail : 1.0f - tail;
        if constexpr (FINE) {
            const float q = mx_poly(z * z, 0.398942277f, -0.0664902079f, 0.00997228273f, -0.00118383716f, 0.000111041128f,
                                    -6.80949178e-06f);
            const float centre = 0.5f + z * q;
            phi = a < 1.25f ? centre : phi;
        }
        return z * phi;
    }
    if constexpr (ACT == kMxActGeluTanh) return z * mx_logistic(1.59576912f * z * (1.0f + 0.044715f * z * z));
    return z;
}
// Calls f(integral_constant of the activation) for results in bfloat16 or fp32.
template <typename F>
__device__ __forceinline__ void mx_by_act(int act, bool bf16, F&& f) {
    if (act == kMxActGelu && !bf16) return f(std::integral_constant<int, kMxActGeluFine>{});
    switch (act) {
        case kMxActRelu: return f(std::integral_constant<int, kMxActRelu>{});
        case kMxActSilu: return f(std::integral_constant<int, kMxActSilu>{});
        case kMxActGelu: return f(std::integral_constant<int, kMxActGelu>{});
        case kMxActGeluTanh: return f(std::integral_constant<int, kMxActGeluTanh>{});
        default: return f(std::integral_constant<int, kMxActNone>{});
    }
}

}  // namespace
}  // namespace nvfp4
