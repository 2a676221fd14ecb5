// nvfp4_mx_parts.h -- what the kernels of the MXFP4 products share: loads
// straight to LDS, unaligned pieces of rows, LDS order within a wave.
#pragma once
#include "nvfp4_device.h"
#include "nvfp4_mx_device.h"

#include <type_traits>
#include <utility>

namespace nvfp4 {
namespace {

// dma16 / dma4 (nvfp4_device.h) with the LDS address as a uniform base plus a
// constant: one scalar instruction a load.  NT: with the non-temporal hint.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int BYTES, int AT, bool NT = false>
__device__ __forceinline__ void mx_dma(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff,
                                       uint32_t lds) {
    if constexpr (BYTES == 16 && NT)
        asm volatile("s_add_u32 m0, %3, %4\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds"
                     :: "v"(voff), "s"(r), "s"(soff), "s"(lds), "n"(AT) : "memory", "m0", "scc");
    else if constexpr (BYTES == 16)
        asm volatile("s_add_u32 m0, %3, %4\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                     :: "v"(voff), "s"(r), "s"(soff), "s"(lds), "n"(AT) : "memory", "m0", "scc");
    else
        asm volatile("s_add_u32 m0, %3, %4\n\tbuffer_load_dword %0, %1, %2 offen lds"
                     :: "v"(voff), "s"(r), "s"(soff), "s"(lds), "n"(AT) : "memory", "m0", "scc");
}
#pragma clang diagnostic pop

// f(integral_constant<int, 0>) ... f(integral_constant<int, N - 1>)
template <typename F, int... I>
__device__ __forceinline__ void mx_each(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void mx_each(F&& f) { mx_each(f, std::make_integer_sequence<int, N>{}); }

// Stores of rows of C that may start anywhere (N need not be a multiple of
// anything): a piece is one access, aligned to its elements only.
typedef unsigned int mx_u2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef unsigned int mx_u4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float mx_f4_any __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ uint32_t mx_bf16_pair(float x, float y) {
    return mx_to_bf16(x) | (uint32_t)mx_to_bf16(y) << 16;
}

// Four consecutive values of a row of N from column `col` on (element `at`),
// rounded.
__device__ __forceinline__ void mx_put4(void* out, bool bf16, int64_t at, int col, int N, mx_f4 f) {
    if (col + 4 <= N) {
        if (bf16)
            *reinterpret_cast<mx_u2_any*>(static_cast<uint16_t*>(out) + at) =
                mx_u2_any{mx_bf16_pair(f[0], f[1]), mx_bf16_pair(f[2], f[3])};
        else
            *reinterpret_cast<mx_f4_any*>(static_cast<float*>(out) + at) = f;
        return;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        if (col + v >= N) break;
        if (bf16)
            static_cast<uint16_t*>(out)[at + v] = mx_to_bf16(f[v]);
        else
            static_cast<float*>(out)[at + v] = f[v];
    }
}

// Orders a wave's LDS accesses among its lanes.
__device__ __forceinline__ void mx_wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Four consecutive values of a row of N from column `col` on, widened; zeros
// past its end and without a row.
__device__ __forceinline__ mx_f4 mx_row4(const void* p, bool bf16, int64_t at, int col, int N) {
    mx_f4 f = {0.0f, 0.0f, 0.0f, 0.0f};
    if (!p) return f;
    if (bf16) {
        const uint16_t* x = static_cast<const uint16_t*>(p) + at;
        if (col + 4 <= N) {
            const mx_u2_any w = *reinterpret_cast<const mx_u2_any*>(x);
#pragma unroll
            for (int v = 0; v < 4; ++v) f[v] = mx_widen(w[v >> 1], v & 1);
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (col + v < N) f[v] = mx_widen(x[v], 0);
        }
    } else {
        const float* x = static_cast<const float*>(p) + at;
        if (col + 4 <= N) {
            f = *reinterpret_cast<const mx_f4_any*>(x);
        } else {
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (col + v < N) f[v] = x[v];
        }
    }
    return f;
}

}  // namespace
}  // namespace nvfp4
