// nvfp4_rows.h -- 16-byte pieces of fp32 / bfloat16 rows that may start
// anywhere (aligned to their elements only), for the kernels that work on
// whole rows (expert routing, norms).
#pragma once
#include "nvfp4_mx_device.h"

namespace nvfp4 {
namespace {

template <typename T, int V>
struct Piece {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Piece<T, V> load_piece(const T* p) {
    Piece<T, V> r;
    __builtin_memcpy(&r, p, sizeof(r));
    return r;
}
// NT: with the non-temporal hint.
template <bool NT, typename T, int V>
__device__ __forceinline__ void store_piece(T* p, const Piece<T, V>& r) {
    if constexpr (NT && sizeof(r) == 16) {
        typedef unsigned int u4 __attribute__((ext_vector_type(4), aligned(2)));
        u4 t;
        __builtin_memcpy(&t, &r, 16);
        __builtin_nontemporal_store(t, reinterpret_cast<u4*>(p));
    } else {
        __builtin_memcpy(p, &r, sizeof(r));
    }
}
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return __builtin_bit_cast(float, (uint32_t)x << 16); }
__device__ __forceinline__ void narrow(float x, float& o) { o = x; }
__device__ __forceinline__ void narrow(float x, uint16_t& o) { o = mx_to_bf16(x); }

}  // namespace
}  // namespace nvfp4
