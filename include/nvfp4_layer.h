/*
 * nvfp4_layer.h -- C ABI of the operators that stand around the MXFP4
 * products (nvfp4_mx.h) in a transformer layer: products with an epilogue.
 *
 * Status codes, pointers, streams, errors, types and sizes as in nvfp4_mx.h.
 * In the library from nvfp4_version() 10700 on.
 */
#ifndef NVFP4_LAYER_H
#define NVFP4_LAYER_H

#include "nvfp4_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations, in fp32:
 *   SILU       z / (1 + exp(-z))
 *   GELU       z * (1 + erf(z / sqrt(2))) / 2
 *   GELU_TANH  z * (1 + tanh(sqrt(2 / pi) * (z + 0.044715 z^3))) / 2 */
enum {
    NVFP4_ACT_NONE = 0,
    NVFP4_ACT_RELU = 1,
    NVFP4_ACT_SILU = 2,
    NVFP4_ACT_GELU = 3,
    NVFP4_ACT_GELU_TANH = 4
};

/* ---- products with an epilogue ---------------------------------------------
 *
 * With z = alpha * (A . B^T) + bias, in fp32 and rounded once at the end,
 *   C = act(z) + residual, or, with a gate operand G of B's sizes,
 *   C = act(alpha * (A . G^T) + gate_bias) * z + residual.
 * Parts that are NULL are left out (a bias or residual of zeros, no gate). */
typedef struct nvfp4_mx_epilogue {
    int activation;          /* NVFP4_ACT_* */
    const void* gate_packed; /* DEVICE, packed like B, and its scales, or both NULL */
    const void* gate_scales;
    const void* bias;        /* DEVICE [N], grouped: [groups][N], or NULL */
    const void* gate_bias;   /* DEVICE, the same for the gate operand (NULL without one) */
    int bias_type;           /* NVFP4_TYPE_* of both biases */
    const void* residual;    /* DEVICE, M x N of the output's type, or NULL; may be out itself
                                (row stride N then), else it must not overlap out */
    int64_t ld_residual;     /* its row stride in elements, at least N (a single row's is not
                                looked at) */
} nvfp4_mx_epilogue;

/* nvfp4_mx_gemm, nvfp4_mx_gemm_quantized and nvfp4_mx_grouped_gemm with an
 * epilogue (NULL: those calls themselves).  The struct is read before the
 * call returns.  Biases and the residual need the alignment of their elements
 * only.  The quantised form again gives the bits of the packed one. */
int nvfp4_mx_gemm_fused(const void* a_packed, const void* a_scales, const void* b_packed,
                        const void* b_scales, float alpha, const nvfp4_mx_epilogue* epilogue,
                        void* out, int out_type, int64_t M, int64_t N, int64_t K, void* stream);
int nvfp4_mx_gemm_quantized_fused(const void* x, int x_type, int64_t ldx, const void* b_packed,
                                  const void* b_scales, float alpha,
                                  const nvfp4_mx_epilogue* epilogue, void* out, int out_type,
                                  int64_t M, int64_t N, int64_t K, void* stream);
int nvfp4_mx_grouped_gemm_fused(const void* a_packed, const void* a_scales, int64_t a_count,
                                const int32_t* a_rows, const void* b_packed, const void* b_scales,
                                const int32_t* row_offsets, int64_t groups, float alpha,
                                const nvfp4_mx_epilogue* epilogue, void* out, int out_type,
                                int64_t M, int64_t N, int64_t K, void* stream);

/* The same calls recorded into a sequence (nvfp4.h, "Recorded sequences"). */
int nvfp4_sequence_add_mx_gemm_fused(nvfp4_sequence_t seq, const void* a_packed,
                                     const void* a_scales, const void* b_packed,
                                     const void* b_scales, float alpha,
                                     const nvfp4_mx_epilogue* epilogue, void* out, int out_type,
                                     int64_t M, int64_t N, int64_t K);
int nvfp4_sequence_add_mx_gemm_quantized_fused(nvfp4_sequence_t seq, const void* x, int x_type,
                                               int64_t ldx, const void* b_packed,
                                               const void* b_scales, float alpha,
                                               const nvfp4_mx_epilogue* epilogue, void* out,
                                               int out_type, int64_t M, int64_t N, int64_t K);
int nvfp4_sequence_add_mx_grouped_gemm_fused(nvfp4_sequence_t seq, const void* a_packed,
                                             const void* a_scales, int64_t a_count,
                                             const int32_t* a_rows, const void* b_packed,
                                             const void* b_scales, const int32_t* row_offsets,
                                             int64_t groups, float alpha,
                                             const nvfp4_mx_epilogue* epilogue, void* out,
                                             int out_type, int64_t M, int64_t N, int64_t K);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_LAYER_H */
