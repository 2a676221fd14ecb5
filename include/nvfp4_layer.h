/*
 * nvfp4_layer.h -- C ABI of the operators that stand around the MXFP4
 * products (nvfp4_mx.h) in a transformer layer: products with an epilogue, a
 * whole layer of experts, and the norms behind one block and before the next
 * with their gradients.
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
 *   GELU_TANH  z * (1 + tanh(sqrt(2 / pi) * (z + 0.044715 z^3))) / 2
 * with the GPU's power of two and reciprocal.  Relative errors, with u = 2^-24: SILU
 * up to 2 (|z| + 8) u, GELU_TANH up to 8 (|x| + 8) u of its exponent x = 1.6 z (1 +
 * 0.045 z^2), GELU up to (1.5 z^2 + 48) u: measured 1.3e-7 for z > -0.5 (7.5e-7 before
 * a result is rounded to bfloat16), 6e-7 at -2, 1.7e-6 at -5. */
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

/* nvfp4_mx_quantize and nvfp4_mx_gemm_fused in one call, or nvfp4_mx_gemm_quantized_fused
 * where that is faster (up to 16 rows, but for many of them by deep B); the same bits.
 *   workspace : DEVICE, 16-byte aligned, for the packed rows: the code and scale bytes that
 *               nvfp4_mx_packed_size(M, K) says, added up.  Free again when the call's work is
 *               done.  Up to 16 rows it may be NULL or smaller: they then take one launch. */
int nvfp4_mx_linear_fused(const void* x, int x_type, int64_t ldx, const void* b_packed,
                          const void* b_scales, float alpha, const nvfp4_mx_epilogue* epilogue,
                          void* out, int out_type, int64_t M, int64_t N, int64_t K,
                          void* workspace, size_t workspace_bytes, void* stream);

/* The products recorded into a sequence (nvfp4.h, "Recorded sequences"). */
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

/* ---- a whole layer of experts ------------------------------------------------
 *
 * For each token t and its choices e = expert_ids[t][j] (nvfp4_moe.h: numbers
 * outside [0, experts) are dropped choices),
 *   z         = q(x[t]) . U_e^T + up_bias[e]
 *   h[t][j]   = act(z), or with gate operands act(q(x[t]) . G_e^T + gate_bias[e]) * z,
 *               rounded to bfloat16
 *   out[t]    = sum over j of weights[t][j] * (q(h[t][j]) . D_e^T + down_bias[e])
 * with q() the rounding of nvfp4_mx_quantize; sums in fp32, out rounded once
 * (zeros for a token without a kept choice).
 *
 * For few tokens (up to 4, with rows that fit a workgroup's LDS when they are
 * quantised) the layer runs in two launches, bound by reading the chosen
 * experts' weights once.  Above that the steps are those of nvfp4_moe_sort,
 * nvfp4_mx_quantize, nvfp4_mx_grouped_gemm_fused twice and nvfp4_moe_combine, in
 * four to six launches, each choice's result in fp32 until the sum.
 * Deterministic either way. */
typedef struct nvfp4_mx_experts {
    int64_t experts;         /* 1 to 2048 */
    int64_t hidden, inner;   /* row lengths of x and out, and of h: multiples of 32 */
    int activation;          /* NVFP4_ACT_* */
    const void* gate_packed; /* DEVICE, `experts` packed operands of inner x hidden, or both NULL */
    const void* gate_scales;
    const void* up_packed;   /* DEVICE, `experts` packed operands of inner x hidden */
    const void* up_scales;
    const void* down_packed; /* DEVICE, `experts` packed operands of hidden x inner */
    const void* down_scales;
    int bias_type;           /* NVFP4_TYPE_* of the biases */
    const void* gate_bias;   /* DEVICE [experts][inner], or NULL */
    const void* up_bias;     /* DEVICE [experts][inner], or NULL */
    const void* down_bias;   /* DEVICE [experts][hidden], or NULL */
} nvfp4_mx_experts;

/* Bytes of workspace for so many tokens of so many choices (0 for none). */
int nvfp4_mx_moe_workspace(const nvfp4_mx_experts* layer, int64_t tokens, int64_t topk,
                           int out_type, size_t* bytes);
/*   x          : DEVICE tokens x hidden of x_type, row stride ldx (as nvfp4_mx_quantize)
 *   expert_ids : DEVICE [tokens][topk] of id_type (NVFP4_INDEX_*)
 *   weights    : DEVICE fp32 [tokens][topk], or NULL: ones; those of dropped choices are ignored
 *   out        : DEVICE tokens x hidden, overwritten; must not alias the inputs
 *   workspace  : DEVICE, 16-byte aligned, needs no initial value; free again when the call's
 *                work is done, so calls that may run at the same time need one each
 * Sizes as nvfp4_moe_sort and the products. */
int nvfp4_mx_moe(const nvfp4_mx_experts* layer, const void* x, int x_type, int64_t ldx,
                 const void* expert_ids, int id_type, const float* weights, int64_t tokens,
                 int64_t topk, void* out, int out_type, void* workspace, size_t workspace_bytes,
                 void* stream);
int nvfp4_sequence_add_mx_moe(nvfp4_sequence_t seq, const nvfp4_mx_experts* layer, const void* x,
                              int x_type, int64_t ldx, const void* expert_ids, int id_type,
                              const float* weights, int64_t tokens, int64_t topk, void* out,
                              int out_type, void* workspace, size_t workspace_bytes);

/* ---- norms around a block's residual ---------------------------------------
 *
 * Behind a block with the result y, and before the next one:
 *   u = post ? y / rms(y) * post_weight : y        rms(x) = sqrt(mean(x^2) + eps)
 *   h = residual_scale * residual + scale * gate * u
 *   n = h / rms(h) * pre_weight                     (pre)
 * by rows, in fp32; h is rounded to its type once, and n is the norm of the
 * rounded h, rounded once: the same as that norm of the stored h in a call of
 * its own.  A mean of squares past fp32's range is an infinity (values of 2^64
 * and more; such a row's norm is zeros, NaN where an infinity stood).  With an
 * eps below 1e-30, beside which small squares count, their sum has that limit
 * (values of 2^64 / sqrt(hidden)), and values below 2^-63 lose bits. */
enum { NVFP4_GATE_NONE = 0, NVFP4_GATE_CHANNEL = 1, NVFP4_GATE_ELEMENT = 2 };
#define NVFP4_NORM_MAX_HIDDEN 16384

typedef struct nvfp4_norm {
    int type;                /* NVFP4_TYPE_* of all rows */
    int weight_type;         /* NVFP4_TYPE_* of the weights and of a CHANNEL gate */
    int64_t rows, hidden;    /* 0 <= rows < 2^31, 1 <= hidden <= NVFP4_NORM_MAX_HIDDEN */
    int post, pre;           /* whether there is a norm behind the block, before the next */
    const void* post_weight; /* DEVICE [hidden], or NULL: ones */
    const void* pre_weight;
    int gate_mode;           /* NVFP4_GATE_* */
    const void* gate;        /* DEVICE; CHANNEL: [hidden], the same for every row; ELEMENT: rows x hidden
                                of `type`, row stride ld_gate; NONE: not looked at */
    int64_t ld_gate;
    float scale, residual_scale, eps;   /* eps >= 0 */
} nvfp4_norm;

/*   y, residual : DEVICE rows x hidden, row strides of at least hidden elements (a single row's
 *                 is not looked at); residual NULL: zeros
 *   h           : DEVICE rows x hidden (stride hidden), or NULL if it is not wanted; may be
 *                 residual or y itself (of stride hidden)
 *   n           : DEVICE rows x hidden (stride hidden), or NULL
 *   n_codes, n_scales : n as a packed MXFP4 operand of rows x hidden instead, the bits of
 *                 nvfp4_mx_quantize(n) (nvfp4_mx_packed_size bytes, 16-byte aligned; hidden a
 *                 multiple of 32), or both NULL
 * With `pre` n or the packed operand is wanted, without it neither, and then h is.
 * Buffers need the alignment of their elements only, but run fastest when rows start on
 * 16-byte boundaries.  Outputs must not overlap inputs otherwise. */
int nvfp4_add_norm(const nvfp4_norm* norm, const void* y, int64_t ld_y, const void* residual,
                   int64_t ld_residual, void* h, void* n, void* n_codes, void* n_scales,
                   void* stream);
int nvfp4_sequence_add_norm(nvfp4_sequence_t seq, const nvfp4_norm* norm, const void* y,
                            int64_t ld_y, const void* residual, int64_t ld_residual, void* h,
                            void* n, void* n_codes, void* n_scales);

/* Gradients of nvfp4_add_norm, for those of h (dh) and n (dn):
 *   dh, dn : DEVICE rows x hidden, row strides ld_dh, ld_dn; dh NULL: zeros; dn given exactly if
 *            `pre`
 *   y      : as given (read with `post` or a gate); h: as it came out (read with `pre`)
 * Outputs, each NULL if it is not wanted, none overlapping anything:
 *   dy, dresidual : DEVICE rows x hidden
 *   dgate         : DEVICE, CHANNEL: fp32 [hidden]; ELEMENT: rows x hidden of `type`
 *   dpost_weight, dpre_weight : DEVICE fp32 [hidden] (with `post`, `pre`)
 *   workspace     : DEVICE, 16-byte aligned, as many bytes as nvfp4_add_norm_grad_workspace
 *            says (the fp32 sums of groups of rows, which a second launch adds in order);
 *            may be NULL if that is 0 or none of dgate (CHANNEL), dpost_weight and
 *            dpre_weight is wanted.  Free again when the call's work is done; calls that may
 *            run at the same time need one each.
 * Sums over rows are fp32, in an order that depends on the sizes only. */
int nvfp4_add_norm_grad_workspace(const nvfp4_norm* norm, size_t* bytes);
int nvfp4_add_norm_grad(const nvfp4_norm* norm, const void* dh, int64_t ld_dh, const void* dn,
                        int64_t ld_dn, const void* y, int64_t ld_y, const void* h, int64_t ld_h,
                        void* dy, void* dresidual, void* dgate, float* dpost_weight,
                        float* dpre_weight, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_LAYER_H */
