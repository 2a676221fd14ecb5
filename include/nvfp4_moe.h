/*
 * nvfp4_moe.h -- C ABI of expert routing: what stands before and behind the
 * grouped products (nvfp4_grouped_gemm, nvfp4_mx_grouped_gemm) of a
 * mixture-of-experts layer, and its gradients.
 *
 * A router gives each of `tokens` tokens `topk` experts.  A choice (t, j) is
 * token t's j-th expert; an expert number outside [0, experts) means that the
 * choice was dropped (over capacity, or the expert lives elsewhere).  The
 * same expert may be chosen twice by one token.
 *
 *   nvfp4_moe_sort         choices -> row_offsets, slots, row_tokens
 *   nvfp4_moe_gather       rows of tokens -> rows in the experts' order
 *   (the experts' products)
 *   nvfp4_moe_combine      rows in the experts' order -> weighted sums of
 *                          each token's choices
 *   nvfp4_moe_combine_grad gradients of combine
 * The gradient of gather is combine without weights.
 * In the library from nvfp4_version() 10600 on.
 *
 * Element type of rows: NVFP4_TYPE_F32 or NVFP4_TYPE_BF16 (nvfp4_mx.h);
 * weights are fp32.  Rows are row-major; the rows in the experts' order are
 * contiguous (stride hidden).  Row buffers need the alignment of their
 * element type only, but run fastest when rows start on 16-byte boundaries;
 * tables are 4-byte aligned (int64 expert numbers: 8), else
 * NVFP4_ERR_MISALIGNED.
 *
 * Sizes: 0 <= tokens < 2^24 (0: nothing but row_offsets is written), 1 <=
 * topk < 2^24, tokens * topk < 2^31, 1 <= experts <= 2048, 1 <= hidden <= 2^22.
 * Status codes and streams as in nvfp4.h.  No workspace, no allocation, no
 * atomics on results: calls may be captured, may run at the same time on
 * several streams, and give the same bits every time.  Slots outside
 * [0, tokens * topk) count as dropped, so a malformed table cannot cause an
 * access outside the buffers.
 */
#ifndef NVFP4_MOE_H
#define NVFP4_MOE_H

#include "nvfp4_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of expert numbers. */
enum { NVFP4_INDEX_I32 = 0, NVFP4_INDEX_I64 = 1 };

/* Sorts the kept choices by expert, those of one expert by token and then by
 * j (stable).
 *   expert_ids  : DEVICE [tokens][topk], int32 or int64 (id_type)
 *   row_offsets : DEVICE int32[experts + 1]: expert e owns rows
 *                 row_offsets[e] .. row_offsets[e+1]-1 of the experts' order;
 *                 the last entry is the number of kept choices
 *   slots       : DEVICE int32[tokens][topk]: the row of each choice, -1 for
 *                 a dropped one
 *   row_tokens  : DEVICE int32[tokens * topk]: the token of each row, -1
 *                 behind the last kept one
 * Everything is overwritten; outputs must not alias expert_ids. */
int nvfp4_moe_sort(const void* expert_ids, int id_type, int64_t tokens, int64_t topk,
                   int64_t experts, int32_t* row_offsets, int32_t* slots, int32_t* row_tokens,
                   void* stream);

/* out[slots[t][j]] = x[t] for every kept choice.
 *   x   : DEVICE tokens x hidden, row stride ldx elements (ldx >= hidden)
 *   out : DEVICE (tokens * topk) x hidden; rows that no choice owns are left
 *         as they were; must not alias x */
int nvfp4_moe_gather(const void* x, int type, int64_t tokens, int64_t topk, int64_t hidden,
                     int64_t ldx, const int32_t* slots, void* out, void* stream);

/* out[t] = sum over the kept choices of weights[t][j] * y[slots[t][j]], summed
 * in fp32 in the order of j and rounded once; zeros for a token without any.
 *   y       : DEVICE (tokens * topk) x hidden; rows of dropped choices are
 *             not read
 *   weights : DEVICE fp32 [tokens][topk], or NULL: ones (the gradient of
 *             nvfp4_moe_gather, given the rows' gradient as y); those of
 *             dropped choices are ignored
 *   out     : DEVICE tokens x hidden (stride hidden), overwritten; must not
 *             alias y */
int nvfp4_moe_combine(const void* y, int type, int64_t tokens, int64_t topk, int64_t hidden,
                      const int32_t* slots, const float* weights, void* out, void* stream);

/* Gradients of nvfp4_moe_combine:
 *   dy[slots[t][j]]  = weights[t][j] * dout[t]        (rounded once)
 *   dweights[t][j]   = sum_h dout[t][h] * y[slots[t][j]][h]   (fp32)
 * for kept choices; dweights of dropped ones are zero, rows of dy that no
 * choice owns are left as they were.
 *   dout     : DEVICE tokens x hidden, row stride ldd elements (>= hidden)
 *   y        : DEVICE (tokens * topk) x hidden, as given to combine
 *   weights  : DEVICE fp32 [tokens][topk], or NULL: ones
 *   dy       : DEVICE (tokens * topk) x hidden; may be y itself (each element
 *              is read before it is written), no other input
 *   dweights : DEVICE fp32 [tokens][topk], overwritten; must not alias the
 *              inputs */
int nvfp4_moe_combine_grad(const void* dout, int64_t ldd, const void* y, int type,
                           int64_t tokens, int64_t topk, int64_t hidden, const int32_t* slots,
                           const float* weights, void* dy, float* dweights, void* stream);

/* The serving calls recorded into a sequence (nvfp4.h, "Recorded
 * sequences"). */
int nvfp4_sequence_add_moe_sort(nvfp4_sequence_t seq, const void* expert_ids, int id_type,
                                int64_t tokens, int64_t topk, int64_t experts,
                                int32_t* row_offsets, int32_t* slots, int32_t* row_tokens);
int nvfp4_sequence_add_moe_gather(nvfp4_sequence_t seq, const void* x, int type, int64_t tokens,
                                  int64_t topk, int64_t hidden, int64_t ldx,
                                  const int32_t* slots, void* out);
int nvfp4_sequence_add_moe_combine(nvfp4_sequence_t seq, const void* y, int type, int64_t tokens,
                                   int64_t topk, int64_t hidden, const int32_t* slots,
                                   const float* weights, void* out);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_MOE_H */
