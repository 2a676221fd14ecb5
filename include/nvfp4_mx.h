/*
 * nvfp4_mx.h -- C ABI of the MXFP4 operators of the library: quantisation,
 * its inverse, the product C = alpha * (A . B^T) and its grouped form.
 *
 * MXFP4 (OCP Microscaling Formats v1.0) holds 32 consecutive elements of a
 * row as FP4 E2M1 codes under one E8M0 scale byte e: element = code value *
 * 2^(e - 127); e = 255 makes the whole block NaN.  Codes as in nvfp4.h:
 * sign(bit 3) | exponent(bits 2:1, bias 1) | mantissa(bit 0), values
 * +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}.  gfx950 multiplies this format directly,
 * so its product runs at the matrix cores' FP4 rate (the 16-element E4M3
 * blocks of nvfp4.h are decoded to fp16 first).
 *
 * Canonical layout (what checkpoints hold; row-major, K contiguous):
 *   codes  [rows][K/2]   byte j of a row holds element 2j in bits 3:0 and
 *                        element 2j+1 in bits 7:4;
 *   scales [rows][K/32]  byte b scales elements 32b .. 32b+31.
 * Packed layout (what the product consumes; made by nvfp4_mx_pack on the
 * host or nvfp4_mx_quantize on the device).  Rows are padded to whole row
 * blocks of 16 (RB of them) and K to whole steps of 128 (C of them) with zero
 * codes and zero scale bytes (exact zeros, so results are unaffected):
 *   packed codes  [RB][C][16][4][16]   (row block, step, row of the row
 *                                       block, place in the row's 64 bytes,
 *                                       16 code bytes): block b (0..3) of a
 *                                       step of row r is at place b ^ (r / 4)
 *   packed scales [RB][ceil(C/4)][16][4][4]  (row block, four steps, row,
 *                                       block of a step, the four steps'
 *                                       bytes)
 * The 1024 code bytes of 16 rows x 128 elements are what one wave feeds to
 * one matrix instruction; a row's 64 of them are contiguous, so that rows can
 * be picked one by one, and the places are such that the lanes of a wave
 * read them from LDS without bank conflicts.
 *
 * In the library from nvfp4_version() 10600 on.
 *
 * Status codes, pointers, streams and errors as in nvfp4.h: every entry point
 * returns an nvfp4_status and never aborts, throws or prints; argument errors
 * are detected on the host before any device work; device buffers are
 * caller-owned and 16-byte aligned (else NVFP4_ERR_MISALIGNED); calls are
 * asynchronous on `stream`.  No entry point here uses a workspace or
 * allocates, so all of them may be captured into graphs and may run at the
 * same time on several streams.  The current device must be the one that the
 * buffers are on.
 *
 * Sizes: rows and M from 0 (nothing is launched) and N from 1 to 2^30, K a
 * positive multiple of 32 up to 2^30.  A call that would take more work-items
 * than one launch holds (2^32) is refused with NVFP4_ERR_INVALID_VALUE: groups
 * x row blocks x steps from about 2^26 when quantising, N from about 2^26 in a
 * product of up to 16 packed rows.
 */
#ifndef NVFP4_MX_H
#define NVFP4_MX_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of unquantised rows (same values as NVFP4_INPUT_*). */
enum { NVFP4_TYPE_F32 = 0, NVFP4_TYPE_BF16 = 1 };

/* Byte sizes of the packed buffers of a rows x K operand. */
int nvfp4_mx_packed_size(int64_t rows, int64_t K, size_t* code_bytes, size_t* scale_bytes);

/* Host-side layout transform, canonical -> packed, and its inverse (which
 * drops the padding): byte permutations, no arithmetic.  HOST memory,
 * caller-owned, no alignment required. */
int nvfp4_mx_pack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                  uint8_t* packed_codes, uint8_t* packed_scales);
int nvfp4_mx_unpack(const uint8_t* packed_codes, const uint8_t* packed_scales, int64_t rows,
                    int64_t K, uint8_t* codes, uint8_t* scales);

/* MXFP4 quantisation into the packed layout.  Per block of 32 elements:
 *   scale byte = max(0, floor(log2(max |x|)) - 2 + 127)   (0 for a zero block)
 *   code       = E2M1 value nearest to x / 2^(byte - 127), ties to the even
 *                code, saturating at 6, with the sign bit of x
 * and a block that holds an infinity or a NaN gets scale byte 255 and zero
 * codes: it reads as NaN, and so do the results that it enters.
 *   x            : DEVICE, `groups` matrices of rows x K values of type
 *                  x_type (NVFP4_TYPE_F32 or NVFP4_TYPE_BF16), row stride ld
 *                  and group stride group_stride elements: ld >= K, both
 *                  multiples of 4 (fp32) or 8 (bfloat16); a single row's or
 *                  group's stride is not looked at
 *   packed_codes,
 *   packed_scales: DEVICE, groups x nvfp4_mx_packed_size(rows, K) bytes
 *                  (group g at g times those); every byte is written
 * groups = 1 for a single operand; several are the weights of the grouped
 * product. */
int nvfp4_mx_quantize(const void* x, int x_type, int64_t groups, int64_t group_stride,
                      int64_t rows, int64_t K, int64_t ld, void* packed_codes,
                      void* packed_scales, void* stream);

/* The values that packed operands stand for, as fp32 or bfloat16 rows.  Exact
 * in both (a code has two significant bits), but that values from 2^128 on are
 * infinities: codes of 4 and more under scale byte 253, of 2 and more under 254,
 * which no finite input is quantised to.  NaN for blocks with scale 255.
 * Buffers and strides as nvfp4_mx_quantize (group_stride >= K: groups must not
 * overlap); writes the rows x K elements of every group and nothing between
 * them. */
int nvfp4_mx_dequantize(const void* packed_codes, const void* packed_scales, int64_t groups,
                        int64_t rows, int64_t K, void* x, int x_type, int64_t group_stride,
                        int64_t ld, void* stream);

/* C = alpha * (A . B^T), fp32 sums, alpha applied once, then rounded to
 * nearest even if out_type is NVFP4_TYPE_BF16 (NVFP4_TYPE_F32: stored as it
 * is).
 *   a_packed, a_scales, b_packed, b_scales : DEVICE, packed A (M rows) and B
 *              (N rows) of depth K
 *   out      : DEVICE, M x N, row-major (ld = N), overwritten; must not alias
 *              the inputs
 * Deterministic: the order of the additions depends on the sizes only. */
int nvfp4_mx_gemm(const void* a_packed, const void* a_scales, const void* b_packed,
                  const void* b_scales, float alpha, void* out, int out_type, int64_t M,
                  int64_t N, int64_t K, void* stream);

/* nvfp4_mx_gemm(nvfp4_mx_quantize(X), B) in one launch, bit for bit, for
 * decode steps, where a second launch costs as much as the product.  Up to K =
 * 8192 it is the faster form; behind that every 16 columns quantise the rows
 * again, which takes about N * K * (6 + M) / 2e8 us and pays while that is less
 * than a launch.
 *   x : DEVICE, M x K values of x_type, row stride ldx elements (as
 *       nvfp4_mx_quantize); M is at most 16 (NVFP4_ERR_UNSUPPORTED above) */
int nvfp4_mx_gemm_quantized(const void* x, int x_type, int64_t ldx, const void* b_packed,
                            const void* b_scales, float alpha, void* out, int out_type,
                            int64_t M, int64_t N, int64_t K, void* stream);

/* Grouped product of a mixture-of-experts layer, as nvfp4_grouped_gemm:
 * group g owns rows row_offsets[g] .. row_offsets[g+1]-1 of C and multiplies
 * by its own operand B_g,
 *   C[r][n] = alpha * sum_k a'[A_row(r)][k] * b'_g[n][k].
 *   a_packed, a_scales : DEVICE, A of a_count rows
 *   a_rows      : DEVICE int32[M], the row of A of each row of C (a router's
 *                 tokens in the experts' order, nvfp4_moe.h: each token's
 *                 activations are quantised once and read where they are), or
 *                 NULL: row r itself, and a_count must be M
 *   b_packed, b_scales : DEVICE, `groups` operands of N x K, concatenated
 *   row_offsets : DEVICE int32[groups + 1], non-decreasing, from 0 to at most
 *                 M
 *   out         : DEVICE, M x N; rows of every group are overwritten, rows
 *                 behind the last group are left as they were
 * Entries of row_offsets are clamped to [0, M] and of
 * a_rows to A's rows: a malformed table gives wrong rows, no access outside
 * the buffers (overlapping groups may then write the same rows).
 * NVFP4_ERR_MISALIGNED unless the tables are 4-byte aligned.
 * Fast while A's packed codes are less than 2 GiB; from there on a kernel
 * without 32-bit offsets runs, which reads the weights again for every 32 rows
 * (8 groups x 256 x 8192, 524272 rows: 0.66 ms, 524304 rows: 8.9 ms): split the
 * groups over calls. */
int nvfp4_mx_grouped_gemm(const void* a_packed, const void* a_scales, int64_t a_count,
                          const int32_t* a_rows, const void* b_packed, const void* b_scales,
                          const int32_t* row_offsets, int64_t groups, float alpha, void* out,
                          int out_type, int64_t M, int64_t N, int64_t K, void* stream);

/* The same calls recorded into a sequence (nvfp4.h, "Recorded sequences"). */
int nvfp4_sequence_add_mx_quantize(nvfp4_sequence_t seq, const void* x, int x_type,
                                   int64_t rows, int64_t K, int64_t ld, void* packed_codes,
                                   void* packed_scales);
int nvfp4_sequence_add_mx_gemm(nvfp4_sequence_t seq, const void* a_packed, const void* a_scales,
                               const void* b_packed, const void* b_scales, float alpha,
                               void* out, int out_type, int64_t M, int64_t N, int64_t K);
int nvfp4_sequence_add_mx_gemm_quantized(nvfp4_sequence_t seq, const void* x, int x_type,
                                         int64_t ldx, const void* b_packed,
                                         const void* b_scales, float alpha, void* out,
                                         int out_type, int64_t M, int64_t N, int64_t K);
int nvfp4_sequence_add_mx_grouped_gemm(nvfp4_sequence_t seq, const void* a_packed,
                                       const void* a_scales, int64_t a_count,
                                       const int32_t* a_rows, const void* b_packed,
                                       const void* b_scales, const int32_t* row_offsets,
                                       int64_t groups, float alpha, void* out, int out_type,
                                       int64_t M, int64_t N, int64_t K);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_MX_H */
