// nvfp4_layer_api.cpp -- host side of the operators around the MXFP4 products
// of a layer (include/nvfp4_layer.h): argument checks, and the jobs that the
// eager entry points run and the sequences record.
#include <hip/hip_runtime.h>

#include "nvfp4_host.h"
#include "nvfp4_layer.h"

using namespace nvfp4;

namespace {

static_assert((int)NVFP4_ACT_NONE == kMxActNone && (int)NVFP4_ACT_RELU == kMxActRelu &&
                  (int)NVFP4_ACT_SILU == kMxActSilu && (int)NVFP4_ACT_GELU == kMxActGelu &&
                  (int)NVFP4_ACT_GELU_TANH == kMxActGeluTanh,
              "the kernels' activations are the header's");

constexpr int64_t kMaxDim = (int64_t)1 << 30;

bool valid_type(int type) { return type == NVFP4_TYPE_F32 || type == NVFP4_TYPE_BF16; }
uintptr_t size_of(int type) { return type == NVFP4_TYPE_BF16 ? 2 : 4; }
bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool valid_act(int act) { return act >= NVFP4_ACT_NONE && act <= NVFP4_ACT_GELU_TANH; }

int run(int status, const Job& job, void* stream) {
    return status != NVFP4_OK ? status : run_job(job, stream);
}

// Gives a prepared product (its status) its epilogue.
int add_epilogue(int status, const nvfp4_mx_epilogue* e, int out_type, Job* job) {
    if (status != NVFP4_OK || !e) return status;
    const MxGemmArgs& g = job->mx_gemm;
    const int64_t ld = g.M > 1 ? e->ld_residual : g.N;
    if (!valid_act(e->activation) || !e->gate_packed != !e->gate_scales ||
        (e->gate_bias && !e->gate_packed) || ((e->bias || e->gate_bias) && !valid_type(e->bias_type)) ||
        (e->residual && (ld < g.N || ld > kMaxDim)))
        return NVFP4_ERR_INVALID_VALUE;
    const uintptr_t bias_size = size_of(e->bias_type);
    if (!aligned(e->gate_packed, 16) || !aligned(e->gate_scales, 16) || !aligned(e->bias, bias_size) ||
        !aligned(e->gate_bias, bias_size) || !aligned(e->residual, size_of(out_type)))
        return NVFP4_ERR_MISALIGNED;
    MxEpilogueArgs& a = job->epilogue;
    a.gate_codes = static_cast<const uint8_t*>(e->gate_packed);
    a.gate_scales = static_cast<const uint8_t*>(e->gate_scales);
    a.bias = e->bias;
    a.gate_bias = e->gate_bias;
    a.bias_bf16 = e->bias_type == NVFP4_TYPE_BF16;
    a.residual = e->residual;
    a.ldr = ld;
    a.act = e->activation;
    if (a.gate_codes) {
        job->launch = +[](const Job& j, hipStream_t s) { return launch_mx_gated(j.mx_gemm, j.epilogue, s); };
        return job->empty || mx_gated_fits(g) ? NVFP4_OK : NVFP4_ERR_INVALID_VALUE;
    }
    job->launch = +[](const Job& j, hipStream_t s) { return launch_mx_fused(j.mx_gemm, j.epilogue, s); };
    return job->empty || mx_fused_fits(g) ? NVFP4_OK : NVFP4_ERR_INVALID_VALUE;
}

int prepare_gemm_fused(const void* a_packed, const void* a_scales, const void* b_packed,
                       const void* b_scales, float alpha, const nvfp4_mx_epilogue* e, void* out,
                       int out_type, int64_t M, int64_t N, int64_t K, Job* job) {
    const int st = prepare_mx_gemm(a_packed, a_scales, nullptr, 0, 0, M, nullptr, b_packed, b_scales,
                                   nullptr, 0, alpha, out, out_type, M, N, K, job);
    return add_epilogue(st, e, out_type, job);
}

int prepare_gemm_quantized_fused(const void* x, int x_type, int64_t ldx, const void* b_packed,
                                 const void* b_scales, float alpha, const nvfp4_mx_epilogue* e,
                                 void* out, int out_type, int64_t M, int64_t N, int64_t K, Job* job) {
    if (!x && M > 0) return NVFP4_ERR_INVALID_VALUE;
    const int st = prepare_mx_gemm(nullptr, nullptr, x, x_type, ldx, M, nullptr, b_packed, b_scales,
                                   nullptr, 0, alpha, out, out_type, M, N, K, job);
    return add_epilogue(st, e, out_type, job);
}

int prepare_grouped_fused(const void* a_packed, const void* a_scales, int64_t a_count,
                          const int32_t* a_rows, const void* b_packed, const void* b_scales,
                          const int32_t* row_offsets, int64_t groups, float alpha,
                          const nvfp4_mx_epilogue* e, void* out, int out_type, int64_t M, int64_t N,
                          int64_t K, Job* job) {
    if (!row_offsets || groups < 1 || groups > kMaxDim) return NVFP4_ERR_INVALID_VALUE;
    const int st = prepare_mx_gemm(a_packed, a_scales, nullptr, 0, 0, a_count, a_rows, b_packed,
                                   b_scales, row_offsets, groups, alpha, out, out_type, M, N, K, job);
    return add_epilogue(st, e, out_type, job);
}

}  // namespace

extern "C" {

int nvfp4_mx_gemm_fused(const void* a_packed, const void* a_scales, const void* b_packed,
                        const void* b_scales, float alpha, const nvfp4_mx_epilogue* epilogue,
                        void* out, int out_type, int64_t M, int64_t N, int64_t K, void* stream) {
    Job job;
    const int st = prepare_gemm_fused(a_packed, a_scales, b_packed, b_scales, alpha, epilogue, out,
                                      out_type, M, N, K, &job);
    return run(st, job, stream);
}

int nvfp4_mx_gemm_quantized_fused(const void* x, int x_type, int64_t ldx, const void* b_packed,
                                  const void* b_scales, float alpha,
                                  const nvfp4_mx_epilogue* epilogue, void* out, int out_type,
                                  int64_t M, int64_t N, int64_t K, void* stream) {
    Job job;
    const int st = prepare_gemm_quantized_fused(x, x_type, ldx, b_packed, b_scales, alpha, epilogue,
                                                out, out_type, M, N, K, &job);
    return run(st, job, stream);
}

int nvfp4_mx_grouped_gemm_fused(const void* a_packed, const void* a_scales, int64_t a_count,
                                const int32_t* a_rows, const void* b_packed, const void* b_scales,
                                const int32_t* row_offsets, int64_t groups, float alpha,
                                const nvfp4_mx_epilogue* epilogue, void* out, int out_type,
                                int64_t M, int64_t N, int64_t K, void* stream) {
    Job job;
    const int st = prepare_grouped_fused(a_packed, a_scales, a_count, a_rows, b_packed, b_scales,
                                         row_offsets, groups, alpha, epilogue, out, out_type, M, N,
                                         K, &job);
    return run(st, job, stream);
}

int nvfp4_sequence_add_mx_gemm_fused(nvfp4_sequence_t seq, const void* a_packed,
                                     const void* a_scales, const void* b_packed,
                                     const void* b_scales, float alpha,
                                     const nvfp4_mx_epilogue* epilogue, void* out, int out_type,
                                     int64_t M, int64_t N, int64_t K) {
    Job job;
    const int st = prepare_gemm_fused(a_packed, a_scales, b_packed, b_scales, alpha, epilogue, out,
                                      out_type, M, N, K, &job);
    return sequence_add(seq, st, job);
}

int nvfp4_sequence_add_mx_gemm_quantized_fused(nvfp4_sequence_t seq, const void* x, int x_type,
                                               int64_t ldx, const void* b_packed,
                                               const void* b_scales, float alpha,
                                               const nvfp4_mx_epilogue* epilogue, void* out,
                                               int out_type, int64_t M, int64_t N, int64_t K) {
    Job job;
    const int st = prepare_gemm_quantized_fused(x, x_type, ldx, b_packed, b_scales, alpha, epilogue,
                                                out, out_type, M, N, K, &job);
    return sequence_add(seq, st, job);
}

int nvfp4_sequence_add_mx_grouped_gemm_fused(nvfp4_sequence_t seq, const void* a_packed,
                                             const void* a_scales, int64_t a_count,
                                             const int32_t* a_rows, const void* b_packed,
                                             const void* b_scales, const int32_t* row_offsets,
                                             int64_t groups, float alpha,
                                             const nvfp4_mx_epilogue* epilogue, void* out,
                                             int out_type, int64_t M, int64_t N, int64_t K) {
    Job job;
    const int st = prepare_grouped_fused(a_packed, a_scales, a_count, a_rows, b_packed, b_scales,
                                         row_offsets, groups, alpha, epilogue, out, out_type, M, N,
                                         K, &job);
    return sequence_add(seq, st, job);
}

}  // extern "C"
