// nvfp4_mx_api.cpp -- host side of the MXFP4 operators and of the expert
// routing (include/nvfp4_mx.h, include/nvfp4_moe.h): argument checks, the
// canonical <-> packed layout transform, and the jobs that the eager entry
// points run and the sequences record.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstring>

#include "nvfp4_host.h"
#include "nvfp4_moe.h"
#include "nvfp4_mx.h"

using namespace nvfp4;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 30;
// work-items of a launch along one grid dimension
constexpr int64_t kMaxItems = ((int64_t)1 << 32) - 1;

bool valid_rows_k(int64_t rows, int64_t K) {
    return rows >= 0 && rows <= kMaxDim && K >= kMxBlock && K <= kMaxDim && K % kMxBlock == 0;
}
bool valid_type(int type) { return type == NVFP4_TYPE_F32 || type == NVFP4_TYPE_BF16; }
bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

}  // namespace

namespace nvfp4 {

int prepare_mx_quantize(bool inverse, const void* x, int x_type, int64_t groups,
                        int64_t group_stride, int64_t rows, int64_t K, int64_t ld, void* codes,
                        void* scales, Job* job) {
    const bool empty = groups == 0 || rows == 0;
    if ((!empty && (!x || !codes || !scales)) || !valid_type(x_type) || groups < 0 ||
        !valid_rows_k(rows, K))
        return NVFP4_ERR_INVALID_VALUE;
    const int64_t per16 = x_type == NVFP4_TYPE_BF16 ? 8 : 4;  // elements in 16 bytes
    // (strides that nothing is reached by are not looked at)
    if (rows <= 1) ld = K;
    if (groups <= 1) group_stride = 0;
    if (ld < K || ld % per16 || group_stride < 0 || group_stride % per16)
        return NVFP4_ERR_INVALID_VALUE;
    if (inverse && groups > 1 && group_stride < K) return NVFP4_ERR_INVALID_VALUE;  // would overlap
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16)) return NVFP4_ERR_MISALIGNED;
    const int64_t RB = mx_row_blocks(rows), C = mx_steps(K);
    // (a wave per fragment; groups * RB * C cannot wrap: each factor is checked first)
    const int64_t most = kMaxItems / 64 - 4;
    if (!empty && (groups > most || RB > most / groups || C > most / (groups * RB)))
        return NVFP4_ERR_INVALID_VALUE;
    *job = Job{};
    job->kind = JOB_LAUNCH;
    job->empty = empty;
    job->launch = inverse ? +[](const Job& j, hipStream_t s) { return launch_mx_dequantize(j.mx_quant, s); }
                          : +[](const Job& j, hipStream_t s) { return launch_mx_quantize(j.mx_quant, s); };
    MxQuantArgs& a = job->mx_quant;
    a.x = const_cast<void*>(x);
    a.bf16 = x_type == NVFP4_TYPE_BF16;
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = static_cast<uint8_t*>(scales);
    a.group_stride = group_stride;
    a.ld = ld;
    a.groups = groups;
    a.rows = (int)rows;
    a.K = (int)K;
    a.RB = (int)RB;
    a.C = (int)C;
    return NVFP4_OK;
}

int prepare_mx_gemm(const void* a_packed, const void* a_scales, const void* x, int x_type,
                    int64_t ldx, int64_t a_count, const int32_t* a_rows, const void* b_packed,
                    const void* b_scales, const int32_t* row_offsets, int64_t groups, float alpha,
                    void* out, int out_type, int64_t M, int64_t N, int64_t K, Job* job) {
    const bool grouped = groups > 0;
    if (M < 0 || M > kMaxDim || N < 1 || !valid_rows_k(N, K) || !valid_type(out_type) ||
        !valid_type(x_type))
        return NVFP4_ERR_INVALID_VALUE;
    if (!b_packed || !b_scales || (M > 0 && (!out || (!x && (!a_packed || !a_scales)))))
        return NVFP4_ERR_INVALID_VALUE;
    if (grouped && (a_count < (M > 0) || a_count > kMaxDim || (!a_rows && a_count != M)))
        return NVFP4_ERR_INVALID_VALUE;
    if (x) {
        const int64_t per16 = x_type == NVFP4_TYPE_BF16 ? 8 : 4;
        if (M <= 1) ldx = K;
        if (ldx < K || ldx % per16) return NVFP4_ERR_INVALID_VALUE;
    }
    if (!aligned(a_packed, 16) || !aligned(a_scales, 16) || !aligned(x, 16) ||
        !aligned(b_packed, 16) || !aligned(b_scales, 16) || !aligned(out, 16) ||
        !aligned(row_offsets, 4) || !aligned(a_rows, 4))
        return NVFP4_ERR_MISALIGNED;
    if (x && M > kMxQuantRows) return NVFP4_ERR_UNSUPPORTED;
    *job = Job{};
    job->kind = JOB_LAUNCH;
    job->empty = M == 0;
    job->launch = +[](const Job& j, hipStream_t s) { return launch_mx_gemm(j.mx_gemm, s); };
    MxGemmArgs& g = job->mx_gemm;
    g.a_codes = static_cast<const uint8_t*>(a_packed);
    g.a_scales = static_cast<const uint8_t*>(a_scales);
    g.x = x;
    g.x_bf16 = x_type == NVFP4_TYPE_BF16;
    g.ldx = ldx;
    g.b_codes = static_cast<const uint8_t*>(b_packed);
    g.b_scales = static_cast<const uint8_t*>(b_scales);
    g.offsets = row_offsets;
    g.a_rows = a_rows;
    g.out = out;
    g.out_bf16 = out_type == NVFP4_TYPE_BF16;
    g.alpha = alpha;
    g.M = (int)M;
    g.N = (int)N;
    g.K = (int)K;
    g.A_rows = (int)(grouped ? a_count : M);
    g.RBa = (int)mx_row_blocks(g.A_rows);
    g.RBb = (int)mx_row_blocks(N);
    g.C = (int)mx_steps(K);
    g.groups = (int)groups;
    // the launch must fit a grid: the kernel that the sizes choose tells
    return job->empty || mx_gemm_fits(g) ? NVFP4_OK : NVFP4_ERR_INVALID_VALUE;
}

}  // namespace nvfp4

namespace {

int prepare_moe(int64_t tokens, int64_t topk, Job* job) {
    if (tokens < 0 || tokens >= ((int64_t)1 << 24) || topk < 1 || topk >= ((int64_t)1 << 24) ||
        tokens * topk > INT32_MAX)
        return NVFP4_ERR_INVALID_VALUE;
    *job = Job{};
    job->kind = JOB_LAUNCH;
    job->moe.tokens = tokens;
    job->moe.topk = (int)topk;
    return NVFP4_OK;
}

}  // namespace

namespace nvfp4 {

int prepare_moe_sort(const void* ids, int id_type, int64_t tokens, int64_t topk, int64_t experts,
                     int32_t* row_offsets, int32_t* slots, int32_t* row_tokens, Job* job) {
    if (!row_offsets || (tokens > 0 && (!ids || !slots || !row_tokens)) || experts < 1 ||
        experts > kMoeMaxExperts || (id_type != NVFP4_INDEX_I32 && id_type != NVFP4_INDEX_I64))
        return NVFP4_ERR_INVALID_VALUE;
    const int st = prepare_moe(tokens, topk, job);
    if (st != NVFP4_OK) return st;
    if (!aligned(ids, id_type == NVFP4_INDEX_I64 ? 8 : 4) || !aligned(row_offsets, 4) ||
        !aligned(slots, 4) || !aligned(row_tokens, 4))
        return NVFP4_ERR_MISALIGNED;
    MoeArgs& a = job->moe;
    a.ids = ids;
    a.wide = id_type == NVFP4_INDEX_I64;
    a.experts = (int)experts;
    a.row_offsets = row_offsets;
    a.slots = slots;
    a.row_tokens = row_tokens;
    job->launch = +[](const Job& j, hipStream_t s) { return launch_moe_sort(j.moe, s); };
    return NVFP4_OK;
}

}  // namespace nvfp4

namespace {

// The row operators: x and out, and for the gradient y and dweights.
int prepare_moe_rows(const void* x, const void* y, int type, int64_t tokens, int64_t topk,
                     int64_t hidden, int64_t ld, const int32_t* slots, const float* weights,
                     void* out, float* dweights, bool grad, Job* job) {
    if (!valid_type(type) || hidden < 1 || hidden > ((int64_t)1 << 22) ||
        (tokens > 0 && (!x || !slots || !out || (grad && (!y || !dweights)))) ||
        (tokens > 1 && (ld < hidden || ld > kMaxDim)))
        return NVFP4_ERR_INVALID_VALUE;
    const int st = prepare_moe(tokens, topk, job);
    if (st != NVFP4_OK) return st;
    const uintptr_t size = type == NVFP4_TYPE_BF16 ? 2 : 4;
    if (!aligned(x, size) || !aligned(y, size) || !aligned(out, size) || !aligned(slots, 4) ||
        !aligned(weights, 4) || !aligned(dweights, 4))
        return NVFP4_ERR_MISALIGNED;
    MoeArgs& a = job->moe;
    a.bf16 = type == NVFP4_TYPE_BF16;
    a.hidden = hidden;
    a.ld_in = tokens > 1 ? ld : hidden;
    a.slots = const_cast<int32_t*>(slots);
    a.x = x;
    a.y = y;
    a.weights = weights;
    a.out = out;
    a.dweights = dweights;
    job->empty = tokens == 0;
    return NVFP4_OK;
}

int prepare_moe_gather(const void* x, int type, int64_t tokens, int64_t topk, int64_t hidden,
                       int64_t ldx, const int32_t* slots, void* out, Job* job) {
    const int st = prepare_moe_rows(x, nullptr, type, tokens, topk, hidden, ldx, slots, nullptr, out,
                                    nullptr, false, job);
    if (st == NVFP4_OK)
        job->launch = +[](const Job& j, hipStream_t s) { return launch_moe_gather(j.moe, s); };
    return st;
}

}  // namespace

namespace nvfp4 {

int prepare_moe_combine(const void* y, int type, int64_t tokens, int64_t topk, int64_t hidden,
                        const int32_t* slots, const float* weights, void* out, Job* job) {
    const int st = prepare_moe_rows(y, nullptr, type, tokens, topk, hidden, hidden, slots, weights,
                                    out, nullptr, false, job);
    if (st == NVFP4_OK)
        job->launch = +[](const Job& j, hipStream_t s) { return launch_moe_combine(j.moe, s); };
    return st;
}

}  // namespace nvfp4

namespace {

int run(int status, const Job& job, void* stream) {
    return status != NVFP4_OK ? status : run_job(job, stream);
}

}  // namespace

extern "C" {

int nvfp4_mx_packed_size(int64_t rows, int64_t K, size_t* code_bytes, size_t* scale_bytes) {
    if (!code_bytes || !scale_bytes || !valid_rows_k(rows, K)) return NVFP4_ERR_INVALID_VALUE;
    const int64_t RB = mx_row_blocks(rows), C = mx_steps(K);
    *code_bytes = (size_t)(RB * C * kMxFrag);
    *scale_bytes = (size_t)(RB * ((C + 3) / 4) * kMxScaleFrag);
    return NVFP4_OK;
}

int nvfp4_mx_pack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t K,
                  uint8_t* packed_codes, uint8_t* packed_scales) {
    if (!codes || !scales || !packed_codes || !packed_scales || !valid_rows_k(rows, K))
        return NVFP4_ERR_INVALID_VALUE;
    const int64_t RB = mx_row_blocks(rows), C = mx_steps(K), Q = (C + 3) / 4;
    const int64_t blocks = K / kMxBlock;
    for (int64_t rb = 0; rb < RB; ++rb)
        for (int64_t b = 0; b < Q * 16; ++b) {  // blocks of a row, up to whole scale words
            const int64_t c = b / 4, kg = b % 4;
            for (int64_t r = 0; r < kMxRows; ++r) {
                const int64_t row = rb * kMxRows + r;
                const bool live = row < rows && b < blocks;
                if (c < C) {
                    uint8_t* d = packed_codes + (rb * C + c) * kMxFrag + mx_code_at((int)r, (int)kg);
                    if (live)
                        std::memcpy(d, codes + row * (K / 2) + b * 16, 16);
                    else
                        std::memset(d, 0, 16);
                }
                packed_scales[(rb * Q + c / 4) * kMxScaleFrag + mx_scale_at((int)r, (int)kg) + c % 4] =
                    live ? scales[row * blocks + b] : 0;
            }
        }
    return NVFP4_OK;
}

int nvfp4_mx_unpack(const uint8_t* packed_codes, const uint8_t* packed_scales, int64_t rows,
                    int64_t K, uint8_t* codes, uint8_t* scales) {
    if (!codes || !scales || !packed_codes || !packed_scales || !valid_rows_k(rows, K))
        return NVFP4_ERR_INVALID_VALUE;
    const int64_t C = mx_steps(K), Q = (C + 3) / 4, blocks = K / kMxBlock;
    for (int64_t row = 0; row < rows; ++row) {
        const int64_t rb = row / kMxRows, r = row % kMxRows;
        for (int64_t b = 0; b < blocks; ++b) {
            const int64_t c = b / 4, kg = b % 4;
            std::memcpy(codes + row * (K / 2) + b * 16,
                        packed_codes + (rb * C + c) * kMxFrag + mx_code_at((int)r, (int)kg), 16);
            scales[row * blocks + b] =
                packed_scales[(rb * Q + c / 4) * kMxScaleFrag + mx_scale_at((int)r, (int)kg) + c % 4];
        }
    }
    return NVFP4_OK;
}

int nvfp4_mx_quantize(const void* x, int x_type, int64_t groups, int64_t group_stride,
                      int64_t rows, int64_t K, int64_t ld, void* packed_codes,
                      void* packed_scales, void* stream) {
    Job job;
    const int st = prepare_mx_quantize(false, x, x_type, groups, group_stride, rows, K, ld,
                                       packed_codes, packed_scales, &job);
    return run(st, job, stream);
}

int nvfp4_mx_dequantize(const void* packed_codes, const void* packed_scales, int64_t groups,
                        int64_t rows, int64_t K, void* x, int x_type, int64_t group_stride,
                        int64_t ld, void* stream) {
    Job job;
    const int st = prepare_mx_quantize(true, x, x_type, groups, group_stride, rows, K, ld,
                                       const_cast<void*>(packed_codes),
                                       const_cast<void*>(packed_scales), &job);
    return run(st, job, stream);
}

int nvfp4_mx_gemm(const void* a_packed, const void* a_scales, const void* b_packed,
                  const void* b_scales, float alpha, void* out, int out_type, int64_t M,
                  int64_t N, int64_t K, void* stream) {
    Job job;
    const int st = prepare_mx_gemm(a_packed, a_scales, nullptr, 0, 0, M, nullptr, b_packed, b_scales,
                                   nullptr, 0, alpha, out, out_type, M, N, K, &job);
    return run(st, job, stream);
}

int nvfp4_mx_gemm_quantized(const void* x, int x_type, int64_t ldx, const void* b_packed,
                            const void* b_scales, float alpha, void* out, int out_type,
                            int64_t M, int64_t N, int64_t K, void* stream) {
    if (!x && M > 0) return NVFP4_ERR_INVALID_VALUE;
    Job job;
    const int st = prepare_mx_gemm(nullptr, nullptr, x, x_type, ldx, M, nullptr, b_packed, b_scales,
                                   nullptr, 0, alpha, out, out_type, M, N, K, &job);
    return run(st, job, stream);
}

int nvfp4_mx_grouped_gemm(const void* a_packed, const void* a_scales, int64_t a_count,
                          const int32_t* a_rows, const void* b_packed, const void* b_scales,
                          const int32_t* row_offsets, int64_t groups, float alpha, void* out,
                          int out_type, int64_t M, int64_t N, int64_t K, void* stream) {
    if (!row_offsets || groups < 1 || groups > kMaxDim) return NVFP4_ERR_INVALID_VALUE;
    Job job;
    const int st = prepare_mx_gemm(a_packed, a_scales, nullptr, 0, 0, a_count, a_rows, b_packed,
                                   b_scales, row_offsets, groups, alpha, out, out_type, M, N, K,
                                   &job);
    return run(st, job, stream);
}

int nvfp4_sequence_add_mx_quantize(nvfp4_sequence_t seq, const void* x, int x_type,
                                   int64_t rows, int64_t K, int64_t ld, void* packed_codes,
                                   void* packed_scales) {
    Job job;
    const int st = prepare_mx_quantize(false, x, x_type, 1, 0, rows, K, ld, packed_codes,
                                       packed_scales, &job);
    return sequence_add(seq, st, job);
}

int nvfp4_sequence_add_mx_gemm(nvfp4_sequence_t seq, const void* a_packed, const void* a_scales,
                               const void* b_packed, const void* b_scales, float alpha,
                               void* out, int out_type, int64_t M, int64_t N, int64_t K) {
    Job job;
    const int st = prepare_mx_gemm(a_packed, a_scales, nullptr, 0, 0, M, nullptr, b_packed, b_scales,
                                   nullptr, 0, alpha, out, out_type, M, N, K, &job);
    return sequence_add(seq, st, job);
}

int nvfp4_sequence_add_mx_gemm_quantized(nvfp4_sequence_t seq, const void* x, int x_type,
                                         int64_t ldx, const void* b_packed,
                                         const void* b_scales, float alpha, void* out,
                                         int out_type, int64_t M, int64_t N, int64_t K) {
    if (!x && M > 0) return NVFP4_ERR_INVALID_VALUE;
    Job job;
    const int st = prepare_mx_gemm(nullptr, nullptr, x, x_type, ldx, M, nullptr, b_packed, b_scales,
                                   nullptr, 0, alpha, out, out_type, M, N, K, &job);
    return sequence_add(seq, st, job);
}

int nvfp4_sequence_add_mx_grouped_gemm(nvfp4_sequence_t seq, const void* a_packed,
                                       const void* a_scales, int64_t a_count,
                                       const int32_t* a_rows, const void* b_packed,
                                       const void* b_scales, const int32_t* row_offsets,
                                       int64_t groups, float alpha, void* out, int out_type,
                                       int64_t M, int64_t N, int64_t K) {
    if (!row_offsets || groups < 1 || groups > kMaxDim) return NVFP4_ERR_INVALID_VALUE;
    Job job;
    const int st = prepare_mx_gemm(a_packed, a_scales, nullptr, 0, 0, a_count, a_rows, b_packed,
                                   b_scales, row_offsets, groups, alpha, out, out_type, M, N, K,
                                   &job);
    return sequence_add(seq, st, job);
}

int nvfp4_moe_sort(const void* expert_ids, int id_type, int64_t tokens, int64_t topk,
                   int64_t experts, int32_t* row_offsets, int32_t* slots, int32_t* row_tokens,
                   void* stream) {
    Job job;
    const int st = prepare_moe_sort(expert_ids, id_type, tokens, topk, experts, row_offsets, slots,
                                    row_tokens, &job);
    return run(st, job, stream);
}

int nvfp4_moe_gather(const void* x, int type, int64_t tokens, int64_t topk, int64_t hidden,
                     int64_t ldx, const int32_t* slots, void* out, void* stream) {
    Job job;
    const int st = prepare_moe_gather(x, type, tokens, topk, hidden, ldx, slots, out, &job);
    return run(st, job, stream);
}

int nvfp4_moe_combine(const void* y, int type, int64_t tokens, int64_t topk, int64_t hidden,
                      const int32_t* slots, const float* weights, void* out, void* stream) {
    Job job;
    const int st = prepare_moe_combine(y, type, tokens, topk, hidden, slots, weights, out, &job);
    return run(st, job, stream);
}

int nvfp4_moe_combine_grad(const void* dout, int64_t ldd, const void* y, int type,
                           int64_t tokens, int64_t topk, int64_t hidden, const int32_t* slots,
                           const float* weights, void* dy, float* dweights, void* stream) {
    Job job;
    const int st = prepare_moe_rows(dout, y, type, tokens, topk, hidden, ldd, slots, weights, dy,
                                    dweights, true, &job);
    if (st == NVFP4_OK)
        job.launch = +[](const Job& j, hipStream_t s) { return launch_moe_combine_grad(j.moe, s); };
    return run(st, job, stream);
}

int nvfp4_sequence_add_moe_sort(nvfp4_sequence_t seq, const void* expert_ids, int id_type,
                                int64_t tokens, int64_t topk, int64_t experts,
                                int32_t* row_offsets, int32_t* slots, int32_t* row_tokens) {
    Job job;
    const int st = prepare_moe_sort(expert_ids, id_type, tokens, topk, experts, row_offsets, slots,
                                    row_tokens, &job);
    return sequence_add(seq, st, job);
}

int nvfp4_sequence_add_moe_gather(nvfp4_sequence_t seq, const void* x, int type, int64_t tokens,
                                  int64_t topk, int64_t hidden, int64_t ldx,
                                  const int32_t* slots, void* out) {
    Job job;
    const int st = prepare_moe_gather(x, type, tokens, topk, hidden, ldx, slots, out, &job);
    return sequence_add(seq, st, job);
}

int nvfp4_sequence_add_moe_combine(nvfp4_sequence_t seq, const void* y, int type, int64_t tokens,
                                   int64_t topk, int64_t hidden, const int32_t* slots,
                                   const float* weights, void* out) {
    Job job;
    const int st = prepare_moe_combine(y, type, tokens, topk, hidden, slots, weights, out, &job);
    return sequence_add(seq, st, job);
}

}  // extern "C"
