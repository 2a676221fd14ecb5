// nvfp4_layer_api.cpp -- host side of the operators around the MXFP4 products
// of a layer (include/nvfp4_layer.h): argument checks, and the jobs that the
// eager entry points run and the sequences record.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "nvfp4_host.h"
#include "nvfp4_layer.h"

using namespace nvfp4;

namespace {

static_assert((int)NVFP4_ACT_NONE == kMxActNone && (int)NVFP4_ACT_RELU == kMxActRelu &&
                  (int)NVFP4_ACT_SILU == kMxActSilu && (int)NVFP4_ACT_GELU == kMxActGelu &&
                  (int)NVFP4_ACT_GELU_TANH == kMxActGeluTanh,
              "the kernels' activations are the header's");
static_assert((int)NVFP4_GATE_CHANNEL == kGateChannel && (int)NVFP4_GATE_ELEMENT == kGateElement &&
                  NVFP4_NORM_MAX_HIDDEN == kNormMaxHidden,
              "and so are the gates and the rows' length");

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

// ---- a whole layer of experts -------------------------------------------------

int check_experts(const nvfp4_mx_experts* l, int64_t tokens, int64_t topk, int out_type) {
    auto valid_depth = [](int64_t K) { return K >= kMxBlock && K <= kMaxDim && K % kMxBlock == 0; };
    if (!l || l->experts < 1 || l->experts > kMoeMaxExperts || !valid_depth(l->hidden) || !valid_depth(l->inner) ||
        l->hidden > ((int64_t)1 << 22) || !valid_act(l->activation) || !valid_type(out_type) || tokens < 0 ||
        tokens >= ((int64_t)1 << 24) || topk < 1 || topk >= ((int64_t)1 << 24) || tokens * topk > kMaxDim)
        return NVFP4_ERR_INVALID_VALUE;
    return NVFP4_OK;
}

// The workspace, part by part.
struct MoeSpace {
    size_t bytes = 0;
    size_t take(int64_t n, size_t size) {
        const size_t at = bytes;
        bytes += ((size_t)n * size + 255) / 256 * 256;
        return at;
    }
    size_t h = 0, offsets = 0, slots = 0, row_tokens = 0, x_codes = 0, x_scales = 0, h_codes = 0, h_scales = 0, y = 0;
    MoeSpace(const nvfp4_mx_experts& l, int64_t tokens, int64_t topk) {
        const int64_t pairs = tokens * topk;
        if (pairs == 0) return;
        h = take(pairs * l.inner, 2);
        if (mx_moe_few(tokens, topk, l.hidden, l.inner)) return;
        auto packed = [&](int64_t rows, int64_t K, size_t* codes, size_t* scales) {
            const int64_t rb = mx_row_blocks(rows), c = mx_steps(K);
            *codes = take(rb * c, kMxFrag);
            *scales = take(rb * ((c + 3) / 4), kMxScaleFrag);
        };
        packed(tokens, l.hidden, &x_codes, &x_scales);
        packed(pairs, l.inner, &h_codes, &h_scales);
        offsets = take(l.experts + 1, 4);
        slots = take(pairs, 4);
        row_tokens = take(pairs, 4);
        y = take(pairs * l.hidden, 4);
    }
};

constexpr int kMoeJobs = 6;

int prepare_mx_moe(const nvfp4_mx_experts* l, const void* x, int x_type, int64_t ldx, const void* ids,
                   int id_type, const float* weights, int64_t tokens, int64_t topk, void* out, int out_type,
                   void* workspace, size_t workspace_bytes, Job* jobs, int* count) {
    *count = 0;
    int st = check_experts(l, tokens, topk, out_type);
    if (st != NVFP4_OK) return st;
    if (!valid_type(x_type) || (id_type != NVFP4_INDEX_I32 && id_type != NVFP4_INDEX_I64) ||
        !l->gate_packed != !l->gate_scales || !l->up_packed || !l->up_scales || !l->down_packed || !l->down_scales ||
        (l->gate_bias && !l->gate_packed) ||
        ((l->gate_bias || l->up_bias || l->down_bias) && !valid_type(l->bias_type)))
        return NVFP4_ERR_INVALID_VALUE;
    const int64_t per16 = x_type == NVFP4_TYPE_BF16 ? 8 : 4;
    if (tokens <= 1) ldx = l->hidden;
    if (ldx < l->hidden || ldx > kMaxDim || ldx % per16) return NVFP4_ERR_INVALID_VALUE;
    const MoeSpace at(*l, tokens, topk);
    if (tokens > 0 && (!x || !ids || !out || !workspace || workspace_bytes < at.bytes)) return NVFP4_ERR_INVALID_VALUE;
    const uintptr_t bias_size = size_of(l->bias_type);
    const void* const whole[] = {x, out, workspace, l->gate_packed, l->gate_scales, l->up_packed,
                                 l->up_scales, l->down_packed, l->down_scales};
    for (const void* p : whole)
        if (!aligned(p, 16)) return NVFP4_ERR_MISALIGNED;
    if (!aligned(ids, id_type == NVFP4_INDEX_I64 ? 8 : 4) || !aligned(weights, 4) || !aligned(l->gate_bias, bias_size) ||
        !aligned(l->up_bias, bias_size) || !aligned(l->down_bias, bias_size))
        return NVFP4_ERR_MISALIGNED;
    if (tokens == 0) return NVFP4_OK;
    uint8_t* const w = static_cast<uint8_t*>(workspace);
    if (mx_moe_few(tokens, topk, l->hidden, l->inner)) {
        Job& job = jobs[0];
        job = Job{};
        job.kind = JOB_LAUNCH;
        job.launch = +[](const Job& j, hipStream_t s) { return launch_mx_moe_few(j.mx_moe, s); };
        MxMoeArgs& a = job.mx_moe;
        a.x = x;
        a.x_bf16 = x_type == NVFP4_TYPE_BF16;
        a.wide = id_type == NVFP4_INDEX_I64;
        a.bias_bf16 = l->bias_type == NVFP4_TYPE_BF16;
        a.out_bf16 = out_type == NVFP4_TYPE_BF16;
        a.ldx = ldx;
        a.ids = ids;
        a.weights = weights;
        a.tokens = (int)tokens;
        a.topk = (int)topk;
        a.experts = (int)l->experts;
        a.hidden = (int)l->hidden;
        a.inner = (int)l->inner;
        a.gate_codes = static_cast<const uint8_t*>(l->gate_packed);
        a.gate_scales = static_cast<const uint8_t*>(l->gate_scales);
        a.up_codes = static_cast<const uint8_t*>(l->up_packed);
        a.up_scales = static_cast<const uint8_t*>(l->up_scales);
        a.down_codes = static_cast<const uint8_t*>(l->down_packed);
        a.down_scales = static_cast<const uint8_t*>(l->down_scales);
        a.gate_bias = l->gate_bias;
        a.up_bias = l->up_bias;
        a.down_bias = l->down_bias;
        a.act = l->activation;
        a.h = reinterpret_cast<uint16_t*>(w + at.h);
        a.out = out;
        *count = 1;
        return NVFP4_OK;
    }
    const int64_t pairs = tokens * topk;
    int32_t* const offsets = reinterpret_cast<int32_t*>(w + at.offsets);
    int32_t* const slots = reinterpret_cast<int32_t*>(w + at.slots);
    int32_t* const row_tokens = reinterpret_cast<int32_t*>(w + at.row_tokens);
    const nvfp4_mx_epilogue up = {l->activation, l->gate_packed, l->gate_scales, l->up_bias,
                                  l->gate_bias, l->bias_type, nullptr, 0};
    const nvfp4_mx_epilogue down = {NVFP4_ACT_NONE, nullptr, nullptr, l->down_bias, nullptr, l->bias_type, nullptr, 0};
    // (rows of h and y behind the last kept choice hold anything: they may be
    // read, but nothing that is used comes of them)
    Job sort, quantize;
    st = prepare_moe_sort(ids, id_type, tokens, topk, l->experts, offsets, slots, row_tokens, &sort);
    if (st == NVFP4_OK)
        st = prepare_mx_quantize(false, x, x_type, 1, 0, tokens, l->hidden, ldx, w + at.x_codes, w + at.x_scales, &quantize);
    if (st != NVFP4_OK) return st;
    Job* next = jobs;
    if (pairs <= kMoeRouteChoices) {
        *next = sort;
        next->mx_quant = quantize.mx_quant;
        next->launch = +[](const Job& j, hipStream_t s) { return launch_moe_route(j.moe, j.mx_quant, s); };
        ++next;
    } else {
        *next++ = sort;
        *next++ = quantize;
    }
    st = prepare_grouped_fused(w + at.x_codes, w + at.x_scales, tokens, row_tokens, l->up_packed, l->up_scales, offsets,
                               l->experts, 1.0f, &up, w + at.h, NVFP4_TYPE_BF16, pairs, l->inner, l->hidden, next);
    if (st != NVFP4_OK) return st;
    const bool packs = l->gate_packed ? mx_gated_packs(next->mx_gemm) : mx_fused_packs(next->mx_gemm);
    if (packs) {
        next->epilogue.q_codes = w + at.h_codes;
        next->epilogue.q_scales = w + at.h_scales;
    }
    ++next;
    if (!packs) {
        st = prepare_mx_quantize(false, w + at.h, NVFP4_TYPE_BF16, 1, 0, pairs, l->inner, l->inner, w + at.h_codes,
                                 w + at.h_scales, next++);
        if (st != NVFP4_OK) return st;
    }
    st = prepare_grouped_fused(w + at.h_codes, w + at.h_scales, pairs, nullptr, l->down_packed, l->down_scales, offsets,
                               l->experts, 1.0f, &down, w + at.y, NVFP4_TYPE_F32, pairs, l->hidden, l->inner, next);
    if (st != NVFP4_OK) return st;
    // (up to about a tile of rows to an expert; the kernel is right for more)
    if (mx_steps(l->inner) <= 4 && pairs <= 16 * l->experts)
        next->launch = +[](const Job& j, hipStream_t s) { return launch_mx_short(j.mx_gemm, j.epilogue, s); };
    ++next;
    st = prepare_moe_combine(w + at.y, NVFP4_TYPE_F32, tokens, topk, l->hidden, slots, weights, out, next);
    if (st != NVFP4_OK) return st;
    if (out_type == NVFP4_TYPE_BF16)
        next->launch = +[](const Job& j, hipStream_t s) { return launch_moe_combine_narrow(j.moe, s); };
    ++next;
    *count = (int)(next - jobs);
    return NVFP4_OK;
}

// ---- norms ----------------------------------------------------------------------

// What forward and gradient share: the operator itself.
int check_norm(const nvfp4_norm* f, NormArgs* a) {
    if (!f || !valid_type(f->type) || f->rows < 0 || f->rows > INT32_MAX || f->hidden < 1 ||
        f->hidden > kNormMaxHidden || f->gate_mode < NVFP4_GATE_NONE || f->gate_mode > NVFP4_GATE_ELEMENT ||
        (f->gate_mode != NVFP4_GATE_NONE && !f->gate && f->rows > 0) || !(f->eps >= 0.0f))
        return NVFP4_ERR_INVALID_VALUE;
    const void* const post_weight = f->post ? f->post_weight : nullptr;
    const void* const pre_weight = f->pre ? f->pre_weight : nullptr;
    const bool element = f->gate_mode == NVFP4_GATE_ELEMENT, channel = f->gate_mode == NVFP4_GATE_CHANNEL;
    if ((post_weight || pre_weight || channel) && !valid_type(f->weight_type)) return NVFP4_ERR_INVALID_VALUE;
    a->ld_gate = f->rows > 1 ? f->ld_gate : f->hidden;
    if (element && (a->ld_gate < f->hidden || a->ld_gate > kMaxDim)) return NVFP4_ERR_INVALID_VALUE;
    const uintptr_t weight_size = size_of(f->weight_type);
    if (!aligned(post_weight, weight_size) || !aligned(pre_weight, weight_size) ||
        (channel && !aligned(f->gate, weight_size)) || (element && !aligned(f->gate, size_of(f->type))))
        return NVFP4_ERR_MISALIGNED;
    a->bf16 = f->type == NVFP4_TYPE_BF16;
    a->weight_bf16 = f->weight_type == NVFP4_TYPE_BF16;
    a->post = f->post != 0;
    a->pre = f->pre != 0;
    a->gate_mode = f->gate_mode;
    a->hidden = (int)f->hidden;
    a->rows = f->rows;
    a->post_weight = post_weight;
    a->pre_weight = pre_weight;
    a->gate = element || channel ? f->gate : nullptr;  // (the forward kernel takes any other one for a channel's)
    a->scale = f->scale;
    a->residual_scale = f->residual_scale;
    a->eps = f->eps;
    return NVFP4_OK;
}

// A row stride to read rows of `hidden` elements with; 0 if it is too small.
int64_t stride_of(const NormArgs& a, int64_t ld) {
    if (a.rows <= 1) return a.hidden;
    return ld < a.hidden || ld > kMaxDim ? 0 : ld;
}

int prepare_norm(const nvfp4_norm* f, const void* y, int64_t ld_y, const void* residual,
                 int64_t ld_residual, void* h, void* n, void* n_codes, void* n_scales, Job* job) {
    *job = Job{};
    NormArgs& a = job->norm;
    const int st = check_norm(f, &a);
    if (st != NVFP4_OK) return st;
    const bool packed = n_codes || n_scales;
    a.ld_y = stride_of(a, ld_y);
    a.ld_residual = residual ? stride_of(a, ld_residual) : a.hidden;
    if ((packed && (!n_codes || !n_scales || n || a.hidden % kMxBlock)) || !a.ld_y || !a.ld_residual)
        return NVFP4_ERR_INVALID_VALUE;
    if (a.rows > 0 && (!y || (a.pre ? !n && !packed : n || packed || !h))) return NVFP4_ERR_INVALID_VALUE;
    const uintptr_t size = size_of(f->type);
    if (!aligned(y, size) || !aligned(residual, size) || !aligned(h, size) || !aligned(n, size) ||
        !aligned(n_codes, 16) || !aligned(n_scales, 16))
        return NVFP4_ERR_MISALIGNED;
    a.y = y;
    a.residual = residual;
    a.h = h;
    a.n = n;
    a.codes = static_cast<uint8_t*>(n_codes);
    a.scales = static_cast<uint8_t*>(n_scales);
    job->kind = JOB_LAUNCH;
    job->empty = a.rows == 0;
    job->launch = +[](const Job& j, hipStream_t s) { return launch_norm(j.norm, s); };
    return NVFP4_OK;
}

size_t grad_workspace(const NormArgs& a) {
    if (a.rows == 0 || !(a.post || a.pre || a.gate_mode == kGateChannel)) return 0;
    return (size_t)norm_grad_parts(a.bf16, a.rows, a.hidden) * 3 * a.hidden * sizeof(float);
}

}  // namespace

extern "C" {

int nvfp4_mx_moe_workspace(const nvfp4_mx_experts* layer, int64_t tokens, int64_t topk,
                           int out_type, size_t* bytes) {
    const int st = check_experts(layer, tokens, topk, out_type);
    if (st != NVFP4_OK || !bytes) return st != NVFP4_OK ? st : NVFP4_ERR_INVALID_VALUE;
    *bytes = MoeSpace(*layer, tokens, topk).bytes;
    return NVFP4_OK;
}

int nvfp4_mx_moe(const nvfp4_mx_experts* layer, const void* x, int x_type, int64_t ldx,
                 const void* expert_ids, int id_type, const float* weights, int64_t tokens,
                 int64_t topk, void* out, int out_type, void* workspace, size_t workspace_bytes,
                 void* stream) {
    Job jobs[kMoeJobs];
    int count;
    int st = prepare_mx_moe(layer, x, x_type, ldx, expert_ids, id_type, weights, tokens, topk, out, out_type,
                            workspace, workspace_bytes, jobs, &count);
    for (int i = 0; i < count && st == NVFP4_OK; ++i) st = run_job(jobs[i], stream);
    return st;
}

int nvfp4_sequence_add_mx_moe(nvfp4_sequence_t seq, const nvfp4_mx_experts* layer, const void* x,
                              int x_type, int64_t ldx, const void* expert_ids, int id_type,
                              const float* weights, int64_t tokens, int64_t topk, void* out,
                              int out_type, void* workspace, size_t workspace_bytes) {
    Job jobs[kMoeJobs];
    int count;
    const int st = prepare_mx_moe(layer, x, x_type, ldx, expert_ids, id_type, weights, tokens, topk, out, out_type,
                                  workspace, workspace_bytes, jobs, &count);
    if (count == 0) {  // refused, or no tokens: a call that does nothing
        jobs[0] = Job{};
        jobs[0].kind = JOB_LAUNCH;
        jobs[0].empty = true;
        count = 1;
    }
    return sequence_add(seq, st, jobs, count);
}

int nvfp4_add_norm(const nvfp4_norm* norm, const void* y, int64_t ld_y, const void* residual,
                   int64_t ld_residual, void* h, void* n, void* n_codes, void* n_scales,
                   void* stream) {
    Job job;
    const int st = prepare_norm(norm, y, ld_y, residual, ld_residual, h, n, n_codes, n_scales, &job);
    return run(st, job, stream);
}

int nvfp4_sequence_add_norm(nvfp4_sequence_t seq, const nvfp4_norm* norm, const void* y,
                            int64_t ld_y, const void* residual, int64_t ld_residual, void* h,
                            void* n, void* n_codes, void* n_scales) {
    Job job;
    const int st = prepare_norm(norm, y, ld_y, residual, ld_residual, h, n, n_codes, n_scales, &job);
    return sequence_add(seq, st, job);
}

int nvfp4_add_norm_grad_workspace(const nvfp4_norm* norm, size_t* bytes) {
    NormArgs a{};
    const int st = check_norm(norm, &a);
    if (st != NVFP4_OK || !bytes) return st != NVFP4_OK ? st : NVFP4_ERR_INVALID_VALUE;
    *bytes = grad_workspace(a);
    return NVFP4_OK;
}

int nvfp4_add_norm_grad(const nvfp4_norm* norm, const void* dh, int64_t ld_dh, const void* dn,
                        int64_t ld_dn, const void* y, int64_t ld_y, const void* h, int64_t ld_h,
                        void* dy, void* dresidual, void* dgate, float* dpost_weight,
                        float* dpre_weight, void* workspace, size_t workspace_bytes, void* stream) {
    Job job;
    NormArgs& a = job.norm;
    const int st = check_norm(norm, &a);
    if (st != NVFP4_OK) return st;
    const bool channel = a.gate_mode == kGateChannel, reads_y = a.post || a.gate_mode != kGateNone;
    const bool summed = (channel && dgate) || dpost_weight || dpre_weight;
    a.ld_dh = dh ? stride_of(a, ld_dh) : a.hidden;
    a.ld_dn = dn ? stride_of(a, ld_dn) : a.hidden;
    a.ld_y = reads_y ? stride_of(a, ld_y) : a.hidden;
    a.ld_h = a.pre ? stride_of(a, ld_h) : a.hidden;
    if (!a.ld_dh || !a.ld_dn || !a.ld_y || !a.ld_h || (dgate && a.gate_mode == kGateNone) ||
        (dpost_weight && !a.post) || (dpre_weight && !a.pre) || (dn && !a.pre))
        return NVFP4_ERR_INVALID_VALUE;
    // (without rows the sums are zeros all the same)
    if (a.rows > 0 && ((reads_y && !y) || (a.pre && (!h || !dn)))) return NVFP4_ERR_INVALID_VALUE;
    if (a.rows > 0 && summed && (!workspace || workspace_bytes < grad_workspace(a))) return NVFP4_ERR_INVALID_VALUE;
    const uintptr_t size = size_of(norm->type);
    if (!aligned(dh, size) || !aligned(dn, size) || !aligned(y, size) || !aligned(h, size) || !aligned(dy, size) ||
        !aligned(dresidual, size) || !aligned(dgate, channel ? 4 : size) || !aligned(dpost_weight, 4) ||
        !aligned(dpre_weight, 4) || !aligned(workspace, 16))
        return NVFP4_ERR_MISALIGNED;
    a.dh = dh;
    a.dn = dn;
    a.y = y;
    a.h_in = h;
    a.dy = dy;
    a.dresidual = dresidual;
    a.dgate = dgate;
    a.dpost_weight = dpost_weight;
    a.dpre_weight = dpre_weight;
    a.partials = summed ? static_cast<float*>(workspace) : nullptr;
    a.parts = a.rows > 0 ? norm_grad_parts(a.bf16, a.rows, a.hidden) : 0;
    job.kind = JOB_LAUNCH;
    job.empty = a.rows == 0 ? !summed : !dy && !dresidual && !dgate && !summed;
    job.launch = +[](const Job& j, hipStream_t s) { return launch_norm_grad(j.norm, s); };
    return run_job(job, stream);
}

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

int nvfp4_mx_linear_fused(const void* x, int x_type, int64_t ldx, const void* b_packed,
                          const void* b_scales, float alpha, const nvfp4_mx_epilogue* epilogue,
                          void* out, int out_type, int64_t M, int64_t N, int64_t K,
                          void* workspace, size_t workspace_bytes, void* stream) {
    size_t codes = 0, scales = 0;
    const int st0 = nvfp4_mx_packed_size(M, K, &codes, &scales);
    if (st0 != NVFP4_OK) return st0;
    const bool room = workspace && workspace_bytes >= codes + scales;
    // One launch where quantising again costs less than a launch of its own, 2.7 us.
    // Up to K = 8192 each of the 256 workgroups quantises the rows once (16 x 65536 x
    // 8192 52 us, 57 + 2.7 in two); behind it for every row block of B, and again of a
    // gate, that it walks: 2e-5 us for each of the values.  One launch and two, us:
    //                           K = 9984      16384         28672
    //    1 row,  768 columns    4.9   7.1    5.9   8.2    7.6   9.8
    //      with a gate          7.5   9.1    9.7  11.2   13.2  14.7
    //    4 rows                 5.3   7.4    6.8   8.6    9.0  10.6
    //      with a gate          8.2   9.5   11.0  11.9   15.8  16.2
    //   16 rows                 8.6   7.9   12.0   9.3   18.2  12.2
    //      with a gate         15.5  10.9   21.9  13.6   34.4  19.6
    //    4 rows, 4608 columns   8.6  11.3   13.3  15.2   20.5  21.7
    //      with a gate         17.3  17.7   24.3  24.5   36.3  35.3
    const bool gate = epilogue && epilogue->gate_packed;
    const double again = 2e-5 * (gate ? 2 : 1) * (double)M * K * (double)((mx_row_blocks(N) + 255) / 256);
    if (M <= kMxQuantRows && (!room || K <= 8192 || again <= 2.7))
        return nvfp4_mx_gemm_quantized_fused(x, x_type, ldx, b_packed, b_scales, alpha, epilogue, out, out_type,
                                             M, N, K, stream);
    if (!room) return NVFP4_ERR_INVALID_VALUE;
    uint8_t* const w = static_cast<uint8_t*>(workspace);
    Job quantize, product;
    int st = prepare_mx_quantize(false, x, x_type, 1, 0, M, K, ldx, w, w + codes, &quantize);
    if (st == NVFP4_OK)
        st = prepare_gemm_fused(w, w + codes, b_packed, b_scales, alpha, epilogue, out, out_type, M, N, K, &product);
    if (st == NVFP4_OK) st = run_job(quantize, stream);
    return run(st, product, stream);
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
