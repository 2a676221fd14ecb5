// nvfp4_mx_moe.hip -- gfx950 kernels of a whole layer of experts for few
// tokens (include/nvfp4_layer.h):
//   h[t][e]  = bf16(act(q(x[t]) . Wg_e^T + bg_e) * (q(x[t]) . Wu_e^T + bu_e))
//   out[t]   = sum over t's experts e of p[t][e] * (q(h[t][e]) . Wd_e^T + bd_e)
// with q() the MXFP4 quantisation and p the router's weight.
//
// Bound by the weights of the experts that were chosen, which are read once:
// every workgroup finds those experts itself from the router's choices, and
// the sum over a token's experts stays in registers, so that nothing but h is
// written on the way.  The weights go straight to the registers of the lanes
// that multiply them, a scale word (four steps, 4 KB of a row block) ahead of
// the one that is multiplied, also past the end of a task.
// x, and in the second launch h, are quantised by every workgroup into an
// image in its LDS, while its first weights are on their way.  256 experts x
// 256 x 6144, top 8, both launches, weights from the last-level cache: 1 token 11 us
// (14.4 from memory, 20 MB), 2 tokens 15, 4 tokens 24 (75 MB, 3.2 TB/s); 5 tokens by the
// calls for more 39.
#include "nvfp4_mx_parts.h"

#include <algorithm>

namespace nvfp4 {
namespace {

// A workgroup's view of the router's choices.
struct MoeChoices {
    int16_t id[kMoeFewChoices];      // expert of each choice, -1: dropped
    int16_t expert[kMoeFewChoices];  // the experts among them, by their first choice
    int count;
};

// Fills it; `first`: LDS for kMoeMaxExperts integers.  Ends with a barrier.
__device__ __forceinline__ void moe_choices(const MxMoeArgs& a, MoeChoices& c, int* first) {
    const int tid = threadIdx.x, lane = tid & 63, n = a.tokens * a.topk;
    for (int i = tid; i < n; i += blockDim.x) {
        const int64_t e = a.wide ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
        const bool kept = e >= 0 && e < a.experts;
        c.id[i] = (int16_t)(kept ? e : -1);
        if (kept) first[e] = n;
    }
    __syncthreads();
    for (int i = tid; i < n; i += blockDim.x)
        if (c.id[i] >= 0) atomicMin(&first[c.id[i]], i);
    __syncthreads();
    if (tid < 64) {
        int found = 0;
        for (int i0 = 0; i0 < n; i0 += 64) {
            const int i = i0 + lane, e = i < n ? c.id[i] : -1;
            const bool leads = e >= 0 && first[e] == i;
            const uint64_t who = __ballot(leads);
            if (leads) c.expert[found + __popcll(who & ((1ull << lane) - 1))] = (int16_t)e;
            found += __popcll(who);
        }
        if (lane == 0) c.count = found;
    }
    __syncthreads();
}

// A token's first choice of expert e, as a row of h; -1: none, or no token.
__device__ __forceinline__ int moe_row(const MxMoeArgs& a, const MoeChoices& c, int e, int token) {
    const int16_t* const id = c.id + min(token, a.tokens - 1) * a.topk;
    int at = -1;
    for (int j0 = 0; j0 < a.topk; j0 += 8) {
        int x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = id[min(j0 + j, a.topk - 1)];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (x[j] == e && at < 0) at = j0 + j;  // (the last choice again: found before)
    }
    return token < a.tokens && at >= 0 ? token * a.topk + at : -1;
}
// The router's weight of the token for the expert, over all its choices of it.
// `weights`: in LDS.
__device__ __forceinline__ float moe_weight(const MxMoeArgs& a, const MoeChoices& c, int e, int at, int token, const float* weights) {
    if (at < 0) return 0.0f;
    float w = weights[at];
    for (int j = at + 1; j < (token + 1) * a.topk; ++j)
        if (c.id[j] == e) w += weights[j];
    return w;
}

// What a wave multiplies at a time: four steps of 16 rows of a weight and of
// its rows of activations (in one tile), a lane's share.
struct MoeFrag {
    mx_u4 b[4], a[4];
    uint32_t sb, sa;
};

// The lane's 16 code bytes of each step of scale word q: `codes` points to its
// place in the row block's step 0.  Steps past the last one: zeros.
__device__ __forceinline__ void moe_steps(const uint8_t* codes, int q, int C, mx_u4 (&w)[4]) {
    const uint8_t* p = codes + (int64_t)q * 4 * kMxFrag;
    const int n = C - 4 * q;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        w[s] = mx_u4{0, 0, 0, 0};
        if (s < n) w[s] = *reinterpret_cast<const mx_u4*>(p + s * kMxFrag);
    }
}
__device__ __forceinline__ uint32_t moe_word(const uint8_t* scales, int q) {
    return *reinterpret_cast<const uint32_t*>(scales + (int64_t)q * kMxScaleFrag);
}
__device__ __forceinline__ mx_f4 moe_multiply(const MoeFrag& f, mx_f4 acc) {
    mx_each<4>([&](auto S) { acc = mx_mfma16<S.value>(f.b[S.value], f.sb, f.a[S.value], f.sa, acc); });
    return acc;
}

// ---- quantised rows in LDS ------------------------------------------------
// Rows of K, padded to whole scale words with zeros: [row][word][step][block]
// of 16 code bytes, and a word of scale bytes for each [row][word][block].
__host__ __device__ constexpr int64_t moe_image_bytes(int64_t rows, int64_t K) {
    return rows * ((K + 4 * kMxStep - 1) / (4 * kMxStep)) * (16 * 16 + 16);
}
template <typename T>
__device__ __forceinline__ void moe_image(const T* x, int64_t ld, int rows, int K, uint8_t* image) {
    const int Q = (K + 4 * kMxStep - 1) / (4 * kMxStep), blocks = Q * 16;
    uint8_t* const scales = image + rows * blocks * 16;
    for (int i = threadIdx.x; i < rows * blocks; i += blockDim.x) {
        const int row = i / blocks, b = i % blocks;
        mx_u4 w = {0, 0, 0, 0};
        uint32_t byte = 0;
        if (b * kMxBlock < K) byte = mx_quant_load(x + row * ld + b * kMxBlock, w);
        *reinterpret_cast<mx_u4*>(image + i * 16) = w;
        scales[((row * Q + (b >> 4)) * 4 + (b & 3)) * 4 + (b >> 2 & 3)] = (uint8_t)byte;
    }
}
// The lane's share of word q of a row (its block l / 16 of each step).
__device__ __forceinline__ void moe_from_image(const uint8_t* image, int rows, int Q, int row, int q, MoeFrag& f) {
    const int kg = (threadIdx.x & 63) >> 4;
    const uint8_t* const p = image + ((row * Q + q) * 16 + kg) * 16;
#pragma unroll
    for (int s = 0; s < 4; ++s) f.a[s] = *reinterpret_cast<const mx_u4*>(p + s * 64);
    f.sa = *reinterpret_cast<const uint32_t*>(image + rows * Q * 256 + ((row * Q + q) * 4 + kg) * 4);
}

// ---------------------------------------------------------------------------
// First kernel.  A task is eight columns of h of one expert (with a gate:
// eight rows of each weight make the 16 of a matrix instruction) or 16
// (without), for all tokens; its waves split K.  h: [choice][inner] bfloat16.
// ---------------------------------------------------------------------------
constexpr int kUpWaves = 8;

template <typename T, bool GATED>
__global__ void __launch_bounds__(kUpWaves * 64) moe_up_few_kernel(MxMoeArgs a) {
    constexpr int COLS = GATED ? 8 : 16;
    extern __shared__ __attribute__((aligned(1024))) uint8_t image[];
    __shared__ MoeChoices choices;
    __shared__ __attribute__((aligned(16))) union { int first[kMoeMaxExperts]; mx_f4 red[kUpWaves][64]; } u;
    const int lane = threadIdx.x & 63, r16 = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int C = (a.hidden + kMxStep - 1) / kMxStep, Q = (C + 3) / 4;
    const int units = a.inner / COLS, RB = a.inner / 16, turn = gridDim.x;
    moe_choices(a, choices, u.first);
    const int total = __builtin_amdgcn_readfirstlane(choices.count) * units;
    int task = blockIdx.x;
    if (task >= total) return;

    const bool second = GATED && r16 >= 8;  // (the lane's row is one of the up weight)
    const uint8_t* const codes = GATED && !second ? a.gate_codes : a.up_codes;
    const uint8_t* const scales = GATED && !second ? a.gate_scales : a.up_scales;
    auto expert_of = [&](int t) { return __builtin_amdgcn_readfirstlane((int)choices.expert[t / units]); };
    auto load = [&](int t, int q) {
        const int unit = t % units, row = GATED ? (unit & 1) * 8 + (r16 & 7) : r16;
        const int64_t rb = (int64_t)expert_of(t) * RB + (GATED ? unit >> 1 : unit);
        MoeFrag f;
        moe_steps(codes + rb * C * kMxFrag + mx_code_at(row, kg), q, C, f.b);
        f.sb = moe_word(scales + rb * Q * kMxScaleFrag + mx_scale_at(row, kg), q);
        return f;
    };
    MoeFrag next;
    if (wave < Q) next = load(task, wave);
    moe_image(static_cast<const T*>(a.x), a.ldx, a.tokens, a.hidden, image);
    __syncthreads();
    for (; task < total; task += turn) {
        const int e = expert_of(task), unit = task % units;
        mx_f4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int q = wave; q < Q; q += kUpWaves) {
            MoeFrag f = next;
            if (q + kUpWaves < Q)
                next = load(task, q + kUpWaves);
            else if (task + turn < total)
                next = load(task + turn, wave);
            moe_from_image(image, a.tokens, Q, min(r16, a.tokens - 1), q, f);
            acc = moe_multiply(f, acc);
        }
        u.red[wave][lane] = acc;
        __syncthreads();
        if (wave == 0) {
            const int at = moe_row(a, choices, e, r16);
            auto sum_of = [&](int from) {
                mx_f4 s = u.red[0][from];
#pragma unroll
                for (int w = 1; w < kUpWaves; ++w) s += u.red[w][from];
                return s;
            };
            if (at >= 0 && (!GATED || kg < 2)) {
                const int col = unit * COLS + 4 * kg;
                const int64_t b = (int64_t)e * a.inner + col;
                mx_f4 z = sum_of(GATED ? lane + 32 : lane) + mx_row4(a.up_bias, a.bias_bf16, b, col, a.inner), gate = z;
                if constexpr (GATED) gate = sum_of(lane) + mx_row4(a.gate_bias, a.bias_bf16, b, col, a.inner);
                mx_by_act(a.act, true, [&](auto ACT) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) z[v] = GATED ? mx_act<ACT.value>(gate[v]) * z[v] : mx_act<ACT.value>(z[v]);
                });
                mx_put4(a.h, true, (int64_t)at * a.inner + col, col, a.inner, z);
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Second kernel.  A task is 16 columns of the result, for all tokens and all
// experts: the waves split the pairs of (expert, scale word of its inner
// dimension), multiply the rows of h, and add them under the router's weights
// in registers; the waves' sums are added in their order at the end of the
// task.  h is quantised into LDS first.
// ---------------------------------------------------------------------------
constexpr int kDownWaves = 8;

__global__ void __launch_bounds__(kDownWaves * 64) moe_down_few_kernel(MxMoeArgs a) {
    extern __shared__ __attribute__((aligned(1024))) uint8_t image[];
    __shared__ MoeChoices choices;
    __shared__ float weights[kMoeFewChoices];
    __shared__ __attribute__((aligned(16))) union { int first[kMoeMaxExperts]; mx_f4 red[kDownWaves][64]; } u;
    const int lane = threadIdx.x & 63, r16 = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int C = (a.inner + kMxStep - 1) / kMxStep, Q = (C + 3) / 4;
    const int RB = (a.hidden + 15) / 16, turn = gridDim.x, pairs = a.tokens * a.topk;
    for (int i = threadIdx.x; i < pairs; i += kDownWaves * 64) weights[i] = a.weights ? a.weights[i] : 1.0f;
    moe_choices(a, choices, u.first);
    const int items = __builtin_amdgcn_readfirstlane(choices.count) * Q;

    struct Item {
        int e, q, at;      // at: the lane's row of h, of token l % 16 (-1: none)
        float weight;      // of that token
        MoeFrag f;
    };
    auto fetch = [&](int cb, int i) {
        Item n;
        n.e = __builtin_amdgcn_readfirstlane((int)choices.expert[i / Q]);
        n.q = i % Q;
        const int64_t rb = (int64_t)n.e * RB + cb;
        moe_steps(a.down_codes + rb * C * kMxFrag + mx_code_at(r16, kg), n.q, C, n.f.b);
        n.f.sb = moe_word(a.down_scales + rb * Q * kMxScaleFrag + mx_scale_at(r16, kg), n.q);
        n.at = moe_row(a, choices, n.e, r16);
        n.weight = moe_weight(a, choices, n.e, n.at, r16, weights);
        return n;
    };
    Item next;
    if (wave < items && (int)blockIdx.x < RB) next = fetch(blockIdx.x, wave);
    moe_image(a.h, a.inner, pairs, a.inner, image);
    __syncthreads();
    for (int cb = blockIdx.x; cb < RB; cb += turn) {
        const int col = cb * 16 + 4 * kg;
        mx_f4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int i = wave; i < items; i += kDownWaves) {
            Item now = next;
            if (i + kDownWaves < items)
                next = fetch(cb, i + kDownWaves);
            else if (cb + turn < RB)
                next = fetch(cb + turn, wave);
            mx_f4 bias = {0.0f, 0.0f, 0.0f, 0.0f};
            if (now.q == 0) bias = mx_row4(a.down_bias, a.bias_bf16, (int64_t)now.e * a.hidden + col, col, a.hidden);
            moe_from_image(image, pairs, Q, max(now.at, 0), now.q, now.f);
            const mx_f4 y = mx_pin(moe_multiply(now.f, bias));
            if (now.at >= 0) sum += now.weight * y;
        }
        u.red[wave][lane] = sum;
        __syncthreads();
        if (wave == 0) {
            mx_f4 s = u.red[0][lane];
#pragma unroll
            for (int w = 1; w < kDownWaves; ++w) s += u.red[w][lane];
            if (r16 < a.tokens) mx_put4(a.out, a.out_bf16, (int64_t)r16 * a.hidden + col, col, a.hidden, s);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Few choices sorted by expert, and x quantised, in one launch: the first
// workgroup sorts, the others quantise, a block to a work-item.  A choice's row
// is the number of kept choices of smaller experts, and of its own before it,
// counted over the list in LDS.  (128 choices of 256 experts, 16 rows of 6144:
// 7.8 us in two launches.)
// ---------------------------------------------------------------------------
constexpr int kRouteWG = 1024;

template <typename T>
__global__ void __launch_bounds__(kRouteWG) moe_route_kernel(MoeArgs s, MxQuantArgs q) {
    __shared__ __attribute__((aligned(16))) int key[kMoeRouteChoices];  // expert and number of each choice
    __shared__ int sorted[kMoeRouteChoices];
    const int tid = threadIdx.x;
    if (blockIdx.x > 0) {
        const int C = q.C, Q = (C + 3) / 4, blocks = Q * 16;
        const int64_t i = (int64_t)(blockIdx.x - 1) * kRouteWG + tid;
        const int64_t row = i / blocks;
        const int b = (int)(i % blocks), c = b >> 2;
        if (row >= (int64_t)q.RB * 16) return;
        mx_u4 w = {0, 0, 0, 0};
        uint32_t byte = 0;
        if (row < q.rows && b * kMxBlock < q.K) byte = mx_quant_load(static_cast<const T*>(q.x) + row * q.ld + b * kMxBlock, w);
        if (c < C) *reinterpret_cast<mx_u4*>(q.codes + ((row >> 4) * C + c) * kMxFrag + mx_code_at(row & 15, b & 3)) = w;
        q.scales[((row >> 4) * Q + c / 4) * kMxScaleFrag + mx_scale_at(row & 15, b & 3) + (c & 3)] = (uint8_t)byte;
        return;
    }
    constexpr int kDropped = INT32_MAX, PER = kRouteWG / kMoeRouteChoices;  // lanes to a choice
    static_assert(PER == 4 && kMoeMaxExperts * kMoeRouteChoices < kDropped, "four lanes to a choice; keys");
    const int n = (int)s.tokens * s.topk;
    if (tid < kMoeRouteChoices) {
        int64_t e = -1;
        if (tid < n) e = s.wide ? static_cast<const int64_t*>(s.ids)[tid] : static_cast<const int32_t*>(s.ids)[tid];
        key[tid] = e >= 0 && e < s.experts ? (int)e * kMoeRouteChoices + tid : kDropped;
        sorted[tid] = kDropped;
    }
    __syncthreads();
    // each lane counts a quarter of the keys that are smaller than its choice's
    const int i = tid / PER, mine = key[i];
    int slot = 0;
#pragma unroll 4
    for (int j = tid % PER * 4; j < n; j += PER * 4) {
        typedef int i4 __attribute__((ext_vector_type(4)));
        const i4 k = *reinterpret_cast<const i4*>(key + j);
        slot += (k[0] < mine) + (k[1] < mine) + (k[2] < mine) + (k[3] < mine);
    }
    slot += __shfl_xor(slot, 1);
    slot += __shfl_xor(slot, 2);
    const bool kept = mine != kDropped;
    if (tid % PER == 0 && i < n) {
        if (kept) sorted[slot] = mine / kMoeRouteChoices;
        s.slots[i] = kept ? slot : -1;
        if (kept) s.row_tokens[slot] = i / s.topk;
    }
    __syncthreads();
    if (tid < n && sorted[tid] == kDropped) s.row_tokens[tid] = -1;  // (no kept choice has this row)
    // an expert's first row: the first sorted choice that is not smaller
    for (int e = tid; e <= s.experts; e += kRouteWG) {
        int lo = 0, hi = n;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (sorted[mid] < e)
                lo = mid + 1;
            else
                hi = mid;
        }
        s.row_offsets[e] = lo;
    }
}

}  // namespace

hipError_t launch_moe_route(const MoeArgs& s, const MxQuantArgs& q, hipStream_t stream) {
    const int64_t blocks = (int64_t)q.RB * 16 * ((q.C + 3) / 4) * 16;
    const dim3 grid((unsigned)(1 + (blocks + kRouteWG - 1) / kRouteWG));
    if (q.bf16)
        hipLaunchKernelGGL((moe_route_kernel<uint16_t>), grid, dim3(kRouteWG), 0, stream, s, q);
    else
        hipLaunchKernelGGL((moe_route_kernel<float>), grid, dim3(kRouteWG), 0, stream, s, q);
    return hipGetLastError();
}

bool mx_moe_few(int64_t tokens, int64_t topk, int64_t hidden, int64_t inner) {
    return tokens <= kMoeFewTokens && tokens * topk <= kMoeFewChoices && moe_image_bytes(tokens, hidden) <= kMoeImageBytes &&
           moe_image_bytes(tokens * topk, inner) <= kMoeImageBytes;
}

hipError_t launch_mx_moe_few(const MxMoeArgs& a, hipStream_t stream) {
    constexpr int kResident = 2 * 256;  // workgroups that the GPU holds at once
    const bool gated = a.gate_codes != nullptr;
    const int64_t experts = std::min(a.tokens * a.topk, a.experts);
    const size_t image = (size_t)moe_image_bytes(a.tokens, a.hidden);
    const dim3 up((unsigned)std::min<int64_t>(experts * (a.inner / (gated ? 8 : 16)), kResident)), block(kUpWaves * 64);
    if (gated) {
        if (a.x_bf16)
            hipLaunchKernelGGL((moe_up_few_kernel<uint16_t, true>), up, block, image, stream, a);
        else
            hipLaunchKernelGGL((moe_up_few_kernel<float, true>), up, block, image, stream, a);
    } else {
        if (a.x_bf16)
            hipLaunchKernelGGL((moe_up_few_kernel<uint16_t, false>), up, block, image, stream, a);
        else
            hipLaunchKernelGGL((moe_up_few_kernel<float, false>), up, block, image, stream, a);
    }
    const hipError_t error = hipGetLastError();
    if (error != hipSuccess) return error;
    hipLaunchKernelGGL(moe_down_few_kernel, dim3((unsigned)std::min((a.hidden + 15) / 16, kResident)), dim3(kDownWaves * 64),
                       (size_t)moe_image_bytes((int64_t)a.tokens * a.topk, a.inner), stream, a);
    return hipGetLastError();
}

}  // namespace nvfp4
