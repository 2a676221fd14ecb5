// nvfp4_mx_moe.hip -- gfx950 kernels of a whole layer of experts for few
// tokens (include/nvfp4_layer.h), in two launches:
//   h[t][e]  = bf16(act(q(x[t]) . Wg_e^T + bg_e) * (q(x[t]) . Wu_e^T + bu_e))
//   out[t]   = sum over t's experts e of p[t][e] * (q(h[t][e]) . Wd_e^T + bd_e)
// with q() the MXFP4 quantisation and p the router's weight.
//
// Bound by the weights of the experts that were chosen, which are read once:
// every workgroup finds those experts itself from the router's choices, the
// rows are quantised where they are multiplied, and the sum over a token's
// experts stays in registers, so nothing but h is written on the way.
#include "nvfp4_mx_parts.h"

#include <algorithm>

namespace nvfp4 {
namespace {

constexpr int kMoeWaves = 4;
constexpr int kMoeWG = kMoeWaves * 64;
constexpr int kMoeTiles = kMoeFewTokens / 16;  // of 16 rows

// LDS of a workgroup.  Three of them fit a CU.
struct MoeLds {
    uint8_t b[kMoeWaves][2][4 * kMxFrag];              // a wave's weights: this item's and the next one's
    uint8_t a[kMoeWaves][4 * kMxFrag + kMxScaleFrag];  // its quantised rows; the sums at the end of a task
    uint32_t list[kMoeWaves][2][kMoeFewTokens];        // rows of this item's and the next one's expert
    int16_t id[kMoeFewChoices], expert[kMoeFewChoices];
};
static_assert(sizeof(MoeLds) <= 160 * 1024 / 3, "three workgroups to a CU");
static_assert(kMoeMaxExperts * 4 <= sizeof(MoeLds::b) && kMoeMaxExperts < 32768, "the table of the experts' first choices");

// Reads the choices and numbers the experts among them in the order of their
// first choice: lds.id (-1: dropped), lds.expert; returns how many there are.
__device__ __forceinline__ int moe_experts(const MxMoeArgs& a, MoeLds& lds) {
    const int tid = threadIdx.x, lane = tid & 63, n = a.tokens * a.topk;
    int* const first = reinterpret_cast<int*>(lds.b);
    __shared__ int count;
    for (int i = tid; i < n; i += kMoeWG) {
        const int64_t e = a.wide ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
        const bool kept = e >= 0 && e < a.experts;
        lds.id[i] = (int16_t)(kept ? e : -1);
        if (kept) first[e] = n;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kMoeWG)
        if (lds.id[i] >= 0) atomicMin(&first[lds.id[i]], i);
    __syncthreads();
    if (tid < 64) {
        int found = 0;
        for (int i0 = 0; i0 < n; i0 += 64) {
            const int i = i0 + lane, e = i < n ? lds.id[i] : -1;
            const bool leads = e >= 0 && first[e] == i;
            const uint64_t who = __ballot(leads);
            if (leads) lds.expert[found + __popcll(who & ((1ull << lane) - 1))] = (int16_t)e;
            found += __popcll(who);
        }
        if (lane == 0) count = found;
    }
    __syncthreads();
    return count;
}

// The tokens of expert e, a bit each, and a row of the wave's list for each:
// token | number of its first choice of e << 16.  weight: the lane's token's,
// over all its choices of e.
__device__ __forceinline__ uint64_t moe_rows(const MxMoeArgs& a, MoeLds& lds, int e, int slot, float& weight) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int at = -1, times = 0;
    if (lane < a.tokens)
        for (int j = a.topk - 1; j >= 0; --j)
            if (lds.id[lane * a.topk + j] == e) {
                at = lane * a.topk + j;
                ++times;
            }
    const uint64_t who = __ballot(at >= 0);
    weight = at < 0 ? 0.0f : a.weights ? a.weights[at] : 1.0f;
    for (int j = at + 1; times > 1; ++j)  // the same expert more than once
        if (lds.id[j] == e) {
            weight += a.weights ? a.weights[j] : 1.0f;
            --times;
        }
    if (at >= 0) lds.list[wave][slot][__popcll(who & ((1ull << lane) - 1))] = (uint32_t)(lane | at << 16);
    mx_wave_fence();
    return who;
}

// Four steps (a scale word) of a row block of 16 rows of a weight, or of eight
// rows of each of two weights (PAIR: half `half` of row block rb of both), to
// LDS; returns the lane's scales.  Steps past the last one are past the
// buffer's range; what they leave in LDS is multiplied by zeros of the rows,
// under scale bytes of zero.
template <bool PAIR>
__device__ __forceinline__ uint32_t moe_load(const uint8_t* codes0, const uint8_t* codes1, const uint8_t* scales0,
                                             const uint8_t* scales1, int64_t rb, int half, int q, int C, uint32_t lds) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, kg = lane >> 4, Q = (C + 3) / 4;
    const int64_t at = (rb * C + 4 * q) * kMxFrag;
    const uint32_t bytes = (uint32_t)min(4, C - 4 * q) * kMxFrag;
    const __amdgpu_buffer_rsrc_t r0 = make_rsrc(codes0 + at, bytes);
    const uint8_t* s = scales0;
    int row = r16;
    if constexpr (PAIR) {
        const __amdgpu_buffer_rsrc_t r1 = make_rsrc(codes1 + at, bytes);
        const uint32_t from = (uint32_t)((lane >> 5) * kMxFrag + half * (kMxFrag / 2) + (lane & 31) * 16);
        mx_each<4>([&](auto I) {  // two steps of one weight, then of the other
            constexpr int i = I.value;
            if constexpr (i % 2 == 0)
                mx_dma<16, i * kMxFrag>(r0, from + i / 2 * 2 * kMxFrag, 0, lds);
            else
                mx_dma<16, i * kMxFrag>(r1, from + i / 2 * 2 * kMxFrag, 0, lds);
        });
        if (r16 >= 8) s = scales1;
        row = half * 8 + (r16 & 7);
    } else {
        mx_each<4>([&](auto I) { mx_dma<16, I.value * kMxFrag>(r0, lane * 16 + I.value * kMxFrag, 0, lds); });
    }
    return *reinterpret_cast<const uint32_t*>(s + (rb * Q + q) * kMxScaleFrag + mx_scale_at(row, kg));
}
// Where the lane's 16 bytes of step S of what moe_load brought lie.
template <bool PAIR, int S>
__device__ __forceinline__ int moe_code_at(int half) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, kg = lane >> 4;
    if constexpr (PAIR) {
        const int row = half * 8 + (r16 & 7);
        return S / 2 * 2 * kMxFrag + (r16 >> 3) * kMxFrag + (S & 1) * (kMxFrag / 2) + (r16 & 7) * 64 + ((kg ^ (row >> 2)) << 4);
    }
    return S * kMxFrag + mx_code_at(r16, kg);
}

// A row's block for the lane, if it has one: lane l takes block l % 16 of scale
// word q of row l / 16 of four.
template <typename T>
__device__ __forceinline__ MxRaw<T> moe_raw(const T* rows, int64_t ld, int row, bool live, int q, int K) {
    const int k = q * 4 * kMxStep + (threadIdx.x & 15) * kMxBlock;
    MxRaw<T> r;
#pragma unroll
    for (int i = 0; i < r.L; ++i) r.v[i] = mx_u4{0, 0, 0, 0};
    if (live && k < K) r = mx_raw_load(rows + row * ld + k);
    return r;
}
// Quantises it to row `to` of the wave's operand.
template <typename T>
__device__ __forceinline__ void moe_quantize(const MxRaw<T>& r, uint8_t* a_lds, int to, bool live) {
    if (!live) return;
    const int s = (threadIdx.x & 15) >> 2, b = threadIdx.x & 3;
    mx_u4 w;
    const uint32_t byte = mx_quant_block(r, w);
    *reinterpret_cast<mx_u4*>(a_lds + s * kMxFrag + mx_code_at(to, b)) = w;
    a_lds[4 * kMxFrag + mx_scale_at(to, b) + s] = (uint8_t)byte;
}

// acc += the weights in b_lds by the rows in a_lds, four steps.  Rows of a_lds
// that nothing was written to give whatever LDS held: not used.
template <bool PAIR>
__device__ __forceinline__ mx_f4 moe_multiply(const uint8_t* b_lds, uint32_t sb, int half, const uint8_t* a_lds, mx_f4 acc) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, kg = lane >> 4;
    const uint32_t sa = *reinterpret_cast<const uint32_t*>(a_lds + 4 * kMxFrag + mx_scale_at(r16, kg));
    mx_each<4>([&](auto S) {
        const mx_u4 wb = *reinterpret_cast<const mx_u4*>(b_lds + moe_code_at<PAIR, S.value>(half));
        const mx_u4 wa = *reinterpret_cast<const mx_u4*>(a_lds + S.value * kMxFrag + mx_code_at(r16, kg));
        acc = mx_mfma16<S.value>(wb, sb, wa, sa, acc);
    });
    return acc;
}

// ---------------------------------------------------------------------------
// First kernel.  A task is eight columns of h of one expert (with a gate: eight
// rows of each weight make the 16 of one matrix instruction) or 16 (without),
// for all its tokens; the workgroups walk the tasks, and a task's waves split K,
// a scale word (512 elements) at a time.  While a wave multiplies one word, the
// weights and the rows of the next are on their way, also past the end of the
// task.
// ---------------------------------------------------------------------------
template <typename T, bool GATED>
__global__ void __launch_bounds__(kMoeWG) moe_up_kernel(MxMoeArgs a) {
    constexpr int COLS = GATED ? 8 : 16;
    __shared__ __attribute__((aligned(1024))) MoeLds lds;
    const int lane = threadIdx.x & 63, r16 = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int C = (a.hidden + kMxStep - 1) / kMxStep, Q = (C + 3) / 4;
    const int units = a.inner / COLS, RB = a.inner / 16;
    const int total = __builtin_amdgcn_readfirstlane(moe_experts(a, lds)) * units, turn = gridDim.x;
    const T* const x = static_cast<const T*>(a.x);
    uint8_t* const a_lds = lds.a[wave];
    float unused;

    auto expert_of = [&](int task) { return __builtin_amdgcn_readfirstlane((int)lds.expert[task / units]); };
    auto load = [&](int task, int q, int slot) {
        const int u = task % units;
        const int64_t rb = (int64_t)expert_of(task) * RB + (GATED ? u >> 1 : u);
        return moe_load<GATED>(GATED ? a.gate_codes : a.up_codes, a.up_codes, GATED ? a.gate_scales : a.up_scales, a.up_scales,
                               rb, u & 1, q, C, lds_addr(lds.b[wave][slot]));
    };
    // rows first .. first + 3 of a list
    auto raw_of = [&](int slot, int rows, int first, int q) {
        const int n = first + (lane >> 4);
        const int token = n < rows ? (int)(lds.list[wave][slot][n] & 0xFFFF) : 0;
        return moe_raw<T>(x, a.ldx, token, n < rows, q, a.hidden);
    };

    int task = blockIdx.x;
    if (task >= total) return;
    int k = 0, slot = 0;  // places of the list and of the weights
    int rows = __popcll(moe_rows(a, lds, expert_of(task), 0, unused));
    uint32_t sb = 0;
    MxRaw<T> raw;
    if (wave < Q) {
        raw = raw_of(0, rows, 0, wave);
        sb = load(task, wave, 0);
    }
    for (; task < total; task += turn) {
        const int e = expert_of(task), u = task % units, tiles = (rows + 15) / 16;
        const bool more = task + turn < total;
        int next_rows = 0;
        if (more) next_rows = __popcll(moe_rows(a, lds, expert_of(task + turn), k ^ 1, unused));
        mx_f4 acc[kMoeTiles];
#pragma unroll
        for (int t = 0; t < kMoeTiles; ++t) acc[t] = mx_f4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int q = wave; q < Q; q += kMoeWaves) {
            wait_vmcnt<0>();
            asm volatile("" ::: "memory");  // the weights have landed
            const MxRaw<T> now = raw;
            const uint32_t sb_now = sb;
            const uint8_t* const b_lds = lds.b[wave][slot];
            slot ^= 1;
            if (q + kMoeWaves < Q) {
                raw = raw_of(k, rows, 0, q + kMoeWaves);
                sb = load(task, q + kMoeWaves, slot);
            } else if (more) {
                raw = raw_of(k ^ 1, next_rows, 0, wave);
                sb = load(task + turn, wave, slot);
            }
#pragma unroll
            for (int t = 0; t < kMoeTiles; ++t) {
                if (t >= tiles) break;
                const int live = min(rows - t * 16, 16);
                moe_quantize(t == 0 ? now : raw_of(k, rows, t * 16, q), a_lds, lane >> 4, (lane >> 4) < live);
                for (int p = 4; p < live; p += 4)
                    moe_quantize(raw_of(k, rows, t * 16 + p, q), a_lds, p + (lane >> 4), p + (lane >> 4) < live);
                mx_wave_fence();
                acc[t] = moe_multiply<GATED>(b_lds, sb_now, u & 1, a_lds, acc[t]);
                mx_wave_fence();
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // LDS is read before it is filled again
        }
        // the waves' sums, added in their order, a tile to a wave
#pragma unroll
        for (int t = 0; t < kMoeTiles; ++t)
            if (t < tiles) reinterpret_cast<mx_f4*>(a_lds)[t * 64 + lane] = acc[t];
        __syncthreads();
        if (wave < tiles) {
            auto sum_of = [&](int from) {
                mx_f4 s = reinterpret_cast<const mx_f4*>(lds.a[0])[wave * 64 + from];
#pragma unroll
                for (int w = 1; w < kMoeWaves; ++w) s += reinterpret_cast<const mx_f4*>(lds.a[w])[wave * 64 + from];
                return s;
            };
            const int n = wave * 16 + r16;
            if (n < rows && (!GATED || kg < 2)) {
                const int col = u * COLS + 4 * kg;
                const int64_t at = (int64_t)e * a.inner + col;
                mx_f4 z = sum_of(lane);
                const mx_f4 bias = mx_row4(a.up_bias, a.bias_bf16, at, col, a.inner);
                if constexpr (GATED)
                    z = mx_act(z + mx_row4(a.gate_bias, a.bias_bf16, at, col, a.inner), a.act) * (sum_of(lane + 32) + bias);
                else
                    z = mx_act(z + bias, a.act);
                mx_put4(a.h, true, (int64_t)(lds.list[wave][k][n] >> 16) * a.inner + col, col, a.inner, z);
            }
        }
        __syncthreads();
        rows = next_rows;
        k ^= 1;
    }
}

// ---------------------------------------------------------------------------
// Second kernel.  A task is 16 columns of the result, for all tokens and all
// experts: the waves split the pairs of (expert, scale word of its inner
// dimension), multiply the expert's rows of h, and add them under the router's
// weights in registers; the waves' sums are added in their order at the end of
// the task.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kMoeWG) moe_down_kernel(MxMoeArgs a) {
    __shared__ __attribute__((aligned(1024))) MoeLds lds;
    const int lane = threadIdx.x & 63, r16 = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int C = (a.inner + kMxStep - 1) / kMxStep, Q = (C + 3) / 4;
    const int RB = (a.hidden + 15) / 16, turn = gridDim.x;
    const int items = __builtin_amdgcn_readfirstlane(moe_experts(a, lds)) * Q;
    const int tiles = (a.tokens + 15) / 16;
    uint8_t* const a_lds = lds.a[wave];

    struct Item {
        int e, q;
        uint64_t who;      // its tokens
        float weight;      // of the lane's token
        uint32_t sb;
        MxRaw<uint16_t> raw;
    };
    auto raw_of = [&](int slot, uint64_t who, int t, int p, int q) {
        const int before = __popcll(who & ((1ull << (t * 16)) - 1)), live = __popc((uint32_t)(who >> (t * 16)) & 0xFFFF);
        const int n = p + (lane >> 4);
        const int row = n < live ? (int)(lds.list[wave][slot][before + n] >> 16) : 0;
        return moe_raw<uint16_t>(a.h, a.inner, row, n < live, q, a.inner);
    };
    auto first_tile = [&](uint64_t who) { return (__ffsll((unsigned long long)who) - 1) >> 4; };
    auto fetch = [&](int cb, int i, int slot) {
        Item n;
        n.e = __builtin_amdgcn_readfirstlane((int)lds.expert[i / Q]);
        n.q = i % Q;
        n.who = moe_rows(a, lds, n.e, slot, n.weight);
        n.raw = raw_of(slot, n.who, first_tile(n.who), 0, n.q);
        n.sb = moe_load<false>(a.down_codes, nullptr, a.down_scales, nullptr, (int64_t)n.e * RB + cb, 0, n.q, C,
                               lds_addr(lds.b[wave][slot]));
        return n;
    };

    int slot = 0;
    Item next{};
    if (wave < items && (int)blockIdx.x < RB) next = fetch(blockIdx.x, wave, 0);
    for (int cb = blockIdx.x; cb < RB; cb += turn) {
        const int col = cb * 16 + 4 * kg;
        mx_f4 sum[kMoeTiles];
#pragma unroll
        for (int t = 0; t < kMoeTiles; ++t) sum[t] = mx_f4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int i = wave; i < items; i += kMoeWaves) {
            wait_vmcnt<0>();
            asm volatile("" ::: "memory");  // the weights have landed
            const Item now = next;
            const int here = slot;
            slot ^= 1;
            if (i + kMoeWaves < items)
                next = fetch(cb, i + kMoeWaves, slot);
            else if (cb + turn < RB)
                next = fetch(cb + turn, wave, slot);
            const int t0 = first_tile(now.who);
            mx_f4 bias = {0.0f, 0.0f, 0.0f, 0.0f};
            if (now.q == 0) bias = mx_row4(a.down_bias, a.bias_bf16, (int64_t)now.e * a.hidden + col, col, a.hidden);
#pragma unroll
            for (int t = 0; t < kMoeTiles; ++t) {
                if (t >= tiles) break;
                const uint32_t who = (uint32_t)(now.who >> (t * 16)) & 0xFFFF;
                if (who == 0) continue;
                const int live = __popc(who), before = __popcll(now.who & ((1ull << (t * 16)) - 1));
                for (int p = 0; p < live; p += 4) {
                    const int n = p + (lane >> 4);
                    const int to = n < live ? (int)(lds.list[wave][here][before + n] & 15) : 0;
                    moe_quantize(p == 0 && t == t0 ? now.raw : raw_of(here, now.who, t, p, now.q), a_lds, to, n < live);
                }
                mx_wave_fence();
                const mx_f4 y = moe_multiply<false>(lds.b[wave][here], now.sb, 0, a_lds, bias);
                mx_wave_fence();
                const float w = __shfl(now.weight, t * 16 + r16);
                if (who >> r16 & 1) sum[t] += w * y;
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // LDS is read before it is filled again
        }
#pragma unroll
        for (int t = 0; t < kMoeTiles; ++t)
            if (t < tiles) reinterpret_cast<mx_f4*>(a_lds)[t * 64 + lane] = sum[t];
        __syncthreads();
        if (wave < tiles) {
            mx_f4 s = reinterpret_cast<const mx_f4*>(lds.a[0])[wave * 64 + lane];
#pragma unroll
            for (int w = 1; w < kMoeWaves; ++w) s += reinterpret_cast<const mx_f4*>(lds.a[w])[wave * 64 + lane];
            const int token = wave * 16 + r16;
            if (token < a.tokens) mx_put4(a.out, a.out_bf16, (int64_t)token * a.hidden + col, col, a.hidden, s);
        }
        __syncthreads();
    }
}

}  // namespace

hipError_t launch_mx_moe_few(const MxMoeArgs& a, hipStream_t stream) {
    constexpr int kResident = 3 * 256;  // workgroups that the GPU holds at once
    const bool gated = a.gate_codes != nullptr;
    const int units = a.inner / (gated ? 8 : 16);
    const int most = std::min<int64_t>((int64_t)std::min(a.tokens * a.topk, a.experts) * units, kResident);
    const dim3 up((unsigned)most), down((unsigned)std::min((a.hidden + 15) / 16, kResident)), block(kMoeWG);
    if (gated) {
        if (a.x_bf16)
            hipLaunchKernelGGL((moe_up_kernel<uint16_t, true>), up, block, 0, stream, a);
        else
            hipLaunchKernelGGL((moe_up_kernel<float, true>), up, block, 0, stream, a);
    } else {
        if (a.x_bf16)
            hipLaunchKernelGGL((moe_up_kernel<uint16_t, false>), up, block, 0, stream, a);
        else
            hipLaunchKernelGGL((moe_up_kernel<float, false>), up, block, 0, stream, a);
    }
    const hipError_t error = hipGetLastError();
    if (error != hipSuccess) return error;
    hipLaunchKernelGGL(moe_down_kernel, down, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace nvfp4
