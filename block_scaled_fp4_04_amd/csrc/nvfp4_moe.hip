// nvfp4_moe.hip -- gfx950 kernels of expert routing: the router's choices
// sorted by expert, token rows laid out in that order and added up again,
// and the gradients (include/nvfp4_moe.h).
//
// All of them are bound by memory.  Nothing is added with atomics into
// results: every output element has one writer that adds in the order of
// the token's choices, so results do not depend on timing.
#include <type_traits>

#include "nvfp4_mx_device.h"

namespace nvfp4 {
namespace {

// ---------------------------------------------------------------------------
// Stable counting sort of tokens * topk choices by expert, in one launch and
// without a workspace.  Workgroup b ranks the choices of its own chunk; for
// where they go it needs how many choices each expert has before the chunk
// and in all, and counts those itself from the whole list: the list is small
// beside the rows it steers (4 bytes for each row of kilobytes) and comes
// from the L2, which costs less than a second launch would.
//
// Within the chunk each wave ranks its own contiguous part 64 choices at a
// time: lanes with the same expert find each other with one ballot per bit
// of the expert number.
// ---------------------------------------------------------------------------
constexpr int kSortWaves = 16;
constexpr int kSortChunk = 4096;  // choices a workgroup ranks
constexpr int kSortPart = kSortChunk / kSortWaves;

// Orders the LDS accesses of a wave's lanes among each other.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <typename I>
__device__ __forceinline__ int expert_of(const I* ids, int64_t i, int E) {
    const I e = ids[i];
    return e >= 0 && e < (I)E ? (int)e : E;  // E: dropped
}

template <typename I, int MAXE>
__global__ void __launch_bounds__(kSortWaves * 64) moe_sort_kernel(MoeArgs a) {
    __shared__ int all[MAXE + 1];             // choices of each expert, then where its rows begin
    __shared__ int base[kSortWaves][MAXE + 1];  // of each wave's part, then where its next choice goes
    __shared__ int before[MAXE + 1];          // before the chunk
    __shared__ int wsum[kSortWaves];
    const I* ids = static_cast<const I*>(a.ids);
    const int E = a.experts;
    const int64_t n = a.tokens * a.topk;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t lo = (int64_t)blockIdx.x * kSortChunk, hi = min(lo + kSortChunk, n);

    for (int e = tid; e <= E; e += kSortWaves * 64) {
        all[e] = before[e] = 0;
        for (int w = 0; w < kSortWaves; ++w) base[w][e] = 0;
    }
    __syncthreads();
    for (int64_t i = tid; i < n; i += kSortWaves * 64) {
        const int e = expert_of(ids, i, E);
        if (i < lo)
            atomicAdd(&before[e], 1);
        else if (i < hi)
            atomicAdd(&base[(i - lo) / kSortPart][e], 1);
        else
            atomicAdd(&all[e], 1);
    }
    __syncthreads();
    // all[e] = where expert e's rows begin; base[w][e] = where wave w's first choice of e goes
    int run = 0;  // rows of the experts before this round
    for (int e0 = 0; e0 < E; e0 += kSortWaves * 64) {
        const int e = e0 + tid;
        int cnt = 0;
        if (e < E) {
            cnt = all[e] + before[e];
            for (int w = 0; w < kSortWaves; ++w) cnt += base[w][e];
        }
        int incl = cnt;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int y = __shfl_up(incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 63) wsum[wave] = incl;
        __syncthreads();
        int start = run + incl - cnt;
        int sum = 0;
        for (int w = 0; w < kSortWaves; ++w) {
            if (w < wave) start += wsum[w];
            sum += wsum[w];
        }
        if (e < E) {
            all[e] = start;
            if (blockIdx.x == 0) a.row_offsets[e] = start;
            int at = start + before[e];
            for (int w = 0; w < kSortWaves; ++w) {
                const int c = base[w][e];
                base[w][e] = at;
                at += c;
            }
        }
        run += sum;
        __syncthreads();
    }
    const int kept = run;
    if (blockIdx.x == 0 && tid == 0) a.row_offsets[E] = kept;

    int bits = 1;
    while ((1 << bits) <= E) ++bits;
    for (int64_t i0 = lo + wave * kSortPart; i0 < min(lo + (wave + 1) * (int64_t)kSortPart, hi); i0 += 64) {
        const int64_t i = i0 + lane;
        const bool in = i < hi;
        const int e = in ? expert_of(ids, i, E) : E;
        uint64_t same = __ballot(in);
        for (int b = 0; b < bits; ++b) {
            const uint64_t m = __ballot((e >> b) & 1);
            same &= ((e >> b) & 1) ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        if (in) {
            int slot = -1;
            if (e < E) {
                slot = base[wave][e] + rank;
                a.row_tokens[slot] = (int)(i / a.topk);
            }
            a.slots[i] = slot;
            if (i >= kept) a.row_tokens[i] = -1;  // rows that no choice fills
        }
        wave_fence();  // every lane has read base before the first lane of an expert moves it on
        if (in && e < E && rank == 0) base[wave][e] += __popcll(same);
        wave_fence();
    }
}

// ---------------------------------------------------------------------------
// Row kernels.  A row is walked in pieces of V elements per lane, V the widest
// that the row length and the addresses allow.
// ---------------------------------------------------------------------------
template <typename T, int V>
struct Piece {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Piece<T, V> load_piece(const T* p) {
    Piece<T, V> r;
    __builtin_memcpy(&r, __builtin_assume_aligned(p, sizeof(T) * V), sizeof(r));
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_piece(T* p, const Piece<T, V>& r) {
    __builtin_memcpy(__builtin_assume_aligned(p, sizeof(T) * V), &r, sizeof(r));
}
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return __builtin_bit_cast(float, (uint32_t)x << 16); }
__device__ __forceinline__ void narrow(float x, float& o) { o = x; }
__device__ __forceinline__ void narrow(float x, uint16_t& o) { o = mx_to_bf16(x); }

// The row of choice (t, j), or -1 where it was dropped (or the table is
// malformed: no access outside the buffers).
__device__ __forceinline__ int64_t slot_of(const MoeArgs& a, int64_t t, int j) {
    const int s = a.slots[t * a.topk + j];
    return s >= 0 && s < a.tokens * a.topk ? s : -1;
}

// out[slot(t, j)] = x[t] for every kept choice: a token's row is read once.
template <typename T, int V>
__global__ void __launch_bounds__(256) moe_gather_kernel(MoeArgs a) {
    const int64_t t = blockIdx.x;
    const int64_t col = ((int64_t)blockIdx.y * 256 + threadIdx.x) * V;
    if (col >= a.hidden) return;
    const Piece<T, V> r = load_piece<T, V>(static_cast<const T*>(a.x) + t * a.ld_in + col);
    for (int j = 0; j < a.topk; ++j) {
        const int64_t s = slot_of(a, t, j);
        if (s >= 0) store_piece<T, V>(static_cast<T*>(a.out) + s * a.hidden + col, r);
    }
}

// out[t] = sum_j w[t][j] * x[slot(t, j)], in fp32 and in the order of j.
template <typename T, int V>
__global__ void __launch_bounds__(256) moe_combine_kernel(MoeArgs a) {
    const int64_t t = blockIdx.x;
    const int64_t col = ((int64_t)blockIdx.y * 256 + threadIdx.x) * V;
    if (col >= a.hidden) return;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.0f;
    for (int j = 0; j < a.topk; ++j) {
        const int64_t s = slot_of(a, t, j);
        if (s < 0) continue;
        const float w = a.weights ? a.weights[t * a.topk + j] : 1.0f;
        const Piece<T, V> r = load_piece<T, V>(static_cast<const T*>(a.x) + s * a.hidden + col);
#pragma unroll
        for (int i = 0; i < V; ++i) sum[i] += w * widen(r.v[i]);
    }
    Piece<T, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) narrow(sum[i], o.v[i]);
    store_piece<T, V>(static_cast<T*>(a.out) + t * a.hidden + col, o);
}

// dy[slot(t, j)] = w[t][j] * dout[t];  dw[t][j] = <dout[t], y[slot(t, j)]>.
// A workgroup per token; the dot products are added over the lanes of a
// wave and then over the waves, in a fixed order.
template <typename T, int V>
__global__ void __launch_bounds__(256) moe_combine_grad_kernel(MoeArgs a) {
    __shared__ float part[4];
    const int64_t t = blockIdx.x;
    const T* g = static_cast<const T*>(a.x) + t * a.ld_in;
    for (int j = 0; j < a.topk; ++j) {
        const int64_t s = slot_of(a, t, j);
        float dot = 0.0f;
        if (s >= 0) {
            const float w = a.weights ? a.weights[t * a.topk + j] : 1.0f;
            for (int64_t col = threadIdx.x * V; col < a.hidden; col += 256 * V) {
                const Piece<T, V> gv = load_piece<T, V>(g + col);
                const Piece<T, V> yv = load_piece<T, V>(static_cast<const T*>(a.y) + s * a.hidden + col);
                Piece<T, V> o;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dot += widen(gv.v[i]) * widen(yv.v[i]);
                    narrow(w * widen(gv.v[i]), o.v[i]);
                }
                store_piece<T, V>(static_cast<T*>(a.out) + s * a.hidden + col, o);
            }
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o);
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
        __syncthreads();
        if (threadIdx.x == 0) a.dweights[t * a.topk + j] = part[0] + part[1] + part[2] + part[3];
        __syncthreads();
    }
}

// Elements per lane: as many as 16 bytes hold, halved until rows and
// addresses are aligned to the piece.
inline int piece_of(const MoeArgs& a) {
    const int size = a.bf16 ? 2 : 4;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out) |
                         reinterpret_cast<uintptr_t>(a.y) | (uintptr_t)(a.hidden * size) |
                         (uintptr_t)(a.ld_in * size);
    int bytes = 16;
    while (bytes > size && (at & (uintptr_t)(bytes - 1))) bytes >>= 1;
    return bytes / size;
}

template <template <typename, int> class K, typename T>
hipError_t pick(const MoeArgs& a, hipStream_t stream) {
    switch (piece_of(a)) {
        case 8: if constexpr (sizeof(T) == 2) return K<T, 8>::go(a, stream);
        case 4: return K<T, 4>::go(a, stream);
        case 2: return K<T, 2>::go(a, stream);
        default: return K<T, 1>::go(a, stream);
    }
}
template <typename T, int V>
struct Gather {
    static hipError_t go(const MoeArgs& a, hipStream_t s) {
        const dim3 grid((unsigned)a.tokens, (unsigned)((a.hidden + 256 * V - 1) / (256 * V)));
        hipLaunchKernelGGL((moe_gather_kernel<T, V>), grid, dim3(256), 0, s, a);
        return hipGetLastError();
    }
};
template <typename T, int V>
struct Combine {
    static hipError_t go(const MoeArgs& a, hipStream_t s) {
        const dim3 grid((unsigned)a.tokens, (unsigned)((a.hidden + 256 * V - 1) / (256 * V)));
        hipLaunchKernelGGL((moe_combine_kernel<T, V>), grid, dim3(256), 0, s, a);
        return hipGetLastError();
    }
};
template <typename T, int V>
struct CombineGrad {
    static hipError_t go(const MoeArgs& a, hipStream_t s) {
        hipLaunchKernelGGL((moe_combine_grad_kernel<T, V>), dim3((unsigned)a.tokens), dim3(256), 0, s, a);
        return hipGetLastError();
    }
};

template <typename I>
hipError_t sort(const MoeArgs& a, hipStream_t stream) {
    const int64_t n = a.tokens * a.topk;
    const dim3 grid((unsigned)(n > 0 ? (n + kSortChunk - 1) / kSortChunk : 1)), block(kSortWaves * 64);
    if (a.experts <= 256)
        hipLaunchKernelGGL((moe_sort_kernel<I, 256>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((moe_sort_kernel<I, kMoeMaxExperts>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_sort(const MoeArgs& a, hipStream_t stream) {
    return a.wide ? sort<int64_t>(a, stream) : sort<int32_t>(a, stream);
}
hipError_t launch_moe_gather(const MoeArgs& a, hipStream_t stream) {
    return a.bf16 ? pick<Gather, uint16_t>(a, stream) : pick<Gather, float>(a, stream);
}
hipError_t launch_moe_combine(const MoeArgs& a, hipStream_t stream) {
    return a.bf16 ? pick<Combine, uint16_t>(a, stream) : pick<Combine, float>(a, stream);
}
hipError_t launch_moe_combine_grad(const MoeArgs& a, hipStream_t stream) {
    return a.bf16 ? pick<CombineGrad, uint16_t>(a, stream) : pick<CombineGrad, float>(a, stream);
}

}  // namespace nvfp4
