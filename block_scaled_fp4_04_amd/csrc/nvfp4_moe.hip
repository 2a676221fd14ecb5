// nvfp4_moe.hip -- gfx950 kernels of expert routing: the router's choices
// sorted by expert, token rows laid out in that order and added up again,
// and the gradients (include/nvfp4_moe.h).
//
// All of them are bound by memory.  Nothing is added with atomics into
// results: every output element has one writer that adds in the order of
// the token's choices, so results do not depend on timing.
#include <algorithm>
#include <type_traits>

#include "nvfp4_mx_device.h"

namespace nvfp4 {
namespace {

// ---------------------------------------------------------------------------
// Stable counting sort of tokens * topk choices by expert.  Workgroup b ranks
// the choices of its own chunk; for where they go it needs how many choices
// each expert has in the chunks before and behind it.
//
// Up to kSortOne choices (OF_LIST) it counts those itself from the whole list,
// in one launch: the list is short and comes from the L2.  Above
// (OF_HISTOGRAMS) a launch before it has counted every chunk, and a launch
// behind it fills row_tokens from slots: the histograms lie in row_tokens
// meanwhile, so neither form needs a workspace.  (65536 choices, 256 experts:
// 17.8 us in one launch, for the 64 rounds of LDS atomics that every
// workgroup makes.)
//
// Within the chunk each wave ranks its own contiguous part 64 choices at a
// time: lanes with the same expert find each other with one ballot per bit
// of the expert number.
// ---------------------------------------------------------------------------
constexpr int kSortWaves = 16;
constexpr int kSortWG = kSortWaves * 64;
constexpr int kSortChunk = 4096;           // choices a workgroup ranks, at least
constexpr int kSortOne = 4 * kSortChunk;
constexpr int kSortMaxChunks = 1024;       // histograms that a workgroup reads

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

// Counts choices [from, to) into table[], the workgroup over; 16 loads in
// flight (behind a kernel that filled the caches each costs a trip to memory).
template <typename I>
__device__ __forceinline__ void count_choices(const I* ids, int64_t from, int64_t to, int E, int* table) {
    constexpr int U = 16;
    for (int64_t r0 = from + threadIdx.x; r0 < to; r0 += U * kSortWG) {
        int e[U];
#pragma unroll
        for (int u = 0; u < U; ++u) e[u] = expert_of(ids, min(r0 + u * kSortWG, to - 1), E);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (r0 + u * kSortWG < to) atomicAdd(table + e[u], 1);
    }
}

template <typename I, int MAXE>
__global__ void __launch_bounds__(kSortWG) moe_histogram_kernel(MoeArgs a, int64_t chunk) {
    __shared__ int hist[MAXE + 1];
    const int64_t lo = blockIdx.x * chunk, hi = min(lo + chunk, a.tokens * a.topk);
    for (int e = threadIdx.x; e <= a.experts; e += kSortWG) hist[e] = 0;
    __syncthreads();
    count_choices(static_cast<const I*>(a.ids), lo, hi, a.experts, hist);
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kSortWG)
        a.row_tokens[(int64_t)blockIdx.x * a.experts + e] = hist[e];
}

enum { OF_LIST, OF_HISTOGRAMS };

template <typename I, int MAXE, int FROM>
__global__ void __launch_bounds__(kSortWG) moe_sort_kernel(MoeArgs a, int64_t chunk) {
    __shared__ int rest[MAXE + 1];              // choices of each expert behind the chunk
    __shared__ int before[MAXE + 1];            // and before it
    __shared__ int base[kSortWaves][MAXE + 1];  // of each wave's part; then where its next one goes
    __shared__ int wsum[kSortWaves];
    const I* ids = static_cast<const I*>(a.ids);
    const int E = a.experts;
    const int64_t n = a.tokens * a.topk;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t lo = blockIdx.x * chunk, hi = min(lo + chunk, n);
    // the wave's part of the chunk: the waves share what there is
    const int64_t part = ((hi - lo + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
    const int64_t p0 = min(lo + wave * part, hi), p1 = min(p0 + part, hi);
    constexpr int U = 4;  // rounds of a wave whose choices are loaded at once
    int mine[U];
    auto load = [&](int64_t i0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * 64 + lane;
            mine[u] = i < p1 ? expert_of(ids, i, E) : E;
        }
    };
    load(p0);
    for (int e = tid; e <= E; e += kSortWG) {
        rest[e] = before[e] = 0;
        for (int w = 0; w < kSortWaves; ++w) base[w][e] = 0;
    }
    __syncthreads();
    for (int64_t i0 = p0; i0 < p1; i0 += U * 64) {
        if (i0 != p0) load(i0);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u * 64 + lane < p1) atomicAdd(&base[wave][mine[u]], 1);
    }
    if constexpr (FROM == OF_LIST) {
        count_choices(ids, 0, lo, E, before);
        count_choices(ids, hi, n, E, rest);
    } else {
        // a thread of several to an expert, each with every share-th chunk
        const int share = max(kSortWG / E, 1);
        for (int k = tid; k < E * share; k += kSortWG) {
            const int e = k % E;
            int b4 = 0, behind = 0;
            for (int c = k / E; c < (int)gridDim.x; c += share) {
                const int h = a.row_tokens[(int64_t)c * E + e];
                b4 += c < (int)blockIdx.x ? h : 0;
                behind += c > (int)blockIdx.x ? h : 0;
            }
            atomicAdd(&before[e], b4);
            atomicAdd(&rest[e], behind);
        }
    }
    __syncthreads();
    // base[w][e] = where wave w's first choice of e goes
    int run = 0;  // rows of the experts before this round
    for (int e0 = 0; e0 < E; e0 += kSortWG) {
        const int e = e0 + tid;
        int c[kSortWaves], cnt = 0;
        if (e < E) {
            cnt = rest[e] + before[e];
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) cnt += c[w] = base[w][e];
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
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const int s = wsum[w];
            start += w < wave ? s : 0;
            run += s;
        }
        if (e < E) {
            if (blockIdx.x == 0) a.row_offsets[e] = start;
            int at = start + before[e];
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                base[w][e] = at;
                at += c[w];
            }
        }
        __syncthreads();
    }
    const int kept = run;
    if (blockIdx.x == 0 && tid == 0) a.row_offsets[E] = kept;

    const int bits = 32 - __clz(E);
    if (p0 + U * 64 < p1) load(p0);  // (else the part's choices are still here)
    for (int64_t i0 = p0; i0 < p1; i0 += U * 64) {
        if (i0 != p0) load(i0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + u * 64 + lane;
            const bool in = i < p1;
            const int e = mine[u];
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
                    if (FROM == OF_LIST) a.row_tokens[slot] = (int)(i / a.topk);
                }
                a.slots[i] = slot;
                if (FROM == OF_LIST && i >= kept) a.row_tokens[i] = -1;  // rows that no choice fills
            }
            wave_fence();  // every lane has read base before the first lane of an expert moves it on
            if (in && e < E && rank == 0) base[wave][e] += __popcll(same);
            wave_fence();
        }
    }
}

__global__ void __launch_bounds__(256) moe_row_tokens_kernel(MoeArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.tokens * a.topk) return;
    const int slot = a.slots[i];
    if (slot >= 0) a.row_tokens[slot] = (int)(i / a.topk);
    if (i >= a.row_offsets[a.experts]) a.row_tokens[i] = -1;
}

// ---------------------------------------------------------------------------
// Row kernels.  A lane takes a piece of V elements, 16 bytes, of a row; rows
// may start anywhere (unaligned 16-byte accesses cost less than narrow
// ones), and a row's last piece is moved back to end with the row: the
// elements that two pieces share are written twice, with the same values
// (but where input and output may be one buffer).  Rows shorter than a piece take V = 1.
// ---------------------------------------------------------------------------
template <typename T, int V>
struct Piece {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Piece<T, V> load_piece(const T* p) {
    Piece<T, V> r;
    __builtin_memcpy(&r, p, sizeof(r));
    return r;
}
// NT: with the non-temporal hint.
template <bool NT, typename T, int V>
__device__ __forceinline__ void store_piece(T* p, const Piece<T, V>& r) {
    if constexpr (NT && sizeof(r) == 16) {
        typedef unsigned int u4 __attribute__((ext_vector_type(4), aligned(2)));
        u4 t;
        __builtin_memcpy(&t, &r, 16);
        __builtin_nontemporal_store(t, reinterpret_cast<u4*>(p));
    } else {
        __builtin_memcpy(p, &r, sizeof(r));
    }
}
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return __builtin_bit_cast(float, (uint32_t)x << 16); }
__device__ __forceinline__ void narrow(float x, float& o) { o = x; }
__device__ __forceinline__ void narrow(float x, uint16_t& o) { o = mx_to_bf16(x); }

// B choices of token t from the j-th on: their rows, -1 where a choice was
// dropped, is past the last one, or the table is malformed (no access outside
// the buffers), and their weights.  One load for all of them, a choice to a
// lane (scalar loads are not to be had: the tables could alias the output);
// made where the whole wave is active.
template <int B>
struct Choices {
    int row[B];
    float weight[B];
    __device__ __forceinline__ Choices(const MoeArgs& a, int64_t t, int j) {
        const int lane = threadIdx.x & 63;
        const int64_t at = t * a.topk + min(j + lane, a.topk - 1);
        const int x = a.slots[at];
        const int slot = j + lane < a.topk && x >= 0 && x < a.tokens * a.topk ? x : -1;
        const int w = __builtin_bit_cast(int, a.weights ? a.weights[at] : 1.0f);
        // (read out here, where every lane is active: behind a branch the
        // load would be made by the lanes that take it)
#pragma unroll
        for (int b = 0; b < B; ++b) {
            row[b] = __builtin_amdgcn_readlane(slot, b);
            weight[b] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(w, b));
        }
    }
};

// out[slot(t, j)] = x[t] for every kept choice: a token's row is read once.
template <typename T, int V, int B, bool NT>
__global__ void __launch_bounds__(256) moe_gather_kernel(MoeArgs a) {
    const int64_t t = blockIdx.x;
    int64_t col = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V;
    const bool in = col < a.hidden;  // (the lanes past the row's end hold choices, too)
    col = min(col, a.hidden - V);
    const Piece<T, V> r = load_piece<T, V>(static_cast<const T*>(a.x) + t * a.ld_in + col);
    for (int j = 0; j < a.topk; j += B) {
        const Choices<B> c(a, t, j);
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (in && c.row[b] >= 0) store_piece<NT, T, V>(static_cast<T*>(a.out) + (int64_t)c.row[b] * a.hidden + col, r);
    }
}

// out[t] = sum_j w[t][j] * x[slot(t, j)], in fp32 and in the order of j.  B
// rows are read at a time (row 0 in the place of a dropped choice's, unused).
template <typename T, int V, int B, bool NT>
__global__ void __launch_bounds__(256) moe_combine_kernel(MoeArgs a) {
    const int64_t t = blockIdx.x;
    int64_t col = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V;
    const bool in = col < a.hidden;  // (the lanes past the row's end hold choices, too)
    col = min(col, a.hidden - V);
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.0f;
    for (int j = 0; j < a.topk; j += B) {
        const Choices<B> c(a, t, j);
        Piece<T, V> r[B];
#pragma unroll
        for (int b = 0; b < B; ++b)
            r[b] = load_piece<T, V>(static_cast<const T*>(a.x) + (int64_t)max(c.row[b], 0) * a.hidden + col);
#pragma unroll
        for (int b = 0; b < B; ++b)
            if (c.row[b] >= 0)
#pragma unroll
                for (int i = 0; i < V; ++i) sum[i] += c.weight[b] * widen(r[b].v[i]);
    }
    Piece<T, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) narrow(sum[i], o.v[i]);
    if (in) store_piece<NT, T, V>(static_cast<T*>(a.out) + t * a.hidden + col, o);
}

// dy[slot(t, j)] = w[t][j] * dout[t];  dw[t][j] = <dout[t], y[slot(t, j)]>.
// A workgroup per token, B choices at a time; the dot products are added
// over the lanes of a wave and then over the waves, in a fixed order.
template <typename T, int V, int B, bool NT>
__global__ void __launch_bounds__(256) moe_combine_grad_kernel(MoeArgs a) {
    __shared__ float part[2][4][B];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    const T* g = static_cast<const T*>(a.x) + t * a.ld_in;
    for (int j = 0, turn = 0; j < a.topk; j += B, turn ^= 1) {
        const Choices<B> c(a, t, j);
        float dot[B];
#pragma unroll
        for (int b = 0; b < B; ++b) dot[b] = 0.0f;
        for (int64_t k = (int64_t)threadIdx.x * V; k < a.hidden; k += (int64_t)blockDim.x * V) {
            const int64_t col = min(k, a.hidden - V);
            const int again = (int)(k - col);  // elements that the piece before has
            const Piece<T, V> gv = load_piece<T, V>(g + col);
            Piece<T, V> yv[B];
#pragma unroll
            for (int b = 0; b < B; ++b)
                yv[b] = load_piece<T, V>(static_cast<const T*>(a.y) + (int64_t)max(c.row[b], 0) * a.hidden + col);
            T* d = static_cast<T*>(a.out) + col;
            if (again == 0) {
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    if (c.row[b] < 0) continue;
                    Piece<T, V> o;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        dot[b] += widen(gv.v[i]) * widen(yv[b].v[i]);
                        narrow(c.weight[b] * widen(gv.v[i]), o.v[i]);
                    }
                    store_piece<NT, T, V>(d + (int64_t)c.row[b] * a.hidden, o);
                }
            } else {  // only its own elements: dy may be y, and the piece before reads the others
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    if (c.row[b] < 0) continue;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        if (i < again) continue;
                        dot[b] += widen(gv.v[i]) * widen(yv[b].v[i]);
                        narrow(c.weight[b] * widen(gv.v[i]), d[(int64_t)c.row[b] * a.hidden + i]);
                    }
                }
            }
        }
#pragma unroll
        for (int b = 0; b < B; ++b) {
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) dot[b] += __shfl_xor(dot[b], o);
            if (lane == 0) part[turn][wave][b] = dot[b];
        }
        __syncthreads();  // (the other half of part is free again behind the next one)
        if ((int)threadIdx.x < B && j + (int)threadIdx.x < a.topk) {
            float sum = part[turn][0][threadIdx.x];
            for (int x = 1; x < waves; ++x) sum += part[turn][x][threadIdx.x];
            a.dweights[t * a.topk + j + threadIdx.x] = sum;
        }
    }
}

enum RowKernel { GATHER, COMBINE, COMBINE_GRAD };

template <RowKernel K, typename T, int V, int B, bool NT>
hipError_t run_rows(const MoeArgs& a, hipStream_t stream) {
    // whole waves, as many as the row has pieces for
    const int64_t pieces = (a.hidden + V - 1) / V;
    const unsigned threads = pieces >= 256 ? 256 : (unsigned)((pieces + 63) / 64 * 64);
    dim3 grid((unsigned)a.tokens);
    if (K != COMBINE_GRAD) grid.y = (unsigned)((pieces + threads - 1) / threads);
    if constexpr (K == GATHER)
        hipLaunchKernelGGL((moe_gather_kernel<T, V, B, NT>), grid, dim3(threads), 0, stream, a);
    else if constexpr (K == COMBINE)
        hipLaunchKernelGGL((moe_combine_kernel<T, V, B, NT>), grid, dim3(threads), 0, stream, a);
    else
        hipLaunchKernelGGL((moe_combine_grad_kernel<T, V, B, NT>), grid, dim3(threads), 0, stream, a);
    return hipGetLastError();
}

// With rows of more than kStreamBytes every store is non-temporal: a
// gather of 65536 rows of 4 KB takes 50 us instead of 59, a combine of them
// with its gradients 139 instead of 171.  (Non-temporal loads slowed that
// down: the gradient reads the rows again.)
template <RowKernel K, typename T, int V, int B>
hipError_t pick_stores(const MoeArgs& a, hipStream_t stream) {
    return a.tokens * a.topk * a.hidden * (int64_t)sizeof(T) > kStreamBytes ? run_rows<K, T, V, B, true>(a, stream)
                                                             : run_rows<K, T, V, B, false>(a, stream);
}

template <RowKernel K, typename T, int V>
hipError_t pick_batch(const MoeArgs& a, hipStream_t stream) {
    if (a.topk >= 7) return pick_stores<K, T, V, 8>(a, stream);
    if (a.topk >= 3) return pick_stores<K, T, V, 4>(a, stream);
    return pick_stores<K, T, V, 2>(a, stream);
}

template <RowKernel K>
hipError_t pick(const MoeArgs& a, hipStream_t stream) {
    if (a.bf16)
        return a.hidden >= 8 ? pick_batch<K, uint16_t, 8>(a, stream)
                             : run_rows<K, uint16_t, 1, 4, false>(a, stream);
    return a.hidden >= 4 ? pick_batch<K, float, 4>(a, stream) : run_rows<K, float, 1, 4, false>(a, stream);
}

template <typename I, int MAXE>
hipError_t sort(const MoeArgs& a, hipStream_t stream) {
    const int64_t n = a.tokens * a.topk;
    if (n <= kSortOne) {
        const dim3 grid((unsigned)std::max<int64_t>((n + kSortChunk - 1) / kSortChunk, 1));
        hipLaunchKernelGGL((moe_sort_kernel<I, MAXE, OF_LIST>), grid, dim3(kSortWG), 0, stream, a, (int64_t)kSortChunk);
        return hipGetLastError();
    }
    // (kSortMaxChunks of at least kSortChunk choices: their histograms, at most
    // half as many words as choices, fit row_tokens)
    static_assert(2 * kMoeMaxExperts <= kSortChunk && kSortOne >= 2 * kSortChunk, "histograms in row_tokens");
    int64_t chunk = (n + kSortMaxChunks - 1) / kSortMaxChunks;
    chunk = std::max<int64_t>((chunk + kSortChunk - 1) / kSortChunk, 1) * kSortChunk;
    const dim3 grid((unsigned)((n + chunk - 1) / chunk));
    hipLaunchKernelGGL((moe_histogram_kernel<I, MAXE>), grid, dim3(kSortWG), 0, stream, a, chunk);
    hipLaunchKernelGGL((moe_sort_kernel<I, MAXE, OF_HISTOGRAMS>), grid, dim3(kSortWG), 0, stream, a, chunk);
    hipLaunchKernelGGL(moe_row_tokens_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <typename I>
hipError_t sort(const MoeArgs& a, hipStream_t stream) {
    // (the tables of up to 2048 experts take 144 KB of LDS)
    return a.experts <= 256 ? sort<I, 256>(a, stream) : sort<I, kMoeMaxExperts>(a, stream);
}

}  // namespace

hipError_t launch_moe_sort(const MoeArgs& a, hipStream_t stream) {
    return a.wide ? sort<int64_t>(a, stream) : sort<int32_t>(a, stream);
}
hipError_t launch_moe_gather(const MoeArgs& a, hipStream_t stream) { return pick<GATHER>(a, stream); }
hipError_t launch_moe_combine(const MoeArgs& a, hipStream_t stream) { return pick<COMBINE>(a, stream); }
hipError_t launch_moe_combine_grad(const MoeArgs& a, hipStream_t stream) { return pick<COMBINE_GRAD>(a, stream); }

}  // namespace nvfp4
