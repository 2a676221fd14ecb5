// nvfp4_mx_short.hip -- gfx950 kernel of the grouped MXFP4 product of short
// rows, K up to 512, by many small groups: the way back of a layer of experts
// (include/nvfp4_layer.h).
//   C[r][n] = sum_k a'[r][k] * b'_g[n][k] + bias[g][n]     rows r of group g
//
// Bound by the weights.  A tile of the grouped product has one or two steps
// here: it is loaded, multiplied and stored one after the other.  So every
// wave works by itself on a run of the units (16 rows of one group, 32
// columns) in the groups' order: the rows stay in its registers from unit to
// unit, and the weights of the two units behind are on their way while one is
// multiplied.  256 experts x (6144 x 256), us with tiles and here: 128
// choices 26.4 and 17.6, 512 choices 52.5 and 36 (138 MB of weights).  With two
// scale words to a row (K up to 1024) it was slower than tiles.
#include "nvfp4_mx_parts.h"

#include <algorithm>

namespace nvfp4 {
namespace {

constexpr int kShortWaves = 4;
constexpr int kShortWG = kShortWaves * 64;

__global__ void __launch_bounds__(kShortWG) mx_short_kernel(MxGemmArgs a, MxEpilogueArgs e) {
    constexpr int NB = 2;  // row blocks of B to a unit
    __shared__ int tiles_to[kMoeMaxExperts];  // row tiles of the groups up to each, itself among them
    __shared__ int of_wave[kShortWaves];
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int C = a.C, G = a.groups;
    auto rows_of = [&](int g, int& r0, int& r1) {
        r0 = min(max(a.offsets[g], 0), a.M);
        r1 = min(max(a.offsets[g + 1], r0), a.M);
    };
    // The groups' tiles, counted up: a run of groups to a thread.
    const int per = (G + kShortWG - 1) / kShortWG, g_lo = min(tid * per, G), g_hi = min(g_lo + per, G);
    int mine = 0;
    for (int g = g_lo; g < g_hi; ++g) {
        int r0, r1;
        rows_of(g, r0, r1);
        mine += (r1 - r0 + 15) / 16;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 63) of_wave[wave] = incl;
    __syncthreads();
    int at = incl - mine;
    for (int w = 0; w < wave; ++w) at += of_wave[w];
    for (int g = g_lo; g < g_hi; ++g) {
        int r0, r1;
        rows_of(g, r0, r1);
        at += (r1 - r0 + 15) / 16;
        tiles_to[g] = at;
    }
    __syncthreads();

    // The wave's units: (tile, columns), columns running fastest.
    const int CB = (a.RBb + NB - 1) / NB;
    const int64_t units = (int64_t)tiles_to[G - 1] * CB, waves = (int64_t)gridDim.x * kShortWaves;
    const int64_t me = (int64_t)blockIdx.x * kShortWaves + wave;
    const int64_t first = units * me / waves, last = units * (me + 1) / waves;
    if (first >= last) return;  // (nothing waits for the wave any more)
    int tile = __builtin_amdgcn_readfirstlane((int)(first / CB));
    int cols = __builtin_amdgcn_readfirstlane((int)(first % CB));
    int left = __builtin_amdgcn_readfirstlane((int)(last - first));

    // A tile's group: the first whose count passes it.
    auto group_of = [&](int t) {
        int lo = 0, hi = G - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (tiles_to[mid] > t)
                hi = mid;
            else
                lo = mid + 1;
        }
        return __builtin_amdgcn_readfirstlane(lo);
    };
    struct Weights {
        mx_u4 w[NB][4];
        uint32_t s[NB];
    };
    auto load_b = [&](int g, int cb) {
        Weights f;
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int64_t rb = (int64_t)g * a.RBb + min(cb * NB + j, a.RBb - 1);  // (past the end: the last one, not stored)
            const uint8_t* const codes = a.b_codes + rb * C * kMxFrag + mx_code_at(r16, kg);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                f.w[j][s] = mx_u4{0, 0, 0, 0};
                if (s < C) f.w[j][s] = *reinterpret_cast<const mx_u4*>(codes + s * kMxFrag);
            }
            f.s[j] = *reinterpret_cast<const uint32_t*>(a.b_scales + rb * kMxScaleFrag + mx_scale_at(r16, kg));
        }
        return f;
    };
    // Walks the units two ahead of the one that is multiplied.
    int tile_b = tile, cols_b = cols, left_b = left, g_b = group_of(tile);
    auto next_b = [&] {
        const Weights f = load_b(g_b, cols_b);
        if (--left_b > 0 && ++cols_b == CB) {
            cols_b = 0;
            g_b = group_of(++tile_b);
        }
        return f;
    };
    Weights now = next_b(), next;
    if (left > 1) next = next_b();

    while (left > 0) {
        const int g = group_of(tile);
        int r0, r1;
        rows_of(g, r0, r1);
        const int m0 = r0 + (tile - (g > 0 ? tiles_to[g - 1] : 0)) * 16, row = m0 + r16;
        const bool live = row < r1;
        mx_u4 wa[4];
        uint32_t sa = 0;
#pragma unroll
        for (int s = 0; s < 4; ++s) wa[s] = mx_u4{0, 0, 0, 0};
        if (live) {
            const uint8_t* const codes = a.a_codes + (int64_t)(row >> 4) * C * kMxFrag + mx_code_at(row & 15, kg);
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (s < C) wa[s] = *reinterpret_cast<const mx_u4*>(codes + s * kMxFrag);
            sa = *reinterpret_cast<const uint32_t*>(a.a_scales + (int64_t)(row >> 4) * kMxScaleFrag + mx_scale_at(row & 15, kg));
        }
        for (; cols < CB && left > 0; ++cols, --left) {
            Weights after;
            if (left > 2) after = next_b();
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const int col = (cols * NB + j) * 16 + 4 * kg;
                mx_f4 acc = mx_row4(e.bias, e.bias_bf16, (int64_t)g * a.N + col, col, a.N);
                mx_each<4>([&](auto S) { acc = mx_mfma16<S.value>(now.w[j][S.value], now.s[j], wa[S.value], sa, acc); });
                acc = mx_pin(acc);
                if (live && col < a.N) mx_put4(a.out, a.out_bf16, (int64_t)row * a.N + col, col, a.N, acc);
            }
            now = next;
            next = after;
        }
        cols = 0;
        ++tile;
    }
}

}  // namespace

hipError_t launch_mx_short(const MxGemmArgs& a, const MxEpilogueArgs& e, hipStream_t stream) {
    hipLaunchKernelGGL(mx_short_kernel, dim3(2 * 256), dim3(kShortWG), 0, stream, a, e);
    return hipGetLastError();
}

}  // namespace nvfp4
