// nvfp4_norm_kernels.h -- gfx950 kernels of the norms around a block's residual and
// of their gradients (include/nvfp4_layer.h).
//
//   u = post ? y * ry * w_post : y         r_x = 1 / sqrt(mean(x^2) + eps)
//   h = residual_scale * residual + scale * gate * u
//   n = h * rh * w_pre
// Bound by memory: a row is read once into registers, its sums go over the
// waves that share it, and everything is written from there.
//
// What a call has (a norm behind the block, a gate, weights of which type) is
// a template argument: with branches on it every load waits for the sums
// before it (16384 x 6144 bfloat16 with all parts 416 us, and 201 without
// them).  A lane takes one 16-byte piece as long as 16 waves hold a row (two to
// a lane 286 us, three 216, four 259; gradients of 8192 x 2048 bfloat16 57 with
// one, 65 with two).
//
// Gradients, with t = dn * w_pre and by rows:
//   dw_pre    += dn * h * rh
//   D          = dh + rh * (t - h * rh * mean(t * h * rh))
//   dresidual  = residual_scale * D
//   dgate      = scale * D * u                    (a CHANNEL gate's: summed)
//   v          = scale * D * gate * w_post        (without post: dy = scale * D * gate)
//   dw_post   += scale * D * gate * y * ry
//   dy         = ry * (v - y * ry * mean(v * y * ry))
// (rh goes with h and ry with y: their cubes leave fp32's normal range from an
// rms of 2^42 on, and below 2^-42)
// 8192 x 2048 bfloat16 with all parts 49 us, 4.1 TB/s, and 5 for the sums' second
// launch: 16 waves a CU at 128 registers.  (Of a form that took 50: the next row's
// loads ahead of the sums spilled, 78 us; pieces of 8 bytes at twice the waves
// spilled, 106; two workgroups of 8 waves a CU 55.6.)  Rows of more than 8192 elements
// spill: 4096 x 9000 bfloat16 584 us.
// Sums over rows: a workgroup keeps those of its rows in registers, adds its
// teams' through LDS and leaves them in the workspace, and a second launch
// adds the workgroups' in order: no atomics, the same bits every time.
#pragma once
#include "nvfp4_rows.h"

#include <algorithm>
#include <type_traits>

namespace nvfp4 {
namespace {

// The pieces of a row that a lane of a team of `threads` takes: the p-th begins
// at column at[p] and has its first skip[p] elements in common with the piece
// before (ODD: a row's last one is moved back to end with the row); skip V:
// none.
template <int V, int P, bool ODD>
struct Columns {
    int at[P], skip[P];
    __device__ __forceinline__ Columns(int hidden, int threads, int lane) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int col = (p * threads + lane) * V;
            at[p] = min(col, hidden - V);
            skip[p] = col >= hidden ? V : ODD ? col - at[p] : 0;
        }
    }
    // Reads a row's pieces, with zeros in the elements that are not the lane's
    // (and in all of them without `live`).
    template <typename T>
    __device__ __forceinline__ void load(const T* row, Piece<T, V> (&x)[P], bool live = true) const {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            x[p] = load_piece<T, V>(row + at[p]);
            if constexpr (ODD) {
#pragma unroll
                for (int i = 0; i < V; ++i) x[p].v[i] = live && i >= skip[p] ? x[p].v[i] : (T)0;
            } else if (!live || skip[p] != 0) {
                x[p] = Piece<T, V>{};
            }
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, int p, const Piece<T, V>& x) const {
        if (skip[p] == 0) {
            store_piece<false, T, V>(row + at[p], x);
        } else if (ODD) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i >= skip[p]) row[at[p] + i] = x.v[i];
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, const float (&x)[P][V]) const {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            Piece<T, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) narrow(x[p][i], o.v[i]);
            store(row, p, o);
        }
    }
};

// Weights: bfloat16 (WB) or fp32 ones; a tensor that is not given is ones.
__device__ const float kNormOnes[8] = {1, 1, 1, 1, 1, 1, 1, 1};
__device__ const uint16_t kNormOnesBf16[8] = {0x3F80, 0x3F80, 0x3F80, 0x3F80, 0x3F80, 0x3F80, 0x3F80, 0x3F80};
template <int V, bool WB>
struct Weights {
    using E = std::conditional_t<WB, uint16_t, float>;
    Piece<E, V> x;
    __device__ __forceinline__ void load(const void* w, int at) {
        const E* p;
        if constexpr (WB)
            p = w ? static_cast<const E*>(w) + at : kNormOnesBf16;
        else
            p = w ? static_cast<const E*>(w) + at : kNormOnes;
        x = load_piece<E, V>(p);
    }
    __device__ __forceinline__ float operator[](int i) const { return widen(x.v[i]); }
};

// Sums of N values over the `waves` waves, from wave `first` of the workgroup
// on, that share a row, in a fixed order.  `turn` alternates between the two
// halves of `part`: a wave writes a half again only behind the barrier of the
// sum in between (of whatever array), which every wave meets with its reads of
// that half done.
template <int N>
__device__ __forceinline__ void team_sum(float (&x)[N], float (*part)[16][N], int& turn, int first, int waves) {
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) x[k] += __shfl_xor(x[k], o);
    if (waves == 1) return;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int k = 0; k < N; ++k) part[turn][threadIdx.x >> 6][k] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = part[turn][first][k];
    for (int w = 1; w < waves; ++w)
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] += part[turn][first + w][k];
    turn ^= 1;
}

// What is the same in every lane, in a scalar register.
__device__ __forceinline__ float uniform(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
}
// Squares are added as x^2 2^-k over a row, 2^k above its length: the sum then
// passes fp32's range where the mean does, not before, and no other bit changes.
// Squares that become too small for that do not count beside an eps of 1e-30;
// with a smaller one k is 0, and small rows keep their bits.  (In scalar registers:
// 16384 x 6144 bfloat16 with all parts 189 us, 206 in vector ones.)
struct Squares {
    float down, mean;  // 2^-k; 2^k / hidden
    __device__ __forceinline__ Squares(int hidden, float eps) {
        const int k = eps >= 1e-30f ? 32 - __builtin_clz(hidden) : 0;
        down = uniform(__builtin_bit_cast(float, (127 - k) << 23));
        mean = uniform(1.0f / (float)hidden * __builtin_bit_cast(float, (127 + k) << 23));
    }
    __device__ __forceinline__ float of(float x) const { return x * down * x; }
};

// ---- forward ------------------------------------------------------------------

// A workgroup takes a row at a time; or, if one wave holds a row, four.
// ELEMENT: a gate for every element; else one for every channel (ones).  The
// bound on registers lets two workgroups of 12 waves share a CU (six waves a
// SIMD: 263 -> 206 us for the call above, now 189, 5.3 TB/s).
template <typename T, int V, int P, bool ODD, bool POST, bool ELEMENT, bool WB>
__global__ void __launch_bounds__(1024, P == 1 ? 6 : 4) norm_kernel(NormArgs a, int64_t rows_out, int waves) {
    __shared__ float part[2][16][1];
    int turn = 0;
    const int lane = threadIdx.x & 63;
    const int teams = waves == 1 ? 4 : 1, threads = waves * 64;
    const int tid = waves == 1 ? lane : (int)threadIdx.x;
    const Columns<V, P, ODD> c(a.hidden, threads, tid);
    const Squares sq(a.hidden, a.eps);
    const int steps = (a.hidden + kMxStep - 1) / kMxStep, words = (steps + 3) / 4;
    // (a team of one wave may leave before the others: it meets no barrier)
    for (int64_t row = (int64_t)blockIdx.x * teams + (waves == 1 ? threadIdx.x >> 6 : 0); row < rows_out;
         row += (int64_t)gridDim.x * teams) {
        uint8_t* const codes = a.codes + (row >> 4) * steps * kMxFrag;
        uint8_t* const scales = a.scales + (row >> 4) * words * kMxScaleFrag;
        const int r16 = (int)(row & 15);
        // zeros in block b of the packed row
        auto clear = [&](int b) {
            if (b < steps * 4) *reinterpret_cast<mx_u4*>(codes + (b >> 2) * kMxFrag + mx_code_at(r16, b & 3)) = mx_u4{0, 0, 0, 0};
            scales[(b >> 4) * kMxScaleFrag + mx_scale_at(r16, b & 3) + (b >> 2 & 3)] = 0;
        };
        if (row >= a.rows) {  // packed rows behind the last one
            for (int b = tid; b < words * 16; b += threads) clear(b);
            continue;
        }
        // (rows stay in registers as they are read and stored; widening a value
        // again costs less than the registers of its fp32 form)
        Piece<T, V> y[P], res[P], gate[P];
        Weights<V, WB> wpost[P], wgate[P], wpre[P];
        c.load(static_cast<const T*>(a.y) + row * a.ld_y, y);
        if (a.residual) {
            c.load(static_cast<const T*>(a.residual) + row * a.ld_residual, res);
        } else {
#pragma unroll
            for (int p = 0; p < P; ++p) res[p] = Piece<T, V>{};
        }
        if constexpr (ELEMENT) c.load(static_cast<const T*>(a.gate) + row * a.ld_gate, gate);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if constexpr (POST) wpost[p].load(a.post_weight, c.at[p]);
            if constexpr (!ELEMENT) wgate[p].load(a.gate, c.at[p]);
            wpre[p].load(a.pre ? a.pre_weight : nullptr, c.at[p]);
        }
        float ry = 1.0f;
        if constexpr (POST) {
            float sum[1] = {0.0f};
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < V; ++i) sum[0] += sq.of(widen(y[p].v[i]));
            team_sum<1>(sum, part, turn, 0, waves);
            ry = rsqrtf(sum[0] * sq.mean + a.eps);
        }
        float sum[1] = {0.0f};  // h^2
#pragma unroll
        for (int p = 0; p < P; ++p) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float u = widen(y[p].v[i]);
                if constexpr (POST) u *= ry * wpost[p][i];
                u *= ELEMENT ? widen(gate[p].v[i]) : wgate[p][i];
                narrow(a.residual_scale * widen(res[p].v[i]) + a.scale * u, y[p].v[i]);  // now h
                const float h2 = sq.of(widen(y[p].v[i]));
                sum[0] += (ODD ? i >= c.skip[p] : c.skip[p] == 0) ? h2 : 0.0f;
            }
            if (a.h) c.store(static_cast<T*>(a.h) + row * a.hidden, p, y[p]);
        }
        if (!a.pre) continue;
        team_sum<1>(sum, part, turn, 0, waves);
        const float rh = rsqrtf(sum[0] * sq.mean + a.eps);
#pragma unroll
        for (int p = 0; p < P; ++p) {
#pragma unroll
            for (int i = 0; i < V; ++i) narrow(widen(y[p].v[i]) * (rh * wpre[p][i]), y[p].v[i]);  // now n
            if (a.n) c.store(static_cast<T*>(a.n) + row * a.hidden, p, y[p]);
        }
        if constexpr (!ODD && V > 1) {
            if (a.codes) {
                // a block's maximum across its lanes, side by side (hidden is
                // a multiple of 32: they all have it or none has)
                constexpr int LPB = kMxBlock / V;
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    mx_u4 v;
                    __builtin_memcpy(&v, &y[p], 16);
                    const uint32_t byte = mx_scale_byte(mx_block_top<LPB>(mx_top<T>(v)));
                    const uint32_t q = byte == 255u ? 0u : mx_codes<T, 0>(0, v, mx_scale(byte));
                    if (c.skip[p] == 0) {
                        const int step = c.at[p] / kMxStep, b = c.at[p] % kMxStep / kMxBlock;
                        uint8_t* d = codes + step * kMxFrag + mx_code_at(r16, b) + c.at[p] % kMxBlock / 2;
                        if constexpr (V == 8)
                            *reinterpret_cast<uint32_t*>(d) = q;
                        else
                            *reinterpret_cast<uint16_t*>(d) = (uint16_t)q;
                        if (lane % LPB == 0)
                            scales[(step >> 2) * kMxScaleFrag + mx_scale_at(r16, b) + (step & 3)] = (uint8_t)byte;
                    }
                }
                // the blocks that fill the last step and the last scale word
                for (int b = a.hidden / kMxBlock + tid; b < words * 16; b += threads) clear(b);
            }
        }
    }
}

// ---- gradients ----------------------------------------------------------------

// Up to 16 waves to a workgroup, as many teams of `waves` as they make, each a
// row at a time.  What is not a lane's own is read as zeros, which add nothing
// anywhere.
constexpr int kGradWaves = 16;

template <typename T, int V, int P, bool ODD, bool POST, int GATE, bool WB>
__global__ void __launch_bounds__(kGradWaves * 64) norm_grad_kernel(NormArgs a, int waves) {
    constexpr bool USE_Y = POST || GATE != kGateNone;
    __shared__ float part[2][16][POST ? 3 : 2], part_dot[2][16][1];
    __shared__ float sums[P == 1 ? kGradWaves * 64 * V : 1];
    int turn = 0;
    const int threads = waves * 64, teams = (int)blockDim.x / threads;
    // (the team in a scalar register, and with it the rows' addresses: 8192 x 2048
    // bfloat16 54.6 us, 58.9 otherwise; rows of several pieces to a lane have one
    // team, and 2053 x 5003 fp32 took 79.4 so, 78.4 otherwise)
    const int tid = threadIdx.x % threads, team = P > 1 ? (int)threadIdx.x / threads : __builtin_amdgcn_readfirstlane((int)threadIdx.x / threads), first_wave = team * waves;
    const Columns<V, P, ODD> c(a.hidden, threads, tid);
    const float mean = uniform(1.0f / (float)a.hidden);
    const Squares sq(a.hidden, a.eps);
    float dpre[P][V], dpost[P][V], dgate[P][V];  // sums over the team's rows
    Weights<V, WB> wpre[P], wpost[P], wgate[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
#pragma unroll
        for (int i = 0; i < V; ++i) dpre[p][i] = dpost[p][i] = dgate[p][i] = 0.0f;
        wpre[p].load(a.pre ? a.pre_weight : nullptr, c.at[p]);
        if constexpr (POST) wpost[p].load(a.post_weight, c.at[p]);
        if constexpr (GATE == kGateChannel) wgate[p].load(a.gate, c.at[p]);
    }

    // (every team makes as many turns: the sums of all teams meet at barriers)
    for (int64_t first = (int64_t)blockIdx.x * teams; first < a.rows; first += (int64_t)gridDim.x * teams) {
        const bool live = first + team < a.rows;
        const int64_t row = live ? first + team : a.rows - 1;
        Piece<T, V> y[P], gate[P], h[P], n[P], dh[P];
#pragma unroll
        for (int p = 0; p < P; ++p) h[p] = n[p] = dh[p] = Piece<T, V>{};
        if (a.pre) {
            c.load(static_cast<const T*>(a.h_in) + row * a.ld_h, h, live);
            c.load(static_cast<const T*>(a.dn) + row * a.ld_dn, n, live);
        }
        if (a.dh) c.load(static_cast<const T*>(a.dh) + row * a.ld_dh, dh, live);
        if constexpr (USE_Y) c.load(static_cast<const T*>(a.y) + row * a.ld_y, y, live);
        if constexpr (GATE == kGateElement) c.load(static_cast<const T*>(a.gate) + row * a.ld_gate, gate, live);
        float sum[POST ? 3 : 2] = {};  // h^2, t h, y^2
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float x = widen(h[p].v[i]);
                sum[0] += sq.of(x);
                sum[1] += widen(n[p].v[i]) * wpre[p][i] * x;
                if constexpr (POST) sum[2] += sq.of(widen(y[p].v[i]));
            }
        if (POST || a.pre) team_sum(sum, part, turn, first_wave, waves);
        // (no norm or no row: nothing but zeros, also with an eps of 0)
        const float rh = live && a.pre ? rsqrtf(sum[0] * sq.mean + a.eps) : 0.0f;
        const float back = sum[1] * mean * rh;  // mean(t h) / rms
        float ry = 0.0f;
        if constexpr (POST) ry = live ? rsqrtf(sum[2] * sq.mean + a.eps) : 0.0f;
        float dot[1] = {0.0f}, d[P][V];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            Piece<T, V> dres, dg;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float x = widen(h[p].v[i]) * rh, g = widen(n[p].v[i]);
                float v = widen(dh[p].v[i]) + rh * (g * wpre[p][i] - back * x);
                dpre[p][i] += g * x;
                narrow(a.residual_scale * v, dres.v[i]);
                v *= a.scale;
                if constexpr (GATE != kGateNone) {
                    const float u = POST ? widen(y[p].v[i]) * ry * wpost[p][i] : widen(y[p].v[i]);
                    if constexpr (GATE == kGateChannel) {
                        dgate[p][i] += v * u;
                        v *= wgate[p][i];
                    } else {
                        narrow(v * u, dg.v[i]);
                        v *= widen(gate[p].v[i]);
                    }
                }
                if constexpr (POST) {
                    const float z = widen(y[p].v[i]) * ry;
                    dpost[p][i] += v * z;
                    v *= wpost[p][i];
                    dot[0] += v * z;
                }
                d[p][i] = v;
            }
            if (a.dresidual && live) c.store(static_cast<T*>(a.dresidual) + row * a.hidden, p, dres);
            if (GATE == kGateElement && a.dgate && live) c.store(static_cast<T*>(a.dgate) + row * a.hidden, p, dg);
        }
        if constexpr (POST) {
            team_sum<1>(dot, part_dot, turn, first_wave, waves);
            const float along = dot[0] * mean;
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < V; ++i) d[p][i] = ry * (d[p][i] - along * (widen(y[p].v[i]) * ry));
        }
        if (a.dy && live) c.store(static_cast<T*>(a.dy) + row * a.hidden, d);
    }

    // The teams' sums, added in their order, to the workspace.
    if (!a.partials) return;
    const auto leave = [&](const float (&x)[P][V], int which) {
        float* const out = a.partials + ((int64_t)blockIdx.x * 3 + which) * a.hidden;
        if constexpr (P == 1) {
            if (teams > 1) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < V; ++i) sums[(team * V + i) * threads + tid] = x[0][i];
                __syncthreads();
                if (team > 0) return;
            }
        }
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float s = x[p][i];
                if constexpr (P == 1)
                    for (int t = 1; t < teams; ++t) s += sums[(t * V + i) * threads + tid];
                if (ODD ? i >= c.skip[p] : c.skip[p] == 0) out[c.at[p] + i] = s;
            }
    };
    if (a.dpre_weight) leave(dpre, 0);
    if (POST && a.dpost_weight) leave(dpost, 1);
    if (GATE == kGateChannel && a.dgate) leave(dgate, 2);
}

// ---- launches -----------------------------------------------------------------

// A row's waves: a piece to a lane up to 16 of them, then two or four.
struct Team {
    int pieces, waves;
};
template <int V>
Team team_of(int hidden) {
    const int n = ((hidden + V - 1) / V + 63) / 64, pieces = n <= 16 ? 1 : n <= 32 ? 2 : 4;
    return {pieces, (n + pieces - 1) / pieces};
}

constexpr int kGradParts = 256;  // one workgroup for each CU

template <int V>
int parts_of(int64_t rows, int hidden) {
    const int teams = kGradWaves / team_of<V>(hidden).waves;
    return (int)std::min<int64_t>((rows + teams - 1) / teams, kGradParts);
}

// Calls f(elements of a piece, pieces of a lane, whether rows end inside one).
template <int V, typename F>
void with_shape(int hidden, F&& f) {
    using std::integral_constant;
    auto odd = [&](auto P) {
        if (hidden % V)
            f(integral_constant<int, V>{}, P, std::true_type{});
        else
            f(integral_constant<int, V>{}, P, std::false_type{});
    };
    if (hidden < V) return f(integral_constant<int, 1>{}, integral_constant<int, 1>{}, std::false_type{});
    const int pieces = team_of<V>(hidden).pieces;
    if (pieces == 1) return odd(integral_constant<int, 1>{});
    if (pieces == 2) return odd(integral_constant<int, 2>{});
    // (16-bit rows of up to kNormMaxHidden take two pieces at most)
    if constexpr (V == 4) odd(integral_constant<int, 4>{});
}
template <typename F>
void with_bool(bool b, F&& f) {
    if (b)
        f(std::true_type{});
    else
        f(std::false_type{});
}

template <typename T, int V>
hipError_t run_norm(const NormArgs& a, hipStream_t stream) {
    const int waves = team_of<V>(a.hidden).waves, teams = waves == 1 ? 4 : 1;
    const int64_t rows = a.codes ? mx_round_up(a.rows, kMxRows) : a.rows;
    // (work-items of a launch stay below 2^32)
    const dim3 grid((unsigned)std::min<int64_t>((rows + teams - 1) / teams, 1 << 20)), block(waves * teams * 64);
    with_shape<V>(a.hidden, [&](auto W, auto P, auto ODD) {
        with_bool(a.post, [&](auto POST) {
            with_bool(a.gate_mode == kGateElement, [&](auto ELEMENT) {
                with_bool(a.weight_bf16, [&](auto WB) {
                    hipLaunchKernelGGL((norm_kernel<T, W.value, P.value, ODD.value, POST.value, ELEMENT.value, WB.value>),
                                       grid, block, 0, stream, a, rows, waves);
                });
            });
        });
    });
    return hipGetLastError();
}

template <typename T, int V>
hipError_t run_grad(const NormArgs& a, hipStream_t stream) {
    const int waves = team_of<V>(a.hidden).waves;
    const dim3 grid((unsigned)a.parts), block(kGradWaves / waves * waves * 64);
    with_shape<V>(a.hidden, [&](auto W, auto P, auto ODD) {
        with_bool(a.post, [&](auto POST) {
            with_bool(a.weight_bf16, [&](auto WB) {
                auto gate = [&](auto GATE) {
                    hipLaunchKernelGGL((norm_grad_kernel<T, W.value, P.value, ODD.value, POST.value, GATE.value, WB.value>),
                                       grid, block, 0, stream, a, waves);
                };
                if (a.gate_mode == kGateNone)
                    gate(std::integral_constant<int, kGateNone>{});
                else if (a.gate_mode == kGateChannel)
                    gate(std::integral_constant<int, kGateChannel>{});
                else
                    gate(std::integral_constant<int, kGateElement>{});
            });
        });
    });
    return hipGetLastError();
}

}  // namespace
}  // namespace nvfp4
