// nvfp4_norm.hip -- gfx950 kernels of the norms around a block's residual and
// of their gradients (include/nvfp4_layer.h).
//
//   u = post ? y * ry * w_post : y         r_x = 1 / sqrt(mean(x^2) + eps)
//   h = residual_scale * residual + scale * gate * u
//   n = h * rh * w_pre
// Bound by memory: a row is read once into registers, its sums go over the
// waves that share it, and everything is written from there.
//
// Gradients, with t = dn * w_pre and by rows:
//   dw_pre    += dn * h * rh
//   D          = dh + rh * t - h * rh^3 * mean(t * h)
//   dresidual  = residual_scale * D
//   dgate      = scale * D * u                    (a CHANNEL gate's: summed)
//   v          = scale * D * gate * w_post        (without post: dy = scale * D * gate)
//   dw_post   += scale * D * gate * y * ry
//   dy         = ry * v - y * ry^3 * mean(v * y)
// Sums over rows: a workgroup keeps those of its rows in registers, adds its
// teams' through LDS and leaves them in the workspace, and a second launch
// adds the workgroups' in order: no atomics, the same bits every time.
#include "nvfp4_rows.h"

#include <algorithm>

namespace nvfp4 {
namespace {

// The pieces of a row that a lane of a team of W waves takes: the p-th begins
// at column at[p] and has its first skip[p] elements in common with the piece
// before (a row's last one is moved back to end with the row); skip V: none.
template <int V, int W, int P, bool ODD>
struct Columns {
    int at[P], skip[P];
    __device__ __forceinline__ Columns(int hidden, int lane) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int col = (p * W * 64 + lane) * V;
            at[p] = min(col, hidden - V);
            skip[p] = col >= hidden ? V : ODD ? col - at[p] : 0;
        }
    }
    __device__ __forceinline__ bool own(int p, int i) const { return ODD ? i >= skip[p] : skip[p] == 0; }
    // Leaves zeros in the elements that are not the lane's.
    __device__ __forceinline__ void mask(float (&x)[P][V]) const {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < V; ++i) x[p][i] = own(p, i) ? x[p][i] : 0.0f;
    }
    template <typename T>
    __device__ __forceinline__ void load(const T* row, Piece<T, V> (&x)[P]) const {
#pragma unroll
        for (int p = 0; p < P; ++p) x[p] = load_piece<T, V>(row + at[p]);
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

// V weights from column `at` on: of either type, ones without any.
template <int V>
__device__ __forceinline__ void load_weights(const void* w, bool bf16, int at, float (&x)[V]) {
    if (!w) {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = 1.0f;
    } else if (bf16) {
        const Piece<uint16_t, V> r = load_piece<uint16_t, V>(static_cast<const uint16_t*>(w) + at);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = widen(r.v[i]);
    } else {
        const Piece<float, V> r = load_piece<float, V>(static_cast<const float*>(w) + at);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = r.v[i];
    }
}

// Sums of N values over the W waves of each team of a workgroup of WAVES, in a
// fixed order; `turn` alternates between the two halves of `part`: a wave
// writes a half again only behind the barrier of the sum in between (of
// whatever array), which every wave meets with its reads of that half done.
template <int W, int WAVES, int N>
__device__ __forceinline__ void team_sum(float (&x)[N], float (*part)[WAVES][N], int& turn) {
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) x[k] += __shfl_xor(x[k], o);
    if constexpr (W > 1) {
        const int wave = threadIdx.x >> 6, first = wave / W * W;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) part[turn][wave][k] = x[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            x[k] = part[turn][first][k];
#pragma unroll
            for (int w = 1; w < W; ++w) x[k] += part[turn][first + w][k];
        }
        turn ^= 1;
    }
}

// ---- forward ------------------------------------------------------------------

// A team of W waves takes a row at a time; teams of one wave share a workgroup
// of four.
template <typename T, int V, int W, int P, bool ODD>
__global__ void __launch_bounds__(W == 1 ? 256 : W * 64) norm_kernel(NormArgs a, int64_t rows_out) {
    constexpr int WAVES = W == 1 ? 4 : W, TEAMS = WAVES / W;
    __shared__ float part[2][WAVES][1];
    int turn = 0;
    const int lane = threadIdx.x & 63, tid = threadIdx.x % (W * 64);
    const Columns<V, W, P, ODD> c(a.hidden, tid);
    const float mean = 1.0f / (float)a.hidden;
    const int steps = (a.hidden + kMxStep - 1) / kMxStep, words = (steps + 3) / 4;
    // (a team of one wave may leave before the others: it meets no barrier)
    for (int64_t row = (int64_t)blockIdx.x * TEAMS + threadIdx.x / (W * 64); row < rows_out;
         row += (int64_t)gridDim.x * TEAMS) {
        uint8_t* const codes = a.codes + (row >> 4) * steps * kMxFrag;
        uint8_t* const scales = a.scales + (row >> 4) * words * kMxScaleFrag;
        const int r16 = (int)(row & 15);
        if (row >= a.rows) {  // packed rows behind the last one: zeros
            for (int b = tid; b < words * 16; b += W * 64) {
                if (b < steps * 4) *reinterpret_cast<mx_u4*>(codes + (b >> 2) * kMxFrag + mx_code_at(r16, b & 3)) = mx_u4{0, 0, 0, 0};
                scales[(b >> 4) * kMxScaleFrag + mx_scale_at(r16, b & 3) + (b >> 2 & 3)] = 0;
            }
            continue;
        }
        Piece<T, V> y[P], res[P], gate[P];
        float u[P][V];
        c.load(static_cast<const T*>(a.y) + row * a.ld_y, y);
        if (a.residual) c.load(static_cast<const T*>(a.residual) + row * a.ld_residual, res);
        if (a.gate_mode == kGateElement) c.load(static_cast<const T*>(a.gate) + row * a.ld_gate, gate);
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < V; ++i) u[p][i] = widen(y[p].v[i]);
        float w[V];
        if (a.post) {
            c.mask(u);
            float sum[1] = {0.0f};
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < V; ++i) sum[0] += u[p][i] * u[p][i];
            team_sum<W, WAVES, 1>(sum, part, turn);
            const float r = rsqrtf(sum[0] * mean + a.eps);
#pragma unroll
            for (int p = 0; p < P; ++p) {
                load_weights<V>(a.post_weight, a.weight_bf16, c.at[p], w);
#pragma unroll
                for (int i = 0; i < V; ++i) u[p][i] *= r * w[i];
            }
        }
        if (a.gate_mode == kGateElement) {
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < V; ++i) u[p][i] *= widen(gate[p].v[i]);
        } else if (a.gate_mode == kGateChannel) {
#pragma unroll
            for (int p = 0; p < P; ++p) {
                load_weights<V>(a.gate, a.weight_bf16, c.at[p], w);
#pragma unroll
                for (int i = 0; i < V; ++i) u[p][i] *= w[i];
            }
        }
        Piece<T, V> h[P];
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float x = a.scale * u[p][i];
                if (a.residual) x += a.residual_scale * widen(res[p].v[i]);
                narrow(x, h[p].v[i]);
                u[p][i] = widen(h[p].v[i]);
            }
        if (a.h)
#pragma unroll
            for (int p = 0; p < P; ++p) c.store(static_cast<T*>(a.h) + row * a.hidden, p, h[p]);
        if (!a.pre) continue;
        c.mask(u);
        float sum[1] = {0.0f};
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < V; ++i) sum[0] += u[p][i] * u[p][i];
        team_sum<W, WAVES, 1>(sum, part, turn);
        const float r = rsqrtf(sum[0] * mean + a.eps);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            load_weights<V>(a.pre_weight, a.weight_bf16, c.at[p], w);
#pragma unroll
            for (int i = 0; i < V; ++i) u[p][i] *= r * w[i];
        }
        if (a.n) c.store(static_cast<T*>(a.n) + row * a.hidden, u);
        if constexpr (!ODD && V > 1) {
            if (a.codes) {
                // a block's maximum across its lanes, side by side (hidden is
                // a multiple of 32: they all have it or none has)
                constexpr int LPB = kMxBlock / V;
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    Piece<T, V> o;
#pragma unroll
                    for (int i = 0; i < V; ++i) narrow(u[p][i], o.v[i]);
                    mx_u4 v;
                    __builtin_memcpy(&v, &o, 16);
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
                // blocks that fill the last step and the last scale word
                for (int b = a.hidden / kMxBlock + tid; b < words * 16; b += W * 64) {
                    if (b < steps * 4) *reinterpret_cast<mx_u4*>(codes + (b >> 2) * kMxFrag + mx_code_at(r16, b & 3)) = mx_u4{0, 0, 0, 0};
                    scales[(b >> 4) * kMxScaleFrag + mx_scale_at(r16, b & 3) + (b >> 2 & 3)] = 0;
                }
            }
        }
    }
}

// ---- gradients ----------------------------------------------------------------

// Workgroups of 16 waves, 16 / W teams, each a row at a time.  parts: the
// workgroups; the sums of their rows are kept only if they are asked for.
constexpr int kGradWaves = 16;

template <typename T, int V, int W, int P, bool ODD>
__global__ void __launch_bounds__(kGradWaves * 64) norm_grad_kernel(NormArgs a) {
    constexpr int TEAMS = kGradWaves / W;
    __shared__ float part[2][kGradWaves][3], part_dot[2][kGradWaves][1];
    __shared__ float sums[TEAMS > 1 ? TEAMS * W * 64 * V * P : 1];
    int turn = 0;
    const int tid = threadIdx.x % (W * 64), team = threadIdx.x / (W * 64);
    const Columns<V, W, P, ODD> c(a.hidden, tid);
    const float mean = 1.0f / (float)a.hidden;
    float dpre[P][V], dpost[P][V], dgate[P][V];  // sums over the team's rows
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < V; ++i) dpre[p][i] = dpost[p][i] = dgate[p][i] = 0.0f;
    const bool use_y = a.post || a.gate_mode != kGateNone;

    // (every team makes as many turns: the sums of all teams meet at barriers)
    for (int64_t first = (int64_t)blockIdx.x * TEAMS; first < a.rows; first += (int64_t)gridDim.x * TEAMS) {
        const bool live = first + team < a.rows;
        const int64_t row = live ? first + team : a.rows - 1;
        Piece<T, V> ydat[P], gdat[P], hdat[P], ndat[P], ddat[P];
        if (a.pre) {
            c.load(static_cast<const T*>(a.h_in) + row * a.ld_h, hdat);
            c.load(static_cast<const T*>(a.dn) + row * a.ld_dn, ndat);
        }
        if (use_y) c.load(static_cast<const T*>(a.y) + row * a.ld_y, ydat);
        if (a.dh) c.load(static_cast<const T*>(a.dh) + row * a.ld_dh, ddat);
        if (a.gate_mode == kGateElement) c.load(static_cast<const T*>(a.gate) + row * a.ld_gate, gdat);
        const auto own = [&](int p, int i) { return live && c.own(p, i); };
        float sum[3] = {0.0f, 0.0f, 0.0f};  // h^2, t h, y^2
        float d[P][V], w[V];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (a.pre) {
                load_weights<V>(a.pre_weight, a.weight_bf16, c.at[p], w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float h = own(p, i) ? widen(hdat[p].v[i]) : 0.0f, t = own(p, i) ? widen(ndat[p].v[i]) * w[i] : 0.0f;
                    sum[0] += h * h;
                    sum[1] += t * h;
                }
            }
            if (a.post)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float y = own(p, i) ? widen(ydat[p].v[i]) : 0.0f;
                    sum[2] += y * y;
                }
        }
        if (a.pre || a.post) team_sum<W, kGradWaves, 3>(sum, part, turn);
        const float rh = rsqrtf(sum[0] * mean + a.eps), ry = rsqrtf(sum[2] * mean + a.eps);
        const float back = rh * rh * rh * (sum[1] * mean);
#pragma unroll
        for (int p = 0; p < P; ++p) {
#pragma unroll
            for (int i = 0; i < V; ++i) d[p][i] = a.dh ? widen(ddat[p].v[i]) : 0.0f;
            if (a.pre) {
                load_weights<V>(a.pre_weight, a.weight_bf16, c.at[p], w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float h = widen(hdat[p].v[i]), g = widen(ndat[p].v[i]);
                    d[p][i] += rh * (g * w[i]) - back * h;
                    dpre[p][i] += own(p, i) ? g * h * rh : 0.0f;
                }
            }
        }
        if (a.dresidual && live)
#pragma unroll
            for (int p = 0; p < P; ++p) {
                Piece<T, V> o;
#pragma unroll
                for (int i = 0; i < V; ++i) narrow(a.residual_scale * d[p][i], o.v[i]);
                c.store(static_cast<T*>(a.dresidual) + row * a.hidden, p, o);
            }
        // d: scale * D, then times the gate
        float dot[1] = {0.0f};
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float wp[V], gate[V];
            if (a.post) load_weights<V>(a.post_weight, a.weight_bf16, c.at[p], wp);
            if (a.gate_mode == kGateChannel) load_weights<V>(a.gate, a.weight_bf16, c.at[p], gate);
            Piece<T, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float x = a.scale * d[p][i];
                if (a.gate_mode != kGateNone) {
                    const float y = widen(ydat[p].v[i]), g = x * (a.post ? y * ry * wp[i] : y);
                    narrow(g, o.v[i]);
                    if (a.gate_mode == kGateChannel) dgate[p][i] += own(p, i) ? g : 0.0f;
                    x *= a.gate_mode == kGateChannel ? gate[i] : widen(gdat[p].v[i]);
                }
                if (a.post) {
                    const float y = own(p, i) ? widen(ydat[p].v[i]) : 0.0f;
                    dpost[p][i] += own(p, i) ? x * y * ry : 0.0f;
                    x *= wp[i];
                    dot[0] += own(p, i) ? x * y : 0.0f;
                }
                d[p][i] = x;
            }
            if (a.gate_mode == kGateElement && a.dgate && live) c.store(static_cast<T*>(a.dgate) + row * a.hidden, p, o);
        }
        if (a.post) {
            team_sum<W, kGradWaves, 1>(dot, part_dot, turn);
            const float along = ry * ry * ry * (dot[0] * mean);
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < V; ++i) d[p][i] = ry * d[p][i] - along * widen(ydat[p].v[i]);
        }
        if (a.dy && live) c.store(static_cast<T*>(a.dy) + row * a.hidden, d);
    }

    // The teams' sums, added in their order, to the workspace.
    if (!a.partials) return;
    const auto leave = [&](const float (&x)[P][V], int which) {
        float* const out = a.partials + ((int64_t)blockIdx.x * 3 + which) * a.hidden;
        if constexpr (TEAMS > 1) {
            __syncthreads();
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int i = 0; i < V; ++i) sums[((team * P + p) * V + i) * W * 64 + tid] = x[p][i];
            __syncthreads();
            if (team > 0) return;
        }
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float s = x[p][i];
                if constexpr (TEAMS > 1)
                    for (int t = 1; t < TEAMS; ++t) s += sums[((t * P + p) * V + i) * W * 64 + tid];
                if (c.own(p, i)) out[c.at[p] + i] = s;
            }
    };
    if (a.dpre_weight) leave(dpre, 0);
    if (a.dpost_weight) leave(dpost, 1);
    if (a.gate_mode == kGateChannel && a.dgate) leave(dgate, 2);
}

// Adds the workgroups' sums: 64 columns to a workgroup, 16 waves that each take
// every sixteenth.
__global__ void __launch_bounds__(1024) norm_grad_sum_kernel(NormArgs a) {
    __shared__ float part[16][64];
    const int which = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float* const out = which == 0 ? a.dpre_weight : which == 1 ? a.dpost_weight
                     : a.gate_mode == kGateChannel ? static_cast<float*>(a.dgate) : nullptr;
    if (!out) return;
    const int col = blockIdx.x * 64 + lane, at = min(col, a.hidden - 1);
    float s = 0.0f;
#pragma unroll 4
    for (int k = wave; k < a.parts; k += 16) s += a.partials[((int64_t)k * 3 + which) * a.hidden + at];
    part[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || col >= a.hidden) return;
#pragma unroll
    for (int w = 1; w < 16; ++w) s += part[w][lane];
    out[col] = s;
}

// ---- launches -----------------------------------------------------------------

template <typename T, int V, int W, int P, bool ODD>
hipError_t run_norm(const NormArgs& a, hipStream_t stream) {
    constexpr int TEAMS = W == 1 ? 4 : 1, THREADS = W == 1 ? 256 : W * 64;
    const int64_t rows = a.codes ? mx_round_up(a.rows, kMxRows) : a.rows;
    // (work-items of a launch stay below 2^32)
    const int64_t grid = std::min<int64_t>((rows + TEAMS - 1) / TEAMS, 1 << 20);
    hipLaunchKernelGGL((norm_kernel<T, V, W, P, ODD>), dim3((unsigned)grid), dim3(THREADS), 0, stream, a, rows);
    return hipGetLastError();
}

template <typename T, int V, int W, int P>
hipError_t run_norm(const NormArgs& a, hipStream_t stream) {
    return a.hidden % V ? run_norm<T, V, W, P, true>(a, stream) : run_norm<T, V, W, P, false>(a, stream);
}

// Waves to a row: as few as keep it in the registers of four pieces a lane.
template <typename T, int V>
hipError_t pick_norm(const NormArgs& a, hipStream_t stream) {
    if (a.hidden < V) return run_norm<T, 1, 1, 1, false>(a, stream);
    const int n = ((a.hidden + V - 1) / V + 63) / 64;  // pieces to a lane of one wave
    if (n <= 1) return run_norm<T, V, 1, 1>(a, stream);
    if (n <= 2) return run_norm<T, V, 1, 2>(a, stream);
    if (n <= 4) return run_norm<T, V, 4, 1>(a, stream);
    if (n <= 8) return run_norm<T, V, 4, 2>(a, stream);
    if (n <= 12) return run_norm<T, V, 4, 3>(a, stream);
    if (n <= 16) return run_norm<T, V, 4, 4>(a, stream);
    if (n <= 32) return run_norm<T, V, 16, 2>(a, stream);
    if constexpr (V == 4) return run_norm<T, V, 16, 4>(a, stream);
    return hipErrorInvalidValue;  // (hidden is at most kNormMaxHidden)
}

// Waves to a row of a gradient: as few as keep it in two pieces a lane.
template <typename T, int V, typename F>
auto with_team(int hidden, F&& f) {
    const int n = ((hidden + V - 1) / V + 63) / 64;
    if (n <= 1) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{});
    if (n <= 2) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 2>{});
    if (n <= 4) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
    if (n <= 8) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
    if (n <= 16) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
    if (V == 8 || n <= 32) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 16>{}, std::integral_constant<int, V == 8 ? 2 : 4>{});
}

constexpr int kGradParts = 256;  // one workgroup of 16 waves for each CU

template <typename T, int V>
int parts_of(int64_t rows, int hidden) {
    if (hidden < V) return (int)std::min<int64_t>((rows + 15) / 16, kGradParts);
    return with_team<T, V>(hidden, [&](auto W, auto) {
        constexpr int teams = kGradWaves / W.value;
        return (int)std::min<int64_t>((rows + teams - 1) / teams, kGradParts);
    });
}

template <typename T, int V>
hipError_t pick_grad(const NormArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)a.parts), block(kGradWaves * 64);
    if (a.rows == 0) {
        // (no rows: the sums are zeros, which the launch below writes)
    } else if (a.hidden < V) {
        hipLaunchKernelGGL((norm_grad_kernel<T, 1, 1, 1, false>), grid, block, 0, stream, a);
    } else {
        with_team<T, V>(a.hidden, [&](auto W, auto P) {
            if (a.hidden % V)
                hipLaunchKernelGGL((norm_grad_kernel<T, V, W.value, P.value, true>), grid, block, 0, stream, a);
            else
                hipLaunchKernelGGL((norm_grad_kernel<T, V, W.value, P.value, false>), grid, block, 0, stream, a);
            return 0;
        });
    }
    if (a.partials || a.rows == 0)
        hipLaunchKernelGGL(norm_grad_sum_kernel, dim3((unsigned)((a.hidden + 63) / 64), 3), dim3(1024), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t stream) {
    return a.bf16 ? pick_norm<uint16_t, 8>(a, stream) : pick_norm<float, 4>(a, stream);
}
hipError_t launch_norm_grad(const NormArgs& a, hipStream_t stream) {
    return a.bf16 ? pick_grad<uint16_t, 8>(a, stream) : pick_grad<float, 4>(a, stream);
}
int norm_grad_parts(bool bf16, int64_t rows, int hidden) {
    return bf16 ? parts_of<uint16_t, 8>(rows, hidden) : parts_of<float, 4>(rows, hidden);
}

}  // namespace nvfp4
