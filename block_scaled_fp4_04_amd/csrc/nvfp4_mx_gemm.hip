// nvfp4_mx_gemm.hip -- gfx950 kernels of the MXFP4 product
//   C[m][n] = alpha * sum_k a'[m][k] * b'[n][k]
// single and grouped, from packed operands or from fp32 / bfloat16
// activations that are quantised on the way (include/nvfp4_mx.h).
//
// The scaled MFMAs of gfx950 take E2M1 codes and E8M0 scales as they are
// held, so nothing is decoded: a lane loads the 16 code bytes of one block
// straight into its operand registers and names one byte of a scale word.
// Products of codes are exact; the sums are kept in fp32.
#include "nvfp4_mx_device.h"

#include <type_traits>

namespace nvfp4 {
namespace {

// ---------------------------------------------------------------------------
// Split kernel: the waves of a workgroup share one output tile of 16 MI x
// 16 NI and split its K range, four steps (one scale word) at a time.  Each
// wave loads its operands straight into registers; the wave tiles are added
// in LDS in wave order, so results do not depend on timing.
//
// A operand of v_mfma_scale_f32_16x16x128: B's rows; B operand: A's rows; so
// lane l ends up with row l % 16 of A and four consecutive columns of C.
//
// GROUPED: group g owns rows offsets[g] .. offsets[g+1]-1 of C; a workgroup
// takes one column tile of one group and walks its rows.  Offsets are
// clamped to [0, M] and row numbers to A's rows, so a malformed table gives
// wrong rows but no access outside the buffers.
// ---------------------------------------------------------------------------
enum { A_PACKED = 0, A_F32 = 1, A_BF16 = 2 };

template <int MI, int NI, int W, int AT, bool GROUPED>
__global__ void __launch_bounds__(W * 64) mx_split_kernel(MxGemmArgs a) {
    __shared__ mx_f4 red[W][MI * NI][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, kg = lane >> 4;
    const int C = a.C, Q = (C + 3) / 4;
    const int tiles_n = (a.RBb + NI - 1) / NI;
    const int tn = (int)(blockIdx.x % (unsigned)tiles_n);
    const int tm = (int)(blockIdx.x / (unsigned)tiles_n);  // row tile, or group
    const int cb0 = tn * NI;
    int r0 = tm * 16 * MI, r1 = min(r0 + 16 * MI, a.M);
    const uint8_t* bc = a.b_codes;
    const uint8_t* bs = a.b_scales;
    if constexpr (GROUPED) {
        r0 = min(max(a.offsets[tm], 0), a.M);
        r1 = min(max(a.offsets[tm + 1], r0), a.M);
        bc += (int64_t)tm * a.RBb * C * kMxFrag;
        bs += (int64_t)tm * a.RBb * Q * kMxScaleFrag;
    }
    // this lane's pieces of the column tile's row blocks (past B's end: its last)
    const uint8_t* bcp[NI];
    const uint8_t* bsp[NI];
#pragma unroll
    for (int j = 0; j < NI; ++j) {
        const int64_t rb = min(cb0 + j, a.RBb - 1);
        bcp[j] = bc + rb * C * kMxFrag + lane * 16;
        bsp[j] = bs + rb * Q * kMxScaleFrag + lane * 4;
    }

    for (int m0 = r0; m0 < r1; m0 += 16 * MI) {
        int64_t arow[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            int r = min(m0 + i * 16 + r16, r1 - 1);
            if (GROUPED && a.a_rows) r = min(max(a.a_rows[r], 0), a.A_rows - 1);
            arow[i] = r;
        }
        mx_f4 acc[MI][NI];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) acc[i][j] = mx_f4{0.0f, 0.0f, 0.0f, 0.0f};

        for (int q = wave; q < Q; q += W) {
            uint32_t sb[NI], sa[MI];
            mx_u4 wb[4][NI], wa[4][MI];
#pragma unroll
            for (int j = 0; j < NI; ++j) sb[j] = *reinterpret_cast<const uint32_t*>(bsp[j] + (int64_t)q * kMxScaleFrag);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int64_t c = min(4 * q + s, C - 1);
#pragma unroll
                for (int j = 0; j < NI; ++j) wb[s][j] = *reinterpret_cast<const mx_u4*>(bcp[j] + c * kMxFrag);
            }
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                if constexpr (AT == A_PACKED) {
                    const int64_t rb = arow[i] >> 4;
                    const int rr = (int)(arow[i] & 15);
                    sa[i] = *reinterpret_cast<const uint32_t*>(a.a_scales + (rb * Q + q) * kMxScaleFrag + kg * 64 + rr * 4);
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int64_t c = min(4 * q + s, C - 1);
                        wa[s][i] = *reinterpret_cast<const mx_u4*>(a.a_codes + (rb * C + c) * kMxFrag + kg * 256 + rr * 16);
                    }
                } else {
                    sa[i] = 0;
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int k = (4 * q + s) * kMxStep + kg * kMxBlock;
                        const bool live = k < a.K;
                        uint32_t byte;
                        const int64_t at = arow[i] * a.ldx + (live ? k : 0);
                        if constexpr (AT == A_F32)
                            byte = mx_quant_load(static_cast<const float*>(a.x) + at, wa[s][i]);
                        else
                            byte = mx_quant_load(static_cast<const uint16_t*>(a.x) + at, wa[s][i]);
                        if (!live) wa[s][i] = mx_u4{0, 0, 0, 0};
                        sa[i] |= (live ? byte : 0u) << (8 * s);
                    }
                }
            }
            const int n = min(4, C - 4 * q);  // steps of this word (uniform)
            auto step = [&](auto S) {
                if (S.value < n) {
#pragma unroll
                    for (int i = 0; i < MI; ++i)
#pragma unroll
                        for (int j = 0; j < NI; ++j)
                            acc[i][j] = mx_mfma16<S.value>(wb[S.value][j], sb[j], wa[S.value][i], sa[i], acc[i][j]);
                }
            };
            step(std::integral_constant<int, 0>{});
            step(std::integral_constant<int, 1>{});
            step(std::integral_constant<int, 2>{});
            step(std::integral_constant<int, 3>{});
        }

        if (m0 != r0) __syncthreads();  // the previous rows' sums are read
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NI; ++j) red[wave][i * NI + j][lane] = acc[i][j];
        __syncthreads();
        for (int f = wave; f < MI * NI; f += W) {
            mx_f4 sum = red[0][f][lane];
#pragma unroll
            for (int w = 1; w < W; ++w) sum += red[w][f][lane];
            const int row = m0 + (f / NI) * 16 + r16;
            const int col = (cb0 + f % NI) * 16 + 4 * kg;
            if (row >= r1 || col >= a.N) continue;
            const int64_t at = (int64_t)row * a.N + col;
            if ((a.N & 3) == 0) {
                if (a.out_bf16) {
                    uint2 o;
                    o.x = mx_to_bf16(a.alpha * sum[0]) | (uint32_t)mx_to_bf16(a.alpha * sum[1]) << 16;
                    o.y = mx_to_bf16(a.alpha * sum[2]) | (uint32_t)mx_to_bf16(a.alpha * sum[3]) << 16;
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = o;
                } else {
                    *reinterpret_cast<mx_f4*>(static_cast<float*>(a.out) + at) = sum * a.alpha;
                }
            } else {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    if (col + v >= a.N) break;
                    if (a.out_bf16)
                        static_cast<uint16_t*>(a.out)[at + v] = mx_to_bf16(a.alpha * sum[v]);
                    else
                        static_cast<float*>(a.out)[at + v] = a.alpha * sum[v];
                }
            }
        }
    }
}

// Launches (a stream given) or only measures the grid: the work-items.
struct Launch {
    const MxGemmArgs& a;
    hipStream_t stream;
    bool dry;
    int64_t items;
    hipError_t error;
};

template <int MI, int NI, int W, int AT, bool GROUPED>
void run_split(Launch& l) {
    const MxGemmArgs& a = l.a;
    const int64_t tiles_n = (a.RBb + NI - 1) / NI;
    const int64_t tiles_m = GROUPED ? a.groups : (a.M + 16 * MI - 1) / (16 * MI);
    l.items = tiles_m * tiles_n * W * 64;
    if (l.dry) return;
    hipLaunchKernelGGL((mx_split_kernel<MI, NI, W, AT, GROUPED>), dim3((unsigned)(tiles_m * tiles_n)),
                       dim3(W * 64), 0, l.stream, a);
    l.error = hipGetLastError();
}

template <int AT>
void run_few_rows(Launch& l) {
    if (l.a.M <= 16) return run_split<1, 1, 16, AT, false>(l);
    if (l.a.M <= 32) return run_split<2, 1, 16, AT, false>(l);
    return run_split<4, 1, 16, AT, false>(l);
}

void choose(Launch& l) {
    const MxGemmArgs& a = l.a;
    if (a.groups > 0) {
        if (a.M / a.groups <= 32) return run_split<2, 4, 4, A_PACKED, true>(l);
        return run_split<4, 4, 8, A_PACKED, true>(l);
    }
    if (!a.a_codes) return a.x_bf16 ? run_few_rows<A_BF16>(l) : run_few_rows<A_F32>(l);
    if (a.M <= 64) return run_few_rows<A_PACKED>(l);
    return run_split<4, 4, 8, A_PACKED, false>(l);
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t stream) {
    Launch l{a, stream, false, 0, hipSuccess};
    choose(l);
    return l.error;
}

bool mx_gemm_fits(const MxGemmArgs& a) {
    Launch l{a, nullptr, true, 0, hipSuccess};
    choose(l);
    return l.items < ((int64_t)1 << 32);
}

}  // namespace nvfp4
