// nvfp4_mx_gemm.hip -- gfx950 kernels of the MXFP4 product
//   C[m][n] = alpha * sum_k a'[m][k] * b'[n][k]
// single and grouped, from packed operands or from fp32 / bfloat16
// activations that are quantised on the way (include/nvfp4_mx.h).
//
// The scaled MFMAs of gfx950 take E2M1 codes and E8M0 scales as they are
// held, so nothing is decoded: a lane loads the 16 code bytes of one block
// straight into its operand registers and names one byte of a scale word.
// Products of codes are exact; the sums are kept in fp32.
#include "nvfp4_device.h"
#include "nvfp4_mx_device.h"

#include <type_traits>
#include <utility>

namespace nvfp4 {
namespace {

// dma16 / dma4 (nvfp4_device.h) with the LDS address as a uniform base plus a
// constant: one scalar instruction a load.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int BYTES, int AT>
__device__ __forceinline__ void mx_dma(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff,
                                       uint32_t lds) {
    if constexpr (BYTES == 16)
        asm volatile("s_add_u32 m0, %3, %4\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                     :: "v"(voff), "s"(r), "s"(soff), "s"(lds), "n"(AT) : "memory", "m0", "scc");
    else
        asm volatile("s_add_u32 m0, %3, %4\n\tbuffer_load_dword %0, %1, %2 offen lds"
                     :: "v"(voff), "s"(r), "s"(soff), "s"(lds), "n"(AT) : "memory", "m0", "scc");
}
#pragma clang diagnostic pop

// f(integral_constant<int, 0>) ... f(integral_constant<int, N - 1>)
template <typename F, int... I>
__device__ __forceinline__ void mx_each(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void mx_each(F&& f) { mx_each(f, std::make_integer_sequence<int, N>{}); }

// Four consecutive columns of C, scaled and rounded; N need not be a multiple
// of anything.
__device__ __forceinline__ void mx_store4(const MxGemmArgs& a, int row, int col, mx_f4 f) {
    if (col >= a.N) return;
    const int64_t at = (int64_t)row * a.N + col;
    if ((a.N & 3) == 0) {
        if (a.out_bf16) {
            uint2 o;
            o.x = mx_to_bf16(a.alpha * f[0]) | (uint32_t)mx_to_bf16(a.alpha * f[1]) << 16;
            o.y = mx_to_bf16(a.alpha * f[2]) | (uint32_t)mx_to_bf16(a.alpha * f[3]) << 16;
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = o;
        } else {
            *reinterpret_cast<mx_f4*>(static_cast<float*>(a.out) + at) = f * a.alpha;
        }
        return;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        if (col + v >= a.N) break;
        if (a.out_bf16)
            static_cast<uint16_t*>(a.out)[at + v] = mx_to_bf16(a.alpha * f[v]);
        else
            static_cast<float*>(a.out)[at + v] = a.alpha * f[v];
    }
}

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
        bcp[j] = bc + rb * C * kMxFrag + mx_code_at(r16, kg);
        bsp[j] = bs + rb * Q * kMxScaleFrag + mx_scale_at(r16, kg);
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
                    sa[i] = *reinterpret_cast<const uint32_t*>(a.a_scales + (rb * Q + q) * kMxScaleFrag + mx_scale_at(rr, kg));
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const int64_t c = min(4 * q + s, C - 1);
                        wa[s][i] = *reinterpret_cast<const mx_u4*>(a.a_codes + (rb * C + c) * kMxFrag + mx_code_at(rr, kg));
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
            if (row < r1) mx_store4(a, row, col, sum);
        }
    }
}

// ---------------------------------------------------------------------------
// Tile kernel: output tiles of BM x BN, four waves in a 2 x 2 grid, each with
// (BM / 2) x (BN / 2) of the tile in 32 x 32 blocks of
// v_mfma_scale_f32_32x32x64_f8f6f4 (measured alone: 6.6 PFLOP/s, against 4.7
// for the 16 x 16 x 128 form: half the operand reads per product).
//
// The fragments of the packed layout (16 rows x one step, 1 KB) go from
// memory to LDS as they are (direct-to-LDS loads, 16 bytes a lane) into a
// ring of NS steps, and the scale words, four steps at a time, to a buffer of
// their own.  A lane then reads its 16 code bytes with one LDS read, 16 lanes
// side by side.  Operands of a 64-element half step are read while the MFMAs
// of the half before run.  One barrier a step, in its middle: every wave has
// then read all of the step's buffer, which takes the loads of step + NS, and
// the next step's loads have landed.
//
// Rows past the operands' ends read as zeros (the buffers' range check) and
// are not stored.  Steps past the last one load it again, unused.
// ---------------------------------------------------------------------------
template <int BM, int BN, int NS, int WM, int KS, bool GROUPED>
__global__ void __launch_bounds__(KS * 256, KS > 1 || BM * BN > 128 * 256 ? KS : 2) mx_tile_kernel(MxGemmArgs a, int tiles_m, int tiles_n) {
    constexpr int WN = 4 / WM;                            // waves along M and N
    constexpr int MI = BM / 32 / WM, NI = BN / 32 / WN;   // 32 x 32 blocks of a wave
    constexpr int AF = BM / 16, BF = BN / 16;             // fragments of a step
    constexpr int CPW = (AF + BF) / 4;                    // of them, a wave's loads
    constexpr int SPW = CPW;                              // a wave's scale loads, every fourth step
    constexpr int STAGE = (AF + BF) * kMxFrag;
    constexpr int SCALES = (AF + BF) * kMxScaleFrag;      // of four steps
    // (NS <= 4: the next scale word's loads, issued in the middle of a word's
    // first step, have landed in the middle of its last one)
    static_assert((AF + BF) % 4 == 0 && NS >= 2 && NS <= 4 && NS * CPW + SPW < 64, "ring");
    constexpr int RING = NS * STAGE + SCALES;
    static_assert(BM * WN * (BN / WN * 2 + 16) <= RING, "the output is staged in the first ring");
    static_assert((KS - 1) * BM * BN * 4 <= KS * RING, "and partial tiles in all");
    __shared__ __attribute__((aligned(1024))) uint8_t lds_all[KS * RING];

    const int lane = threadIdx.x & 63;
    const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave = wave_all & 3, team = KS > 1 ? wave_all >> 2 : 0;
    uint8_t* lds = lds_all + team * RING;
    const int wm = wave / WN, wn = wave % WN;
    const int C = a.C, Q = (C + 3) / 4;

    // Consecutive workgroups go to the eight XCDs in turn: each XCD gets a
    // contiguous range of tiles, so that the tiles that run together share
    // their operands in its L2: walked in groups of 8 along M, or, grouped,
    // row block by row block in the groups' order.
    auto tile_of = [&](int total) {  // -1: none
        const int x = blockIdx.x & 7, per = total >> 3, more = total & 7;
        const int k = blockIdx.x >> 3;
        return k < per + (x < more) ? x * per + min(x, more) + k : -1;
    };
    int tn, m0, row_end = a.M;
    int64_t b_first;  // first row block of this tile's B
    if constexpr (GROUPED) {
        // Row blocks are numbered in group order, ceil(rows / BM) to a group;
        // the grid is an upper bound.  Each thread counts those of a run of
        // groups, and the one whose run holds this tile's publishes it.
        constexpr int NW = 4 * KS;
        int* sch = reinterpret_cast<int*>(lds_all);
        const int tid = threadIdx.x;
        const int per = (a.groups + NW * 64 - 1) / (NW * 64);
        const int g_lo = (int)min((int64_t)tid * per, (int64_t)a.groups), g_hi = min(g_lo + per, a.groups);
        auto rows_of = [&](int g, int& r0, int& r1) {
            r0 = min(max(a.offsets[g], 0), a.M);
            r1 = min(max(a.offsets[g + 1], r0), a.M);
        };
        int64_t cnt = 0;  // (a malformed table may count up to groups * M rows)
        for (int g = g_lo; g < g_hi; ++g) {
            int r0, r1;
            rows_of(g, r0, r1);
            cnt += (r1 - r0 + BM - 1) / BM;
        }
        const int mine = (int)min(cnt, (int64_t)1 << 22);  // (M < 2^28: no more in a sound one)
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int y = __shfl_up(incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 63) sch[wave_all] = incl;
        __syncthreads();
        // (the XCDs share the tiles that there are, not the grid's bound)
        int64_t sum = 0;
        for (int w = 0; w < NW; ++w) sum += sch[w];
        const int t = tile_of((int)min(sum, (int64_t)tiles_m) * tiles_n);
        if (t < 0) return;  // past the last row block: the whole workgroup leaves
        tn = t % tiles_n;
        int64_t at = t / tiles_n - (incl - mine);
        for (int w = 0; w < wave_all; ++w) at -= sch[w];
        if (at >= 0 && at < mine)
            for (int g = g_lo; g < g_hi; ++g) {
                int r0, r1;
                rows_of(g, r0, r1);
                const int n = (r1 - r0 + BM - 1) / BM;
                if (at < n) {
                    sch[NW] = g;
                    sch[NW + 1] = r0 + (int)at * BM;
                    sch[NW + 2] = r1;
                    break;
                }
                at -= n;
            }
        __syncthreads();
        const int g = __builtin_amdgcn_readfirstlane(sch[NW]);
        m0 = __builtin_amdgcn_readfirstlane(sch[NW + 1]);
        row_end = __builtin_amdgcn_readfirstlane(sch[NW + 2]);
        b_first = (int64_t)g * a.RBb + (int64_t)tn * BF;
        __syncthreads();  // everyone has read before the ring fills
    } else {
        constexpr int GROUP_M = 8;
        const int t = tile_of(tiles_m * tiles_n);
        const int in_group = GROUP_M * tiles_n;
        const int first_m = (t / in_group) * GROUP_M;
        const int gsize = min(tiles_m - first_m, GROUP_M);
        tn = (t % in_group) / gsize;
        m0 = (first_m + (t % in_group) % gsize) * BM;
        b_first = (int64_t)tn * BF;
    }
    const int n0 = tn * BN;

    // The tile's part of each operand: row blocks from its first one to the
    // operand's end or the tile's; A of a grouped product is addressed whole,
    // row by row.
    const int rba = GROUPED ? a.RBa : min(AF, a.RBa - m0 / 16), rbb = min(BF, a.RBb - tn * BF);
    const int64_t a_first = GROUPED ? 0 : m0 / 16;
    const __amdgpu_buffer_rsrc_t rac = make_rsrc(a.a_codes + a_first * C * kMxFrag, (uint32_t)rba * C * kMxFrag);
    const __amdgpu_buffer_rsrc_t rbc = make_rsrc(a.b_codes + b_first * C * kMxFrag, (uint32_t)rbb * C * kMxFrag);
    const __amdgpu_buffer_rsrc_t ras = make_rsrc(a.a_scales + a_first * Q * kMxScaleFrag, (uint32_t)rba * Q * kMxScaleFrag);
    const __amdgpu_buffer_rsrc_t rbs = make_rsrc(a.b_scales + b_first * Q * kMxScaleFrag, (uint32_t)rbb * Q * kMxScaleFrag);
    const uint32_t lds0 = lds_addr(lds);
    // Row of A that a lane brings for fragment f of the tile (grouped): a
    // fragment's lanes fill it in order, four to a row.
    auto a_row = [&](int f) {
        const int r = min(m0 + f * 16 + (lane >> 2), row_end - 1);
        return (uint32_t)(a.a_rows ? min(max(a.a_rows[r], 0), a.A_rows - 1) : r);
    };

    // A wave's loads: number i is fragment wave * CPW + i of a step's codes, or
    // of a scale word.  Where they come from in the operands' memory, per lane:
    uint32_t code_at[CPW], scale_at[SPW];
#pragma unroll
    for (int i = 0; i < CPW; ++i) {
        const int f = wave * CPW + i;
        const uint32_t k = (uint32_t)(f < AF ? f : f - AF);
        code_at[i] = k * (uint32_t)C * kMxFrag + lane * 16;
        scale_at[i] = k * (uint32_t)Q * kMxScaleFrag + lane * 4;
        if (GROUPED && f < AF) {
            const uint32_t r = a_row(f);
            code_at[i] = (r >> 4) * (uint32_t)C * kMxFrag + mx_code_at(r & 15, (lane & 3) ^ (lane >> 4));
            scale_at[i] = (r >> 4) * (uint32_t)Q * kMxScaleFrag + mx_scale_at(r & 15, lane & 3);
        }
    }
    // The team's steps, c0 .. c0 + steps - 1: whole scale words, shared evenly.
    const int q0 = KS > 1 ? (int)((int64_t)Q * team / KS) : 0;
    const int c0 = 4 * q0;
    const int steps = KS > 1 ? min(4 * (int)((int64_t)Q * (team + 1) / KS), C) - c0 : C;
    // Load number I of the team's step c into buffer `stage`, and of its scale
    // word q.
    auto load_code = [&](auto I, int c, int stage) {
        constexpr int i = I.value;
        mx_dma<16, i * kMxFrag>(wave * CPW + i < AF ? rac : rbc, code_at[i], (uint32_t)min(c0 + c, C - 1) * kMxFrag,
                                lds0 + (uint32_t)(stage * STAGE + wave * CPW * kMxFrag));
    };
    auto load_scale = [&](auto I, int q) {
        constexpr int i = I.value;
        mx_dma<4, NS * STAGE + i * kMxScaleFrag>(wave * CPW + i < AF ? ras : rbs, scale_at[i],
                                                 (uint32_t)min(q0 + q, Q - 1) * kMxScaleFrag,
                                                 lds0 + (uint32_t)(wave * CPW * kMxScaleFrag));
    };

    mx_f16 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

    // A lane's place in a 32-row block of a fragment pair: row l % 32, and
    // block 2 * half + l / 32 of the step.
    const int q32 = lane & 31, kgl = lane >> 5;
    const int fa = wm * (AF / WM), fb = AF + wn * (BF / WN);  // the wave's first fragments
    const uint8_t* lane_code[2];  // of each half
#pragma unroll
    for (int h = 0; h < 2; ++h) lane_code[h] = lds + (q32 >> 4) * kMxFrag + mx_code_at(q32 & 15, 2 * h + kgl);
    const uint8_t* lane_sa = lds + NS * STAGE + ((q32 >> 4) + fa) * kMxScaleFrag + mx_scale_at(q32 & 15, kgl);
    const uint8_t* lane_sb = lane_sa + (fb - fa) * kMxScaleFrag;

    struct Half { mx_u4 a[MI], b[NI]; };
    struct Scales { uint32_t a[MI][2], b[NI][2]; };
    constexpr int P = MI + NI;   // 32-row blocks of a wave: LDS reads of a half
    constexpr int MM = MI * NI;  // MFMAs of a half
    // the MFMA of a half behind which LDS read i is issued
    constexpr auto slot_of = [](int i) { return P <= MM ? i : i * MM / P; };
    // LDS read number I of a half
    auto read = [&](auto I, Half& h, int stage, int half) {
        constexpr int i = I.value;
        const uint8_t* p = lane_code[half] + stage * STAGE;
        if constexpr (i < MI)
            h.a[i] = *reinterpret_cast<const mx_u4*>(p + (fa + 2 * i) * kMxFrag);
        else
            h.b[i - MI] = *reinterpret_cast<const mx_u4*>(p + (fb + 2 * (i - MI)) * kMxFrag);
    };
    // the two scale words of 32-row block I
    auto read_scale = [&](auto I, Scales& s) {
        constexpr int i = I.value;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if constexpr (i < MI)
                s.a[i][h] = *reinterpret_cast<const uint32_t*>(lane_sa + 2 * i * kMxScaleFrag + h * 8);
            else
                s.b[i - MI][h] = *reinterpret_cast<const uint32_t*>(lane_sb + 2 * (i - MI) * kMxScaleFrag + h * 8);
    };
    Scales sc, sn;
    auto mfma = [&](auto N, auto S, const Half& h, int half) {
        constexpr int i = N.value / NI, j = N.value % NI;
        acc[i][j] = mx_mfma32<S.value>(h.b[j], sc.b[j][half], h.a[i], sc.a[i][half], acc[i][j]);
    };

    // fill the ring
    mx_each<SPW>([&](auto I) { load_scale(I, 0); });
    mx_each<NS>([&](auto c) { mx_each<CPW>([&](auto I) { load_code(I, c.value, c.value); }); });
    wait_vmcnt<(NS - 1) * CPW>();  // step 0 and the first scale word
    wg_barrier();
    Half h0, h1;
    mx_each<P>([&](auto I) { read_scale(I, sc); });
    mx_each<P>([&](auto I) { read(I, h0, 0, 0); });

    // One step.  The order is fixed (the scheduling barriers): behind each
    // MFMA one LDS read and its share of the loads, which issue while the
    // MFMA runs; left to itself the compiler moves the reads to their uses
    // and the MFMAs wait for each.
    int c = 0, stage = 0;
    auto step = [&](auto S) {
        constexpr int s = S.value;
        mx_each<MM>([&](auto N) {
            mfma(N, S, h0, 0);
            mx_each<P>([&](auto I) { if constexpr (slot_of(I.value) == N.value) read(I, h1, stage, 1); });
            __builtin_amdgcn_sched_barrier(0);
        });
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        // step c + 1 has landed: what may be in flight was issued in the last
        // NS - 2 steps (the scales in a word's first one)
        wait_vmcnt<(NS - 2) * CPW + (s > 0 && s <= NS - 2 ? SPW : 0)>();
        wg_barrier();
        __builtin_amdgcn_sched_barrier(0);
        const int freed = stage;
        stage = stage + 1 == NS ? 0 : stage + 1;
        mx_each<MM>([&](auto N) {
            constexpr int n = N.value;
            mfma(N, S, h1, 1);
            mx_each<P>([&](auto I) {
                if constexpr (slot_of(I.value) == n) read(I, h0, stage, 0);
                if constexpr (s == 3 && MM - 1 - slot_of(I.value) == n) read_scale(I, sn);
            });
            mx_each<(n + 1) * CPW / MM - n * CPW / MM>([&](auto I) {
                constexpr int i = n * CPW / MM + I.value;
                load_code(std::integral_constant<int, i>{}, c + NS, freed);
                if constexpr (s == 0) load_scale(std::integral_constant<int, i>{}, c / 4 + 1);
            });
            __builtin_amdgcn_sched_barrier(0);
        });
        if constexpr (s == 3) sc = sn;
        ++c;
    };
    // whole scale words, then the steps that are left (one loop exit: the
    // accumulators stay where they are)
    for (int q = steps / 4; q > 0; --q) mx_each<4>(step);
    if (steps & 3) {
        step(std::integral_constant<int, 0>{});
        if ((steps & 3) > 1) step(std::integral_constant<int, 1>{});
        if ((steps & 3) > 2) step(std::integral_constant<int, 2>{});
    }
    // a team with fewer steps than another meets it at the barriers that are left
    if constexpr (KS > 1)
        for (int k = 4 * ((Q + KS - 1) / KS) - steps; k > 0; --k) wg_barrier();
    wait_vmcnt<0>();  // the ring's last loads, before its memory is used again
    __syncthreads();

    // The teams' sums, added in their order: each but the first leaves its own
    // in LDS.
    if constexpr (KS > 1) {
        mx_f4* part = reinterpret_cast<mx_f4*>(lds_all) + wave * (MM * 256) + lane;
        if (team > 0)
            mx_each<MM * 4>([&](auto K) {
                constexpr int k = K.value, m = k / 4, v = k % 4 * 4;
                const mx_f16& x = acc[m / NI][m % NI];
                part[(team - 1) * (4 * MM * 256) + k * 64] = mx_f4{x[v], x[v + 1], x[v + 2], x[v + 3]};
            });
        __syncthreads();
        if (team == 0)
            mx_each<MM * 4>([&](auto K) {
                constexpr int k = K.value, m = k / 4, v = k % 4 * 4;
                mx_f16& x = acc[m / NI][m % NI];
                for (int t = 0; t < KS - 1; ++t) {
                    const mx_f4 y = part[t * (4 * MM * 256) + k * 64];
                    x[v] += y[0]; x[v + 1] += y[1]; x[v + 2] += y[2]; x[v + 3] += y[3];
                }
            });
        __syncthreads();
    }

    // Epilogue.  Block (i, j) of lane l: row 32 i + l % 32, columns 32 j +
    // 8 (v / 4) + 4 (l / 32) + v % 4.
    constexpr int PM = BM / WM, PN = BN / WN;  // the wave's part
    const int row0 = m0 + wm * PM, col0 = n0 + wn * PN;
    if (a.out_bf16 && (a.N & 7) == 0) {
        // through LDS, a wave's part each, so that whole lines are stored
        constexpr int ROW = PN * 2 + 16;  // bytes, 16 of them padding
        uint8_t* part = lds_all + wave * PM * ROW;
        if (KS == 1 || team == 0) {
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NI; ++j)
#pragma unroll
                    for (int v = 0; v < 16; v += 4) {
                        uint32_t o[2];
                        o[0] = mx_to_bf16(a.alpha * acc[i][j][v]) | (uint32_t)mx_to_bf16(a.alpha * acc[i][j][v + 1]) << 16;
                        o[1] = mx_to_bf16(a.alpha * acc[i][j][v + 2]) | (uint32_t)mx_to_bf16(a.alpha * acc[i][j][v + 3]) << 16;
                        __builtin_memcpy(__builtin_assume_aligned(part + (i * 32 + q32) * ROW + (j * 32 + 2 * v + 4 * kgl) * 2, 8), o, 8);
                    }
        }
        __syncthreads();
        if (KS > 1 && team > 0) return;
        constexpr int LPR = PN / 8;        // lanes that store a row's part
        constexpr int RPS = 64 / LPR;      // rows a store covers
        const int r = lane / LPR, col = col0 + (lane % LPR) * 8;
#pragma unroll 4
        for (int k = 0; k < PM; k += RPS) {
            const int row = row0 + k + r;
            mx_u4 o;
            __builtin_memcpy(&o, __builtin_assume_aligned(part + (k + r) * ROW + (lane % LPR) * 16, 16), 16);
            if (row < row_end && col < a.N)
                *reinterpret_cast<mx_u4*>(static_cast<uint16_t*>(a.out) + (int64_t)row * a.N + col) = o;
        }
    } else if (KS == 1 || team == 0) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const int row = row0 + i * 32 + q32;
#pragma unroll
            for (int j = 0; j < NI; ++j)
#pragma unroll
                for (int v = 0; v < 16; v += 4) {
                    const mx_f4 f = {acc[i][j][v], acc[i][j][v + 1], acc[i][j][v + 2], acc[i][j][v + 3]};
                    if (row < row_end) mx_store4(a, row, col0 + j * 32 + 2 * v + 4 * kgl, f);
                }
        }
    }
}

// Steps up to which the tile kernel's 32-bit offsets hold (16 row blocks of
// them stay below 2 GiB).
constexpr int kMxTileSteps = (int)((1u << 31) / (16 * kMxFrag)) - 1;

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

template <int BM, int BN, int NS, int WM, int KS, bool GROUPED>
void run_tile(Launch& l) {
    const MxGemmArgs& a = l.a;
    // (grouped: each group adds at most one broken row block)
    const int64_t tiles_m = ((int64_t)a.M + BM - 1) / BM + (GROUPED ? a.groups : 0), tiles_n = ((int64_t)a.N + BN - 1) / BN;
    l.items = tiles_m * tiles_n * KS * 256;
    if (l.dry) return;
    hipLaunchKernelGGL((mx_tile_kernel<BM, BN, NS, WM, KS, GROUPED>), dim3((unsigned)(tiles_m * tiles_n)), dim3(KS * 256), 0,
                       l.stream, a, (int)tiles_m, (int)tiles_n);
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
        const char* e = getenv("MXV"); const int v = e ? atoi(e) : 0;
        if (v == 10) return run_split<2, 4, 4, A_PACKED, true>(l);
        if (v == 11) return run_split<4, 4, 8, A_PACKED, true>(l);
        if (v == 12) return run_split<1, 4, 8, A_PACKED, true>(l);
        if (v == 13) return run_split<2, 2, 8, A_PACKED, true>(l);
        if (v == 14) return run_split<2, 4, 8, A_PACKED, true>(l);
        if (v == 1) return run_tile<128, 256, 3, 2, 1, true>(l);
        if (v == 2) return run_tile<64, 256, 3, 1, 1, true>(l);
        if (v == 20) return run_tile<64, 64, 4, 2, 4, true>(l);
        if (v == 21) return run_tile<64, 64, 4, 2, 2, true>(l);
        if (v == 22) return run_tile<64, 128, 4, 2, 2, true>(l);
        if (v == 3) return run_tile<256, 256, 4, 2, 1, true>(l);
        if (v == 8) return run_tile<128, 128, 3, 2, 1, true>(l);
        return run_tile<128, 128, 4, 2, 1, true>(l);
    }
    if (!a.a_codes) return a.x_bf16 ? run_few_rows<A_BF16>(l) : run_few_rows<A_F32>(l);
    if (a.M <= 64) return run_few_rows<A_PACKED>(l);
    const char* e = getenv("MXV"); const int v = e ? atoi(e) : 0;
    if (v == 1) return run_tile<128, 256, 3, 2, 1, false>(l);
    if (v == 2) return run_tile<64, 256, 3, 1, 1, false>(l);
    if (v == 3) return run_tile<256, 256, 4, 2, 1, false>(l);
    if (v == 4) return run_tile<128, 128, 4, 2, 1, false>(l);
    if (v == 5) return run_tile<128, 128, 4, 2, 2, false>(l);
    if (v == 20) return run_tile<64, 64, 4, 2, 4, false>(l);
    if (v == 21) return run_tile<64, 64, 4, 2, 2, false>(l);
    if (v == 22) return run_tile<64, 128, 4, 2, 2, false>(l);
    if (v == 24) return run_tile<64, 128, 3, 2, 4, false>(l);
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
