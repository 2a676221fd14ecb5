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

#include <algorithm>
#include <type_traits>
#include <utility>

namespace nvfp4 {
namespace {

// dma16 / dma4 (nvfp4_device.h) with the LDS address as a uniform base plus a
// constant: one scalar instruction a load.  NT: with the non-temporal hint.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int BYTES, int AT, bool NT = false>
__device__ __forceinline__ void mx_dma(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff,
                                       uint32_t lds) {
    if constexpr (BYTES == 16 && NT)
        asm volatile("s_add_u32 m0, %3, %4\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds"
                     :: "v"(voff), "s"(r), "s"(soff), "s"(lds), "n"(AT) : "memory", "m0", "scc");
    else if constexpr (BYTES == 16)
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

// Stores of rows of C that may start anywhere (N need not be a multiple of
// anything): a piece is one access, aligned to its elements only.
typedef unsigned int mx_u2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef unsigned int mx_u4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float mx_f4_any __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ uint32_t mx_bf16_pair(float x, float y) {
    return mx_to_bf16(x) | (uint32_t)mx_to_bf16(y) << 16;
}

// Four consecutive columns of C, scaled and rounded.
__device__ __forceinline__ void mx_store4(const MxGemmArgs& a, int row, int col, mx_f4 f) {
    const int64_t at = (int64_t)row * a.N + col;
    f *= a.alpha;
    if (col + 4 <= a.N) {
        if (a.out_bf16)
            *reinterpret_cast<mx_u2_any*>(static_cast<uint16_t*>(a.out) + at) =
                mx_u2_any{mx_bf16_pair(f[0], f[1]), mx_bf16_pair(f[2], f[3])};
        else
            *reinterpret_cast<mx_f4_any*>(static_cast<float*>(a.out) + at) = f;
        return;
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        if (col + v >= a.N) break;
        if (a.out_bf16)
            static_cast<uint16_t*>(a.out)[at + v] = mx_to_bf16(f[v]);
        else
            static_cast<float*>(a.out)[at + v] = f[v];
    }
}

// ---------------------------------------------------------------------------
// Skinny kernel, for few rows of A: a workgroup takes 16 columns of C (one row
// block of B) and its 16 waves split K a scale word (four steps) at a time.
// Each wave copies its 4 KB of B straight to a part of LDS of its own and
// reads its operands from there (in the packed layout a wave's rows are 64
// bytes apart: loaded straight to registers they cost the address unit twice
// the time, 3.7 against 3.2 us at 1 x 768 x 6144); the waves' sums are added
// in LDS in wave order, so results do not depend on timing.
//
// First operand of v_mfma_scale_f32_16x16x128_f8f6f4: B's rows; second: A's
// rows; so lane l ends up with row l % 16 of A and four consecutive columns.
//
// A_F32, A_BF16: the wave quantises its piece of the activations itself, four
// rows of sixteen blocks at a time, a block to a lane, and hands the codes
// to the lanes that multiply them through LDS.  (With a lane quantising the
// four blocks that it multiplies, one row cost as much as sixteen: 5.0 us
// at 1 x 768 x 6144, where packed operands take 3.4.)  A workgroup then walks
// the row blocks of B that its turn comes to: with one scale word to a wave (K
// up to 8192) the rows are quantised once and the next row block is loaded
// while the sums of this one are added.
//
// GROUPED (operands past the tile kernel's 32-bit offsets): group g owns rows
// offsets[g] .. offsets[g+1]-1 of C; a workgroup takes one row block of one
// group's B and walks the group's rows.  Offsets are clamped to [0, M] and row
// numbers to A's rows, so a malformed table gives wrong rows but no access
// outside the buffers.
//
// NT: B loaded non-temporally.
// ---------------------------------------------------------------------------
enum { A_PACKED = 0, A_F32 = 1, A_BF16 = 2 };

// Orders a wave's LDS accesses among its lanes.
__device__ __forceinline__ void mx_wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int MI, int AT, bool GROUPED, bool NT>
__global__ void __launch_bounds__(1024) mx_skinny_kernel(MxGemmArgs a) {
    constexpr int W = 16;
    static_assert(AT == A_PACKED || MI == 1, "quantised rows: one row block");
    __shared__ __attribute__((aligned(1024))) uint8_t b_lds[W][4 * kMxFrag];
    __shared__ __attribute__((aligned(1024))) uint8_t a_lds[AT == A_PACKED ? 1 : W][4 * kMxFrag + kMxScaleFrag];
    __shared__ mx_f4 red[W][MI][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, kg = lane >> 4;
    const int C = a.C, Q = (C + 3) / 4;
    const int cb0 = (int)(blockIdx.x % (unsigned)a.RBb);  // (first) row block of B
    const int tm = (int)(blockIdx.x / (unsigned)a.RBb);   // row tile, or group
    const int turn = AT == A_PACKED ? a.RBb : (int)gridDim.x;
    const bool once = AT != A_PACKED && Q <= W;
    int r0 = tm * 16 * MI, r1 = min(r0 + 16 * MI, a.M);
    int64_t b_first = 0;
    if constexpr (GROUPED) {
        r0 = min(max(a.offsets[tm], 0), a.M);
        r1 = min(max(a.offsets[tm + 1], r0), a.M);
        b_first = (int64_t)tm * a.RBb;
    }
    const int at_code = mx_code_at(r16, kg), at_scale = mx_scale_at(r16, kg);
    const uint32_t b_base = lds_addr(b_lds[wave]);
    // Loads scale word q of row block cb of B: the codes to LDS, the lane's
    // scales returned.
    auto load_b = [&](int cb, int q) {
        const int n = min(4, C - 4 * q);  // steps of this word
        const uint8_t* bc = a.b_codes + (b_first + cb) * C * kMxFrag;
        const __amdgpu_buffer_rsrc_t rb = make_rsrc(bc + (int64_t)q * 4 * kMxFrag, (uint32_t)n * kMxFrag);
        mx_each<4>([&](auto S) {
            if (S.value < n) mx_dma<16, S.value * kMxFrag, NT>(rb, lane * 16, S.value * kMxFrag, b_base);
        });
        const uint8_t* bs = a.b_scales + (b_first + cb) * Q * kMxScaleFrag;
        return *reinterpret_cast<const uint32_t*>(bs + (int64_t)q * kMxScaleFrag + at_scale);
    };
    bool first = true, loaded = false;
    uint32_t sb = 0;

    for (int cb = cb0; cb < a.RBb; cb += turn)
    for (int m0 = r0; m0 < r1; m0 += 16 * MI) {
        const uint8_t *ac[MI], *as[MI];  // this lane's block of its row, at step 0
        bool live[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            int r = m0 + i * 16 + r16;
            live[i] = r < r1;
            if (GROUPED && a.a_rows && live[i]) r = min(max(a.a_rows[r], 0), a.A_rows - 1);
            ac[i] = a.a_codes + (int64_t)(r >> 4) * C * kMxFrag + mx_code_at(r & 15, kg);
            as[i] = a.a_scales + (int64_t)(r >> 4) * Q * kMxScaleFrag + mx_scale_at(r & 15, kg);
        }
        mx_f4 acc[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[i] = mx_f4{0.0f, 0.0f, 0.0f, 0.0f};

        for (int q = wave; q < Q; q += W) {
            const int n = min(4, C - 4 * q);  // steps of this word
            if (!loaded) sb = load_b(cb, q);
            loaded = false;
            mx_u4 wa[4][MI];
            uint32_t sa[MI];
            if constexpr (AT == A_PACKED) {
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    sa[i] = 0;
#pragma unroll
                    for (int s = 0; s < 4; ++s) wa[s][i] = mx_u4{0, 0, 0, 0};
                    if (live[i]) {
                        sa[i] = *reinterpret_cast<const uint32_t*>(as[i] + (int64_t)q * kMxScaleFrag);
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            wa[s][i] = *reinterpret_cast<const mx_u4*>(ac[i] + (int64_t)min(4 * q + s, C - 1) * kMxFrag);
                    }
                }
            } else {
                using T = std::conditional_t<AT == A_F32, float, uint16_t>;
                const int s = (lane & 15) >> 2, b = lane & 3;  // the lane's block
                const int k = (4 * q + s) * kMxStep + b * kMxBlock;
                for (int p = 0; p < r1 - m0 && !(once && cb != cb0); p += 4) {
                    const int row = p + (lane >> 4);
                    if (m0 + row < r1) {
                        mx_u4 w = {0, 0, 0, 0};
                        uint32_t byte = 0;
                        if (k < a.K) byte = mx_quant_load(static_cast<const T*>(a.x) + (int64_t)(m0 + row) * a.ldx + k, w);
                        uint8_t* d = a_lds[wave];
                        *reinterpret_cast<mx_u4*>(d + s * kMxFrag + mx_code_at(row, b)) = w;
                        d[4 * kMxFrag + mx_scale_at(row, b) + s] = (uint8_t)byte;
                    }
                }
                mx_wave_fence();
                // (rows past the last one: whatever LDS holds, not stored)
                sa[0] = *reinterpret_cast<const uint32_t*>(a_lds[wave] + 4 * kMxFrag + at_scale);
#pragma unroll
                for (int t = 0; t < 4; ++t) wa[t][0] = *reinterpret_cast<const mx_u4*>(a_lds[wave] + t * kMxFrag + at_code);
            }
            wait_vmcnt<0>();
            asm volatile("" ::: "memory");  // B has landed
            mx_each<4>([&](auto S) {
                if (S.value < n) {
                    const mx_u4 wb = *reinterpret_cast<const mx_u4*>(b_lds[wave] + S.value * kMxFrag + at_code);
#pragma unroll
                    for (int i = 0; i < MI; ++i) acc[i] = mx_mfma16<S.value>(wb, sb, wa[S.value][i], sa[i], acc[i]);
                }
            });
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // LDS is read before it is filled again
            mx_wave_fence();
            if (once && cb + turn < a.RBb) {
                sb = load_b(cb + turn, q);
                loaded = true;
            }
        }

        if (!first) __syncthreads();  // the previous sums are read
        first = false;
#pragma unroll
        for (int i = 0; i < MI; ++i) red[wave][i][lane] = acc[i];
        __syncthreads();
        for (int f = wave; f < MI; f += W) {
            mx_f4 sum = red[0][f][lane];
#pragma unroll
            for (int w = 1; w < W; ++w) sum += red[w][f][lane];
            const int row = m0 + f * 16 + r16;
            if (row < r1) mx_store4(a, row, cb * 16 + 4 * kg, sum);
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
    constexpr int APW = AF / 4, BPW = BF / 4;             // of them, a wave's loads: first A's, then B's
    constexpr int CPW = APW + BPW;
    constexpr int SPW = CPW;                              // a wave's scale loads, every fourth step
    constexpr int STAGE = (AF + BF) * kMxFrag;
    constexpr int SCALES = (AF + BF) * kMxScaleFrag;      // of four steps
    // Step c's place in the ring is filled again, for step c + NS, from the
    // middle of step c on; a scale word is in registers before its first step,
    // from whose middle on the next word's loads fill the buffer.  They have
    // landed by the middle of the word's last step, where it is read: no more
    // than two steps' loads are in flight there.
    static_assert(NS == 3 || NS == 4, "scales are read three steps behind their loads");
    // scale loads among those issued at the `many` steps before step k
    constexpr auto scale_loads = [](int k, int many) {
        int n = 0;
        for (int d = 1; d <= many; ++d) n += ((k - d) & 3) == 0 ? SPW : 0;
        return n;
    };
    static_assert(AF % 4 == 0 && BF % 4 == 0 && (NS + 1) * CPW + SPW < 64, "ring");
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
    bool stream = false;
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
        // (M < 2^28 and groups < 2^30: at most 2^22 full ones and 2^22 broken
        // ones in a sound table; the sum over a wave stays below 2^31)
        const int mine = (int)min(cnt, (int64_t)1 << 24);
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
                    sch[NW + 3] = n;
                    break;
                }
                at -= n;
            }
        __syncthreads();
        const int g = __builtin_amdgcn_readfirstlane(sch[NW]);
        m0 = __builtin_amdgcn_readfirstlane(sch[NW + 1]);
        row_end = __builtin_amdgcn_readfirstlane(sch[NW + 2]);
        b_first = (int64_t)g * a.RBb + (int64_t)tn * BF;
        stream = __builtin_amdgcn_readfirstlane(sch[NW + 3]) == 1 &&
                 (int64_t)a.groups * a.RBb * (C * kMxFrag + Q * kMxScaleFrag) > kStreamBytes;
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

    // A wave's loads: number i < APW is fragment wave * APW + i of A's part of a
    // step's codes, or of a scale word, and the others are BPW of B's.  Where
    // they come from in the operands' memory, per lane:
    uint32_t code_at[CPW], scale_at[SPW];
#pragma unroll
    for (int i = 0; i < CPW; ++i) {
        const uint32_t k = (uint32_t)(i < APW ? wave * APW + i : wave * BPW + i - APW);
        code_at[i] = k * (uint32_t)C * kMxFrag + lane * 16;
        scale_at[i] = k * (uint32_t)Q * kMxScaleFrag + lane * 4;
        if (GROUPED && i < APW) {
            const uint32_t r = a_row((int)k);
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
    auto load_code = [&](auto I, auto NT, int c, int stage) {
        constexpr int i = I.value;
        const uint32_t from = (uint32_t)min(c0 + c, C - 1) * kMxFrag;
        if constexpr (i < APW)
            mx_dma<16, i * kMxFrag>(rac, code_at[i], from, lds0 + (uint32_t)(stage * STAGE + wave * APW * kMxFrag));
        else
            mx_dma<16, (AF + i - APW) * kMxFrag, NT.value>(rbc, code_at[i], from,
                                                           lds0 + (uint32_t)(stage * STAGE + wave * BPW * kMxFrag));
    };
    auto load_scale = [&](auto I, int q) {
        constexpr int i = I.value;
        const uint32_t from = (uint32_t)min(q0 + q, Q - 1) * kMxScaleFrag;
        if constexpr (i < APW)
            mx_dma<4, NS * STAGE + i * kMxScaleFrag>(ras, scale_at[i], from, lds0 + (uint32_t)(wave * APW * kMxScaleFrag));
        else
            mx_dma<4, NS * STAGE + (AF + i - APW) * kMxScaleFrag>(rbs, scale_at[i], from,
                                                                  lds0 + (uint32_t)(wave * BPW * kMxScaleFrag));
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

    auto pipeline = [&](auto NT) {
        // fill the ring
        mx_each<NS>([&](auto c) {
            mx_each<CPW>([&](auto I) { load_code(I, NT, c.value, c.value); });
            if constexpr (c.value == 0) mx_each<SPW>([&](auto I) { load_scale(I, 0); });
        });
        wait_vmcnt<(NS - 1) * CPW>();  // the first scale word and step 0
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
            // NS - 2 steps
            wait_vmcnt<(NS - 2) * CPW + scale_loads(s, NS - 2)>();
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
                    load_code(std::integral_constant<int, i>{}, NT, c + NS, freed);
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
    };
    // A group of one row block reads its weights once: non-temporally, if
    // those of all groups are more than kStreamBytes (256 experts x 256
    // columns, 16 rows: 42.5 -> 38.6 us; groups of several row blocks share theirs
    // in the L2, which keeps such loads for less long: 128 rows 76 -> 80 us).
    if (GROUPED && stream)
        pipeline(std::bool_constant<GROUPED>{});
    else
        pipeline(std::false_type{});
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
    if (a.out_bf16) {
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
                        const uint32_t o[2] = {mx_bf16_pair(a.alpha * acc[i][j][v], a.alpha * acc[i][j][v + 1]),
                                               mx_bf16_pair(a.alpha * acc[i][j][v + 2], a.alpha * acc[i][j][v + 3])};
                        __builtin_memcpy(__builtin_assume_aligned(part + (i * 32 + q32) * ROW + (j * 32 + 2 * v + 4 * kgl) * 2, 8), o, 8);
                    }
        }
        __syncthreads();
        if (KS > 1 && team > 0) return;
        const bool stream_out = 2 * (int64_t)a.M * a.N > kStreamBytes;  // (28672 x 8192 x 2048: 309 -> 308 us)
        constexpr int LPR = PN / 8;        // lanes that store a row's part
        constexpr int RPS = 64 / LPR;      // rows a store covers
        const int r = lane / LPR, col = col0 + (lane % LPR) * 8;
#pragma unroll 4
        for (int k = 0; k < PM; k += RPS) {
            const int row = row0 + k + r;
            mx_u4 o;
            __builtin_memcpy(&o, __builtin_assume_aligned(part + (k + r) * ROW + (lane % LPR) * 16, 16), 16);
            if (row >= row_end || col >= a.N) continue;
            uint16_t* d = static_cast<uint16_t*>(a.out) + (int64_t)row * a.N + col;
            if (col + 8 > a.N) {
#pragma unroll
                for (int v = 0; v < 7; ++v)
                    if (col + v < a.N) d[v] = (uint16_t)(o[v >> 1] >> (v & 1) * 16);
            } else if (stream_out) {
                __builtin_nontemporal_store((mx_u4_any)o, reinterpret_cast<mx_u4_any*>(d));
            } else {
                *reinterpret_cast<mx_u4_any*>(d) = o;
            }
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

template <int MI, int AT, bool GROUPED, bool NT = false>
void run_skinny(Launch& l) {
    const MxGemmArgs& a = l.a;
    // (with activations to quantise a workgroup takes most of a CU's LDS, and the
    // GPU has 256)
    const int64_t tiles = AT == A_PACKED ? (GROUPED ? a.groups : (a.M + 16 * MI - 1) / (16 * MI)) * (int64_t)a.RBb
                                         : std::min(a.RBb, 256);
    l.items = tiles * 1024;
    if (l.dry) return;
    hipLaunchKernelGGL((mx_skinny_kernel<MI, AT, GROUPED, NT>), dim3((unsigned)tiles), dim3(1024), 0, l.stream, a);
    l.error = hipGetLastError();
}

template <int BM, int BN, int NS, int WM, int KS, bool GROUPED>
void run_tile(Launch& l) {
    const MxGemmArgs& a = l.a;
    // (grouped: each group that has rows adds at most one broken row block.
    // With one row block for every group instead, 8 rows for 256 experts x 2048
    // x 6144 took 24.2 us, now 13.1; and many groups were refused)
    const int64_t tiles_m = ((int64_t)a.M + BM - 1) / BM + (GROUPED ? std::min(a.groups, a.M) : 0), tiles_n = ((int64_t)a.N + BN - 1) / BN;
    l.items = tiles_m * tiles_n * KS * 256;
    if (l.dry) return;
    hipLaunchKernelGGL((mx_tile_kernel<BM, BN, NS, WM, KS, GROUPED>), dim3((unsigned)(tiles_m * tiles_n)), dim3(KS * 256), 0,
                       l.stream, a, (int)tiles_m, (int)tiles_n);
    l.error = hipGetLastError();
}

// The kernel by sizes.  Times are of K = 6144 unless they say otherwise, with
// operands beyond the L2; "short" ranges of K run on one team of waves, long
// ones on two.
constexpr int kMxShort = 24;  // steps

template <bool GROUPED>
void run_small_tiles(Launch& l) {
    // 512 x 512 x 512: 3.6 us on one team, 4.3 on two; 300 x 1000 x 1024: 4.1
    // and 4.5; 96 x 256 x 2048: 4.7 and 4.9; 256 x 4096 x 4096: 8.1 and 7.8; 512
    // x 2048 x 6144: 10.4 and 9.4; 1000 x 300 x 8192: 11.9 and 10.0.
    if (l.a.C <= kMxShort) return run_tile<64, 64, 4, 2, 1, GROUPED>(l);
    return run_tile<64, 64, 4, 2, 2, GROUPED>(l);
}

void choose(Launch& l) {
    const MxGemmArgs& a = l.a;
    const int64_t M = a.M, N = a.N, G = a.groups;
    // (a bound on the) tiles of rows x cols
    auto tiles = [&](int64_t rows, int64_t cols) {
        return ((M + rows - 1) / rows + std::min(G, M)) * ((N + cols - 1) / cols);
    };
    if (G > 0) {
        // the tile kernel addresses A with 32-bit offsets and numbers row blocks in 32 bits
        if (a.C > kMxTileSteps || M >= 1 << 28 || (int64_t)a.RBa * a.C * kMxFrag >= (int64_t)1 << 31)
            return run_skinny<2, A_PACKED, true>(l);
        // Few tiles, so that one tile's time counts (8 experts x 2048 columns,
        // 16 rows each: 13.4 us, 18.1 with 64 x 256 tiles); about even at 64
        // experts x 512 x K 2048 with 16 rows (640 tiles).
        if (tiles(64, 64) <= 640) return run_small_tiles<true>(l);
        // From 128 rows each (dropped ones among them), larger tiles read the
        // weights less often (256 experts x 256 columns, 128 rows: 73 us, 77 with
        // one token less and 64 x 256 tiles, in three runs; 16 x 2048 x K 2048,
        // 1024 rows: 56 against 64), if they are enough to fill the GPU or the
        // weights come from memory (8 x 2048, 256 rows: 27 against 33; but 4 x
        // 768, 1024 rows: 25 against 20).
        const int64_t weights = G * a.RBb * a.C * kMxFrag;
        if (M >= 128 * G && (tiles(128, 256) >= 256 || weights >= 32 << 20))
            return run_tile<128, 256, 3, 2, 1, true>(l);
        // 64 x 256 tiles stream the weights of small groups at the memory's
        // rate (256 experts x 256 columns, 16 rows: 39 us, 49 with 128 x 128);
        // narrow weights would leave them half empty.
        if (N <= 128) return run_tile<128, 128, 4, 2, 1, true>(l);
        return run_tile<64, 256, 3, 1, 1, true>(l);
    }
    const int64_t weights = a.RBb * ((int64_t)a.C * kMxFrag + (a.C + 3) / 4 * kMxScaleFrag);
    if (!a.a_codes) {  // (1 x 131072 x 8192: 98 -> 87 us with the weights non-temporal)
        if (weights > kStreamBytes) return a.x_bf16 ? run_skinny<1, A_BF16, false, true>(l) : run_skinny<1, A_F32, false, true>(l);
        return a.x_bf16 ? run_skinny<1, A_BF16, false>(l) : run_skinny<1, A_F32, false>(l);
    }
    // Up to 16 rows always the kernel that quantises too: the same bits (1 x
    // 768: 3.5 us, 7.3 with 64 x 64 tiles; 16 x 6144: 7.1 and 8.4).
    if (M <= kMxQuantRows) {
        // (weights of more than kStreamBytes: 1 x 131072 x 8192 89 -> 81 us, 16 rows
        // 117 -> 111)
        return weights > kStreamBytes ? run_skinny<1, A_PACKED, false, true>(l) : run_skinny<1, A_PACKED, false>(l);
    }
    // Up to 64 rows while its workgroups fit the GPU at once (64 x 768: 5.3
    // against 7.4 us; 64 x 6144: 14.0 against 8.8).
    if ((M <= 64 && (M + 31) / 32 * a.RBb <= 256) || a.C > kMxTileSteps) return run_skinny<2, A_PACKED, false>(l);
    // The smallest tiles that one round of the 256 CUs holds (256 x 4096 x 4096,
    // 256 tiles of 64 x 64: 7.9 us, 9.6 with 64 x 128; 400 x 4096 x 4096, 224 of
    // 64 x 128: 9.0, 10.3 with 64 x 64, 10.6 with 128 x 128).
    if (tiles(64, 64) <= 256) return run_small_tiles<false>(l);
    if (tiles(64, 128) <= 256) return run_tile<64, 128, 4, 2, 1, false>(l);
    // 256 x 256 for large sizes that are deep or many (4096 x 4096 x 8192: 63 us,
    // 64 with 128 x 256; 8192 x 8192 x 4096: 148 and 150; but 4096 x 8192 x 4096:
    // 71 and 67), unless they would be half empty (128 x 65536 x 8192: 71, 61 with
    // 128 x 128).
    const int64_t large = tiles(256, 256);
    if (M > 128 && large >= 256 && (a.C > 32 || large >= 1024)) return run_tile<256, 256, 4, 2, 1, false>(l);
    // 128 x 256, two to a CU, unless a few of them need a second round (256 x
    // 32768 x 8192, 256 tiles: 44 us, 49 with 128 x 128; 2048 x 6144 x 6144, 384: 44
    // and 46; 3000 x 3000 x 6144, 288: 39 and 37; 1237 x 2056 x 6112, 90: 21 and 15).
    const int64_t wide = tiles(128, 256);
    if (wide >= 360 || (wide >= 180 && wide <= 256)) return run_tile<128, 256, 3, 2, 1, false>(l);
    run_tile<128, 128, 4, 2, 1, false>(l);
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
