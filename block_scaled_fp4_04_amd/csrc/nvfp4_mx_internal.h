// nvfp4_mx_internal.h -- launch arguments shared by the host library and the gfx950
// kernels of the MXFP4 operators (include/nvfp4_mx.h) and of the expert
// routing (include/nvfp4_moe.h); not part of the public ABI.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

// Packed MXFP4 geometry (include/nvfp4_mx.h, "Packed layout").
constexpr int kMxBlock = 32;     // elements that share a scale
constexpr int kMxStep = 128;     // elements of a row per step (one MFMA deep)
constexpr int kMxRows = 16;      // rows of a row block
constexpr int kMxFrag = 1024;    // code bytes of 16 rows x one step
constexpr int kMxScaleFrag = 256;  // scale bytes of 16 rows x four steps

// Where block b (0..3) of a step of row r (0..15) starts in a fragment, and its
// four scale bytes in a scale fragment.
__host__ __device__ constexpr int mx_code_at(int r, int b) { return r * 64 + ((b ^ (r >> 2)) << 4); }
__host__ __device__ constexpr int mx_scale_at(int r, int b) { return r * 16 + b * 4; }

// Results of more bytes than this are stored non-temporally, and inputs and
// weights of more are loaded so: what is written or read once then does not pass
// through the 256 MB last-level cache, which a call that uses it again would
// have found it in.  The border is a compromise of the two.  Used once (three
// buffers in turn) the hint is the faster one from about 96 MB on; used again by
// the next call it is from about 256 MB on.  us without and with it:
//                              128 MB       192 MB       256 MB       320 MB
//   quantise fp32, once      28.3  26.5   40.9  38.3   53.4  50.0   66.4  62.1
//   dequantise and quantise  47.1  49.9   69.9  72.8   98.9  95.2   152   119
//   gather and combine       53.2  59.0   76.3  87.1   124   116    168   147
//   weights of experts
//     three sets in turn     31.7  30.3   40.1  37.1   59.8  55.7   70.4  61.5
//     the same again         23.4  27.0   32.7  35.6   51.8  54.1   66.2  60.6
//   weights of one row
//     three sets in turn     25.9  24.3   38.4  35.0   50.5  46.0   62.2  55.9
//     the same again         22.0  21.1   31.0  32.3   40.4  43.3   57.1  53.3
constexpr int64_t kStreamBytes = (int64_t)192 << 20;

inline int64_t mx_round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline int64_t mx_steps(int64_t K) { return mx_round_up(K, kMxStep) / kMxStep; }
inline int64_t mx_row_blocks(int64_t rows) { return mx_round_up(rows, kMxRows) / kMxRows; }

// Quantisation (x -> codes, scales) or its inverse (codes, scales -> x).
struct MxQuantArgs {
    void* x;               // groups x rows x K values (fp32, or bfloat16 if bf16)
    bool bf16;
    uint8_t* codes;        // groups x [RB][C][16][4][16]
    uint8_t* scales;       // groups x [RB][Q][16][4][4]
    int64_t group_stride;  // elements between groups of x
    int64_t ld;            // elements between rows of x
    int64_t groups;
    int rows, K;
    int RB, C;             // row blocks of a group, steps
};
hipError_t launch_mx_quantize(const MxQuantArgs& a, hipStream_t stream);
hipError_t launch_mx_dequantize(const MxQuantArgs& a, hipStream_t stream);

// Product C = alpha * A . B^T, single (groups = 0) or grouped.
struct MxGemmArgs {
    const uint8_t* a_codes;    // packed A, or null
    const uint8_t* a_scales;
    const void* x;             // A as fp32 / bfloat16 rows (a_codes null), row stride ldx elements
    int64_t ldx;
    const uint8_t* b_codes;    // packed B (groups of them)
    const uint8_t* b_scales;
    const int32_t* offsets;    // [groups + 1] row offsets (device), or null
    const int32_t* a_rows;     // [M] row of A of each output row (device), or null: the row itself
    void* out;                 // M x N, fp32 or bfloat16
    float alpha;
    int M, N, K;               // output rows, output columns, depth
    int A_rows;                // logical rows of A
    int RBa, RBb;              // row blocks of A, of one B
    int C;                     // steps
    int groups;
    bool x_bf16, out_bf16;
};
// Rows of A up to which the one-launch product from activations runs.
constexpr int kMxQuantRows = 16;
hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t stream);
// Whether the grid of the kernel that the sizes choose stays within the
// runtime's limit on work-items.
bool mx_gemm_fits(const MxGemmArgs& a);

// Expert routing.
constexpr int kMoeMaxExperts = 2048;
struct MoeArgs {
    const void* ids;         // tokens x topk expert numbers (int32, or int64 if wide)
    bool wide;
    bool bf16;               // element type of the rows: bfloat16, else fp32
    int64_t tokens;
    int topk, experts;
    int64_t hidden, ld_in;   // row length, row stride of the input in token order
    int32_t* row_offsets;    // [experts + 1]
    int32_t* slots;          // [tokens][topk]
    int32_t* row_tokens;     // [tokens * topk]
    const void* x;           // gather: token rows; combine: expert-order rows
    const void* y;           // combine_grad: expert-order rows
    const float* weights;    // [tokens][topk], or null: ones
    void* out;               // gather, combine: result; combine_grad: dy
    float* dweights;         // combine_grad
};
hipError_t launch_moe_sort(const MoeArgs& a, hipStream_t stream);
hipError_t launch_moe_gather(const MoeArgs& a, hipStream_t stream);
hipError_t launch_moe_combine(const MoeArgs& a, hipStream_t stream);
hipError_t launch_moe_combine_grad(const MoeArgs& a, hipStream_t stream);

}  // namespace nvfp4
