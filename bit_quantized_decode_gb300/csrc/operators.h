// Declarations of the operators beyond the single decode linear: the typed
// row quantizer, the INT8 x INT8 product for any number of tokens, the expert
// router and the few-token mixture-of-experts kernel.
#pragma once
#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace w4k {

// Element types of activations and outputs (W4_F32, W4_F16, W4_BF16).
enum ElemType { T_F32 = 0, T_F16 = 1, T_BF16 = 2 };
__host__ __device__ constexpr int elem_bytes(int t) { return t == T_F32 ? 4 : 2; }

// What a launch needs to know of the current device (w4a8_api.cu).
struct DeviceFacts {
    int sms;
    int smem_optin;
    unsigned* err;
};
bool device_facts(DeviceFacts* out);

// ---------------------------------------------------- row quantizer (quant_rows.cu)
struct QuantRowsArgs {
    const void* x;        // [M][K] of xtype
    const float* gamma;   // RMSNorm weight [K], or null
    float eps;
    int M, K;
    int8_t* qx;           // [M][K] codes, or null
    float* sx;            // [M]
    uint4* xh;            // the codes as fp16 in token tiles (f16_word), or null
    int nt;               // tokens per tile of xh
    int cluster;          // blocks per token (set by the launch)
};
// fp16 codes: 16-byte words of eight K values; a token tile's words of one K
// group follow each other, so (tile, K range) is one contiguous run.
__host__ __device__ inline size_t f16_word(int m, int k8, int K8, int nt)
{
    return (static_cast<size_t>(m / nt) * K8 + k8) * nt + m % nt;
}
cudaError_t launch_quant_rows(const QuantRowsArgs& a, int xtype, bool pdl, cudaStream_t s);
// int8 codes [M][K] -> the fp16 layout above.
cudaError_t launch_expand_codes(const int8_t* qx, int M, int K, uint4* xh, int nt, bool pdl, cudaStream_t s);

// ------------------------------------------- INT8 x INT8 product (gemm_w8.cu)
constexpr int kG8Rows = 128;                    // weight rows per tile (MMA M)
constexpr int kG8MaxTok = 128;                  // tokens per tile at most (MMA N)
constexpr int kG8StageChunks = 4;               // 32-weight chunks per stage: 128 K
constexpr int kG8WBytes = kG8Rows * 32 * kG8StageChunks;
constexpr int kG8AccStages = 8;                 // stages per accumulator: 1024 K keep the fp32 sums exact
constexpr int kG8TmemCols = 512;
constexpr int kG8ACols = 16 * kG8StageChunks;   // tensor-memory columns of one converted stage
constexpr int kG8MaxStages = 7;
constexpr int kG8MaxSplit = 8;
constexpr int kG8Threads = 576;

struct Gemm8Args {
    CUtensorMap wmap;         // the weights as [T row tiles][C chunks x 256 bytes]
    const uint8_t* w;         // w8_repack units
    const float* s_w;         // [N]
    const float* bias;        // [N] or null
    const uint4* xh;          // fp16 codes (QuantRowsArgs::xh)
    const float* sx;          // [M]
    const float* residual;    // [M][N] or null
    void* y;                  // [M][N] of ytype
    int ytype;
    int M, N, K, C, T;
    int nt;                   // tokens per tile (a multiple of 16)
    int n_tt, n_g;            // token tiles, row groups
    int splits;               // K splits per tile = cluster size (1: persistent blocks)
    int stages;               // ring slots in shared memory and converted stages in tensor memory
    unsigned* err;
};

struct Gemm8Smem {
    int ring, red, bars, tmem, total;
};
// Stages that tensor memory holds beside two accumulators of nt columns.
__host__ __device__ inline int gemm8_max_stages(int nt) { return (kG8TmemCols - 2 * nt) / kG8ACols; }
__host__ __device__ inline Gemm8Smem gemm8_smem(int stages, int nt, int splits)
{
    Gemm8Smem L;
    int o = 0;
    L.ring = o;  o += stages * (kG8WBytes + nt * 64 * kG8StageChunks);
    L.red = o;   o += splits > 1 ? kG8Rows * nt * 4 : 0;
    L.bars = o;  o += (3 * kG8MaxStages + 4) * 8;
    L.tmem = o;  o += 16;
    L.total = o;
    return L;
}
// The same product with pairs of blocks (cta_group::2) on tiles of 256 rows by
// up to 192 tokens (gemm_w8_pair.cu); nt is then the tokens of one block, half
// a tile.
constexpr int kP8MaxTok = 192;
constexpr int kP8Threads = 640;
constexpr int kP8ABufs = 4;                     // converted half stages (64 K) in tensor memory
constexpr int kP8ACols = 32;
constexpr int kP8MaxStages = 8;
struct Pair8Smem {
    int ring, bars, tmem, total;
};
__host__ __device__ inline Pair8Smem pair8_smem(int stages, int nt)
{
    Pair8Smem L;
    int o = 0;
    L.ring = o;  o += stages * (kG8WBytes + nt * 64 * kG8StageChunks);
    L.bars = o;  o += (2 * kP8MaxStages + 2 * kP8ABufs + 4) * 8;
    L.tmem = o;  o += 16;
    L.total = o;
    return L;
}
cudaError_t launch_gemm_w8_pair(Gemm8Args& a, int grid, size_t smem, bool pdl, cudaStream_t s);
cudaError_t encode_w8_map(Gemm8Args& a);
cudaError_t launch_gemm_w8(Gemm8Args& a, int grid, size_t smem, bool pdl, cudaStream_t s);

// ------------------------------- INT8 x INT8 product of up to eight tokens (gemv_w8.cu)
constexpr int kV8Warps = 12;
constexpr int kV8Threads = kV8Warps * 32;
constexpr int kV8MaxTok = 8;
constexpr int kV8FusedTok = 2;                  // tokens that the kernel quantizes itself, at most,
constexpr int kV8FusedValues = 16384;           // and activations (two tokens of 3584: 6.7 us, of 18944: 18.8 against 15.3 us)

struct Gemv8Args {
    const uint8_t* w;         // w8_repack units
    const float* s_w;         // [N]
    const float* bias;        // [N] or null
    const void* x;            // [M][K] of xtype (fused), else null
    int xtype;
    const float* gamma;       // RMSNorm weight (fused), or null
    float eps;
    const int8_t* qx_in;      // [M][K] codes (not fused)
    const float* sx_in;       // [M]
    int8_t* qx_out;           // fused: block 0 writes the codes here, or null
    float* sx_out;            // fused: and the scales
    const float* residual;    // [M][N] or null
    void* y;
    int ytype;
    int M, N, K;
    int share;                // warps per row tile (1, 2 or 4): each a share of K
    int slot;                 // bytes of a ring slot
    unsigned* err;
};
// Ring of two slots per warp, the codes, partial sums, scales, block sums, barriers.
__host__ __device__ inline int gemv8_smem(int slot, int M, int K)
{
    return kV8Warps * 2 * slot + M * K + kV8Warps * 8 * kV8MaxTok * 4 + 16 * kV8MaxTok + 4 * 4 * kV8Warps + (2 * kV8Warps + 1) * 8 + 64;
}
cudaError_t launch_gemv_w8(const Gemv8Args& a, int grid, size_t smem, bool pdl, cudaStream_t s);

// ------------------------------------------------ expert router (moe_route.cu)
constexpr int kRtThreads = 512;
constexpr int kRtWarps = kRtThreads / 32;
constexpr int kRtMaxTok = 4;                    // tokens per cluster at most
constexpr int kRtMaxCluster = 16;

// Words that the experts kernel finds prepared: a zero ticket counter, then
// a value that no result takes (the fp32 NaN with all bits set), by which a
// reader sees that a word has not been written yet.
constexpr int kMxHead = 32;                     // words: the ticket counter and padding
constexpr unsigned kMxNoValue = 0xffffffffu;
struct MoeFill {
    uint4* p;
    unsigned values;          // 16-byte words of values behind the head
};

struct RouteArgs {
    const void* x;            // [M][K] of xtype
    const float* gamma;       // RMSNorm weight, or null
    float eps;
    const float* w;           // [E][K]
    const float* sel;         // [E] selection bias (sigmoid), or null
    int E, top_k;
    int sigmoid;              // scores: 0 softmax, 1 sigmoid
    int renorm;
    float scale;
    int M, K;
    int tok;                  // tokens per cluster
    int cluster;
    int parts;                // warps per expert
    int* ids;                 // [M][top_k]
    float* weights;           // [M][top_k]
    int8_t* qx;               // [M][K] codes of the (normalized) tokens, or null
    float* sx;                // [M], or null
    MoeFill fill;             // the experts kernel's workspace, prepared here (words 0: none)
};
// x as fp32, the partial sums of an expert's warps, logits and selection keys (cluster leader), block sums.
__host__ __device__ inline int route_smem(int tok, int K, int E)
{
    return 4 * (tok * K + kRtWarps * kRtMaxTok * 2 + 2 * tok * ((E + 3) & ~3) + 2 * kRtWarps * kRtMaxTok);
}
cudaError_t launch_moe_route(const RouteArgs& a, int xtype, bool pdl, cudaStream_t s);

// ------------------------------------------ mixture-of-experts kernel (moe_experts.cu)
constexpr int kMxTok = 8;                       // pairs of one entry at most (an expert and some of its tokens)
constexpr int kMxMaxSlots = 20;                 // chosen and shared experts per token
constexpr int kMxMaxPairs = 16 * kMxMaxSlots;
constexpr int kMxMaxExperts = 1024;             // routed and shared
constexpr int kMxSeg = 1024;                    // hidden values per quantizing task
__host__ __device__ constexpr int mx_add(int tok) { return tok <= 2 ? 128 : 256; }   // outputs per adding task

struct MoeArgs {
    const uint8_t* w_gu;      // per expert: gate and up rows paired per tile (w4_repack_glu / w8_repack_glu)
    const uint8_t* w_dn;      // per expert: w4_repack / w8_repack
    const float* s_gu;        // [E + S][2 I]
    const float* b_gu;        // [E + S][2 I] or null
    const float* s_dn;        // [E + S][H]
    const float* b_dn;        // [E + S][H] or null
    const int8_t* qx;         // [M][H]
    const float* sx;          // [M]
    const int* ids;           // [M][top_k]
    const float* weights;     // [M][top_k]
    const float* residual;    // [M][H] or null
    void* y;                  // [M][H] of ytype
    int ytype, glu;
    int M, H, I, E, S, top_k;
    int stage_x;              // the tokens' codes are copied into shared memory
    int batch0, batch;        // tickets that a block takes at once: at its start, later
    float inv_x16;            // 16 / H
    float inv_t1, inv_t2, inv_seg, inv_add;   // 1 / (tickets of a gate/up and of a down matrix, quantizing tasks of a
                              // pair, adding tasks of a token)
    unsigned* ticket;         // zero at the start
    float* h;                 // [pairs][I], kMxNoValue at the start, and so
    float* part;              // [pairs][H]
    unsigned long long* qdone;   // [pairs][quantizing tasks]: scale and code sum of a finished piece
    int8_t* qh;               // [pairs][I] codes
    unsigned* err;
};
// Launch shape for `tok` pairs per entry (1, 2 or 8) on `most` bytes of shared memory.
struct MoePlan {
    int warps, tiles;         // per block; weight tiles to a ticket
    bool staged;              // the tokens' codes go into shared memory
    bool fits;
    size_t smem;
};
MoePlan moe_plan(int fmt, int tok, int M, int H, size_t most);
cudaError_t launch_moe_experts(int fmt, int tok, const MoeArgs& a, int grid, int warps, size_t smem, bool pdl, cudaStream_t s);
cudaError_t launch_moe_fill(const MoeFill& f, bool pdl, cudaStream_t s);

}  // namespace w4k
