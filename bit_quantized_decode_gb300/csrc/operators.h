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
constexpr int kG8Threads = 640;

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
cudaError_t launch_gemm_w8(Gemm8Args& a, int grid, size_t smem, bool pdl, cudaStream_t s);

}  // namespace w4k
