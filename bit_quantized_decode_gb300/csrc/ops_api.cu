// C ABI of the INT8 x INT8 linear (declared in include/w4a8.h): argument
// checks, launch plan and dispatch.  No entry point allocates memory or
// synchronises.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/w4a8.h"
#include "operators.h"

using namespace w4k;

static_assert(W4_F32 == T_F32 && W4_F16 == T_F16 && W4_BF16 == T_BF16, "public element types");

namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline w4_status cuda_status(cudaError_t e) { return e == cudaSuccess ? W4_OK : W4_ERR_CUDA; }
inline bool elem_type(int t) { return t == W4_F32 || t == W4_F16 || t == W4_BF16; }

// Token tiles of a call: as few as hold M, evenly filled, in sixteens.
inline int token_tiles(int M) { return (M + kG8MaxTok - 1) / kG8MaxTok; }
inline int tile_tokens(int M)
{
    const int n = token_tiles(M);
    return n > 0 ? ((M + n - 1) / n + 15) / 16 * 16 : 16;
}

w4_status check_w8_shape(int M, int N, int K)
{
    if (M < 0 || N < 0 || K <= 0) return W4_ERR_INVALID_ARG;
    if (K % 32 != 0 || K > W4_MAX_K || M > W4_MAX_TOKENS || N > (1 << 30) - 8) return W4_ERR_UNSUPPORTED_SHAPE;
    const long long tiles = static_cast<long long>((N + kG8Rows - 1) / kG8Rows) * ((M + 15) / 16);
    return tiles > (1 << 30) ? W4_ERR_UNSUPPORTED_SHAPE : W4_OK;
}

// Tiles and K splits of an M x N x K product on a device of `sms` SMs.
bool plan_gemm8(const DeviceFacts& d, Gemm8Args& a, int& grid, size_t& smem)
{
    a.C = a.K / 32;
    a.T = (a.N + kRows - 1) / kRows;
    a.n_g = (a.N + kG8Rows - 1) / kG8Rows;
    a.n_tt = token_tiles(a.M);
    a.nt = tile_tokens(a.M);
    const int tiles = a.n_g * a.n_tt;
    const int nst = (a.C + kG8StageChunks - 1) / kG8StageChunks;
    a.splits = 1;
    while (a.splits < kG8MaxSplit && tiles * 2 * a.splits <= d.sms && nst >= 4 * a.splits) a.splits *= 2;
    a.stages = gemm8_max_stages(a.nt) < kG8MaxStages ? gemm8_max_stages(a.nt) : kG8MaxStages;
    while (a.stages > 2 && gemm8_smem(a.stages, a.nt, a.splits).total > d.smem_optin) --a.stages;
    smem = static_cast<size_t>(gemm8_smem(a.stages, a.nt, a.splits).total);
    grid = a.splits > 1 ? tiles * a.splits : (tiles < d.sms ? tiles : d.sms);
    return smem <= static_cast<size_t>(d.smem_optin);
}

w4_status run_gemm8(const void* w, const float* s_w, const float* bias, const uint4* xh, const float* sx,
                    const float* residual, int M, int N, int K, void* y, int y_type, cudaStream_t s)
{
    DeviceFacts d;
    if (!device_facts(&d)) return W4_ERR_CUDA;
    Gemm8Args a = {};
    a.w = static_cast<const uint8_t*>(w);
    a.s_w = s_w;
    a.bias = bias;
    a.xh = xh;
    a.sx = sx;
    a.residual = residual;
    a.y = y;
    a.ytype = y_type;
    a.M = M;
    a.N = N;
    a.K = K;
    a.err = d.err;
    int grid = 0;
    size_t smem = 0;
    if (!plan_gemm8(d, a, grid, smem)) return W4_ERR_UNSUPPORTED_SHAPE;
    return cuda_status(launch_gemm_w8(a, grid, smem, true, s));
}

w4_status check_w8_operands(const void* w, const float* s_w, const float* bias, const void* y, int y_type)
{
    if (!w || !s_w || !y) return W4_ERR_INVALID_ARG;
    if (!aligned(w, 16) || !aligned(s_w, 4) || (bias && !aligned(bias, 4)) ||
        !aligned(y, static_cast<size_t>(elem_bytes(y_type))))
        return W4_ERR_MISALIGNED;
    return W4_OK;
}

}  // namespace

extern "C" {

size_t w8a8_workspace_bytes(int M, int N, int K)
{
    if (check_w8_shape(M, N, K) != W4_OK) return 0;
    return static_cast<size_t>(token_tiles(M)) * tile_tokens(M) * K * 2;
}

w4_status w8a8_matmul(const void* w, const float* s_w, const float* bias, const int8_t* qx, const float* sx, int M,
                      int N, int K, void* y, int y_type, void* workspace, size_t ws_bytes, w4_stream_t st)
{
    w4_status r = check_w8_shape(M, N, K);
    if (r != W4_OK) return r;
    if (!elem_type(y_type)) return W4_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return W4_OK;
    r = check_w8_operands(w, s_w, bias, y, y_type);
    if (r == W4_ERR_INVALID_ARG || !qx || !sx || !workspace) return W4_ERR_INVALID_ARG;
    if (ws_bytes < w8a8_workspace_bytes(M, N, K)) return W4_ERR_UNSUPPORTED_SHAPE;
    if (r != W4_OK || !aligned(qx, 16) || !aligned(sx, 4) || !aligned(workspace, 16)) return W4_ERR_MISALIGNED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(st);
    uint4* xh = static_cast<uint4*>(workspace);
    r = cuda_status(launch_expand_codes(qx, M, K, xh, tile_tokens(M), false, s));
    if (r != W4_OK) return r;
    return run_gemm8(w, s_w, bias, xh, sx, nullptr, M, N, K, y, y_type, s);
}

w4_status w8a8_linear(const void* w, const float* s_w, const float* bias, const void* x, int x_type, int M, int N,
                      int K, void* y, int y_type, int8_t* qx, float* sx, const w4_fusion* f, unsigned flags,
                      void* workspace, size_t ws_bytes, w4_stream_t st)
{
    w4_status r = check_w8_shape(M, N, K);
    if (r != W4_OK) return r;
    if (!elem_type(x_type) || !elem_type(y_type) || (flags & ~W4_FLAG_PDL) != 0) return W4_ERR_INVALID_ARG;
    if (f != nullptr && f->glu != W4_GLU_NONE)
        return f->glu < W4_GLU_NONE || f->glu > W4_GLU_GELU_TANH ? W4_ERR_INVALID_ARG : W4_ERR_UNSUPPORTED_SHAPE;
    const float* gamma = f != nullptr ? f->norm_weight : nullptr;
    const float* residual = f != nullptr ? f->residual : nullptr;
    if (gamma != nullptr && (!(f->norm_eps > 0.0f) || !(f->norm_eps < 3.0e38f))) return W4_ERR_INVALID_ARG;
    if (M == 0) return W4_OK;
    r = N > 0 ? check_w8_operands(w, s_w, bias, y, y_type) : W4_OK;
    if (r == W4_ERR_INVALID_ARG || !x || !sx || !workspace) return W4_ERR_INVALID_ARG;
    if (ws_bytes < w8a8_workspace_bytes(M, N, K)) return W4_ERR_UNSUPPORTED_SHAPE;
    if (r != W4_OK || !aligned(x, 16) || (qx && !aligned(qx, 16)) || !aligned(sx, 4) || !aligned(workspace, 16) ||
        (gamma && !aligned(gamma, 16)) || (residual && !aligned(residual, 4)))
        return W4_ERR_MISALIGNED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(st);
    QuantRowsArgs q = {};
    q.x = x;
    q.gamma = gamma;
    q.eps = gamma != nullptr ? f->norm_eps : 0.0f;
    q.M = M;
    q.K = K;
    q.qx = qx;
    q.sx = sx;
    q.xh = N > 0 ? static_cast<uint4*>(workspace) : nullptr;
    q.nt = tile_tokens(M);
    r = cuda_status(launch_quant_rows(q, x_type, (flags & W4_FLAG_PDL) != 0, s));
    if (r != W4_OK || N == 0) return r;
    return run_gemm8(w, s_w, bias, q.xh, sx, residual, M, N, K, y, y_type, s);
}

}  // extern "C"
