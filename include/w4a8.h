/*
 * w4a8.h -- C ABI of the GB300 (sm_103a) bit-quantized decode GEMV library.
 *
 * The library computes the batch-1 (and few-token) decode linear layer
 *     y[m][j] = W[j][:] . x[m][:] + b[j]
 * with 4-bit (or 8-bit) weights and per-token INT8 activations, as defined on
 *   [Orin-INT4]   "Jetson Orin AGX INT4 推理优化实践：super 分支从 9 tok/s 到 24 tok/s"
 *   [310B-Gemma4] "在香橙派上跑 Gemma4：vLLM 适配昇腾 310B 的内核开发实录"
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers unless a parameter says "host".  The caller
 *     allocates and frees every buffer; the library allocates nothing and keeps
 *     no state beyond cached device attributes and one device error word.
 *   - Work is enqueued on the caller's stream `s` and nothing synchronises.
 *   - Arguments are checked on the host before any launch; a failed check
 *     returns an error and launches nothing.  A launch failure returns
 *     W4_ERR_CUDA.  Kernels never trap: a bounded wait that runs out sets the
 *     device error word (see w4_device_error) and the kernel returns.
 *   - M = 0 or N = 0 is a valid empty call (returns W4_OK, launches nothing).
 *   - Shapes: 1 <= M <= 16 tokens (the INT8 x INT8 linear takes any number), K > 0,
 *     K % 32 == 0.
 *   - Alignment: weight buffers, qx and x must be 16-byte aligned; float
 *     arrays 4-byte aligned.  A violation returns W4_ERR_MISALIGNED.
 *
 * Formats ("canonical" = the format a caller stores, before repacking):
 *   W4    per-row symmetric INT4 [Orin-INT4] §"从 FP 线性层到 INT4 DP4A 的数学推导":
 *         uint32 [N][K/8], weight k of a word in bits 4k..4k+3 (two's complement,
 *         §"DP4A 做了什么"), plus float s_w[N].
 *   Q4_0  [310B-Gemma4] §3.1: 18-byte blocks [N][K/32]: fp16 d (little endian),
 *         then 16 nibble bytes; byte i holds element i (low) and i+16 (high);
 *         element value n - 8, weight d*(n - 8).
 *   I8G32 [310B-Gemma4] §3.2 (lm_head widened to int8 with per-group fp16
 *         scales): int8 q [N][K] plus fp16 d [N][K/32]; weight d*q.
 *
 * Device ("repacked") layouts, produced by the *_repack calls and consumed by
 * the GEMVs.  Rows are grouped in tiles of 8 (T = ceil(N/8) tiles; rows past N
 * are zero).  C = K/32 chunks of 32 weights per row.  Unit (t, c, r) is the
 * 32 weights of row 8t+r in chunk c; units are stored in (t, c, r) order:
 *   W4, Q4_0: 16 bytes per unit at ((t*C + c)*8 + r)*16.  Word w (0..3) of the
 *         unit holds weights 32c+8w+b in the low nibble of byte b and
 *         32c+8w+4+b in the high nibble.  W4 stores each nibble biased,
 *         n = q + 8 in 0..15; Q4_0 stores 4-bit two's complement n - 8.
 *         Padded rows are zero bytes and never reach the output.
 *         Q4_0 then has a plane of fp16 d, one per unit, at byte
 *         T*8*C*16 + ((t*C + c)*8 + r)*2.
 *   I8G32: 32 bytes per unit (the 32 int8 in order) at ((t*C + c)*8 + r)*32,
 *         then the fp16 d plane at byte T*8*C*32 + ((t*C + c)*8 + r)*2.
 *   Q6G32 (the I8G32 values, q in [-32, 31], packed in 6 bits; a layout of
 *         this library, [310B-Gemma4] §3.2 widens them to int8 instead):
 *         n = q + 32.  A low plane of 16 bytes per unit at ((t*C + c)*8 + r)*16
 *         holding n & 15 with the W4 nibble places; a high plane of 8 bytes per
 *         unit at T*8*C*16 + ((t*C + c)*8 + r)*8 holding n >> 4, weight
 *         32c+16h+4s+b in bits 2s..2s+1 of byte b of word h; then the fp16 d
 *         plane at T*8*C*24 + ((t*C + c)*8 + r)*2.  0.8125 bytes per weight.
 */
#ifndef W4A8_H
#define W4A8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* w4_stream_t; /* a cudaStream_t; NULL = legacy default stream */

typedef enum {
    W4_OK = 0,
    W4_ERR_INVALID_ARG = 1,       /* null pointer, negative size, bad shard table */
    W4_ERR_UNSUPPORTED_SHAPE = 2, /* M > 16, K % 32 != 0, K too large, buffer too small */
    W4_ERR_MISALIGNED = 3,        /* a pointer breaks the alignment rule above */
    W4_ERR_CUDA = 4,              /* a CUDA runtime call or launch failed */
    W4_ERR_DEVICE_TIMEOUT = 5     /* a kernel's bounded wait ran out (see w4_device_error) */
} w4_status;

/* Human-readable name of a status.  Never NULL. */
const char* w4_status_str(w4_status st);

/* Library ABI version (increases on incompatible change). */
int w4_version(void);

/* Largest K each GEMV accepts.  Row sums of biased products n * x
 * (|n x| <= 15 * 127) are accumulated in int32, which bounds K near 1.1e6;
 * the library accepts K <= 131072. */
#define W4_MAX_K 131072
#define W4_MAX_M 16
#define W4_MAX_SHARDS 8

/* Flags for the *_linear calls. */
#define W4_FLAG_PDL 1u /* launch as a programmatic dependent of the previous kernel in
                          the stream.  Legal only when the previous kernel does not
                          write this call's weight buffer (weights are prefetched
                          before the dependency wait); inputs x/qx/sx and outputs are
                          touched only after it. */

/* ------------------------------------------------------------------------
 * Launch tuning (process-wide; value 0 restores the automatic choice).
 *   W4_TUNE_BLOCKS_PER_SM  1: one GEMV block per SM with the whole shared
 *                          memory; 2: half of it, so that a GEMV launched with
 *                          W4_FLAG_PDL is resident beside the previous one.
 *                          Default: 2 for one token (when a ring fits), 1 for
 *                          several.
 *   W4_TUNE_MAX_STAGES     cap on the ring depth per warp (>= 2).
 *   W4_TUNE_GRID_BLOCKS    cap on the grid size (default: the SM count).
 *   W4_TUNE_TC_MIN_M       per-row INT4 calls with at least this many tokens
 *                          run on the tensor cores (default 0: 3; 17: never).
 *   W4_TUNE_K_SPLITS       DP4A GEMVs of one or two tokens: K split over a
 *                          cluster of 2, 4 or 8 blocks sharing a tile range
 *                          (where each split keeps at least 16 chunks of 32 K);
 *                          0 or 1: no split, the default (a split measured
 *                          slower on every shape tried).
 *   W4_TUNE_GROUP_LAUNCH_TOKENS  Q4_0 / I8G32 / Q6G32 calls with more tokens
 *                          than this run as launches of at most this many
 *                          tokens (1..16; default 0: 8).
 *   W4_TUNE_CHAIN_PREFETCH_KB  w4a8_linear_chain: weight bytes (KB, at most
 *                          4096) each block prefetches into L2 ahead of the
 *                          weights it copies into shared memory (default
 *                          0: none; below 32 none).
 * Returns W4_ERR_INVALID_ARG for an unknown key or an out-of-range value.
 * Not thread-safe with concurrent launches; set before launching.
 * ------------------------------------------------------------------------ */
#define W4_TUNE_BLOCKS_PER_SM 0
#define W4_TUNE_MAX_STAGES 1
#define W4_TUNE_GRID_BLOCKS 2
#define W4_TUNE_TC_MIN_M 3
#define W4_TUNE_CHAIN_PREFETCH_KB 4
#define W4_TUNE_K_SPLITS 5
#define W4_TUNE_GROUP_LAUNCH_TOKENS 6
w4_status w4_set_tuning(int key, int value);
int w4_get_tuning(int key); /* current value, -1 for an unknown key */

/* ------------------------------------------------------------------------
 * Launch plan: what a GEMV or linear call launches on a device, computed on
 * the host from a description of the device (no CUDA call, so it also runs
 * without a GPU).  The launch path takes its decisions through the same
 * functions, with the current tuning (w4_set_tuning).
 *   fmt:  W4_FMT_W4, W4_FMT_Q4_0, W4_FMT_I8G32 or W4_FMT_Q6G32.
 *   M, N, K: the call's shapes (N outputs; a gated call reads 2N weight rows).
 *   what: 0 for the *_gemv call on int8 codes, or W4_PLAN_LINEAR for the
 *         *_linear call on float x, with W4_PLAN_NORM (RMSNorm fused in, a
 *         *_linear_fused option) and W4_PLAN_GLU (gated, W4 and Q4_0 only).
 *   dev:  host; the device attributes of the same names (SM count, shared
 *         memory per SM, shared memory per block reserved by the system,
 *         opt-in maximum per block).  w4_describe_device fills it for the
 *         current device.
 *   out:  host; path (W4_PATH_*), quantize_launches (1 when a *_linear call
 *         quantizes x in a kernel of its own first, else 0), and the GEMV
 *         launch: grid, threads, smem_bytes (dynamic, per block), stages
 *         (weight-ring depth), k_splits (K splits per tile range, which form
 *         one thread-block cluster: per 128-row group on the tensor cores, per
 *         range of 8-row tiles on DP4A; 1 without a split), gemv_launches
 *         (GEMV kernels per call: 0 without a GEMV; 2 for a Q4_0 / I8G32 /
 *         Q6G32 call of more than 8 tokens, which runs tokens 0-7 and the
 *         rest as two launches of one kernel over the same weights, both
 *         as the fields above describe; otherwise 1).
 * Paths:
 *   W4_PATH_NONE          nothing (M = 0, or N = 0 where only the quantizer
 *                         of a *_linear call runs);
 *   W4_PATH_FUSED         one DP4A GEMV launch with the activation quantizer
 *                         (and the norm) in its prologue;
 *   W4_PATH_CODES_SMEM    DP4A GEMV on int8 codes staged in shared memory;
 *   W4_PATH_CODES_GLOBAL  DP4A GEMV reading the int8 codes from global memory;
 *   W4_PATH_TENSOR_CORES  tensor-core GEMV on int8 codes (per-row INT4).
 * Returns W4_ERR_INVALID_ARG for a null pointer, an unknown fmt or flag, a
 * non-positive device field, W4_PLAN_NORM without W4_PLAN_LINEAR or a GLU on
 * I8G32 / Q6G32, and otherwise the shape status the call would return.
 * ------------------------------------------------------------------------ */
#define W4_FMT_W4 0
#define W4_FMT_Q4_0 1
#define W4_FMT_I8G32 2
#define W4_FMT_Q6G32 3
#define W4_PLAN_LINEAR 1u
#define W4_PLAN_NORM 2u
#define W4_PLAN_GLU 4u
#define W4_PATH_NONE 0
#define W4_PATH_FUSED 1
#define W4_PATH_CODES_SMEM 2
#define W4_PATH_CODES_GLOBAL 3
#define W4_PATH_TENSOR_CORES 4
typedef struct {
    int sms;
    int smem_per_sm;
    int smem_reserved;
    int smem_optin;
} w4_device_desc;
typedef struct {
    int path;
    int quantize_launches;
    int grid;
    int threads;
    int smem_bytes;
    int stages;
    int k_splits;
    int gemv_launches;
} w4_launch_plan;
w4_status w4_plan(int fmt, int M, int N, int K, unsigned what, const w4_device_desc* dev, w4_launch_plan* out);
/* The current device's description (W4_ERR_CUDA without a usable device). */
w4_status w4_describe_device(w4_device_desc* out);

/* ------------------------------------------------------------------------
 * Load time: quantize float weights (device kernels).
 * ------------------------------------------------------------------------ */

/* Per-row symmetric INT4, [Orin-INT4] §"从 FP 线性层到 INT4 DP4A 的数学推导":
 * s_w[j] = max_i |W[j][i]| / 7 (the page leaves s^W open; this maps the row's
 * absmax to the top code, as s^x does for x), q = clip(rint(W / s_w), -8, 7),
 * packed into canonical W4 words.  W: float [N][K] (16-B aligned, row-major);
 * packed: uint32 [N][K/8]; s_w: float [N].  K % 8 == 0. */
w4_status w4_quantize_rows(const float* W, int N, int K, uint32_t* packed, float* s_w, w4_stream_t s);

/* Q4_0 blocks, [310B-Gemma4] §3.1: d = fp16(max|w| / 8) per 32-block,
 * n = clip(rint(w / d), -8, 7) + 8.  W: float [N][K]; blocks: [N][K/32][18]. */
w4_status q4_0_quantize(const float* W, int N, int K, uint8_t* blocks, w4_stream_t s);

/* int8 + fp16 group-32 scales, [310B-Gemma4] §3.2: d = fp16(max|w| / 32),
 * q = clip(rint(w / d), -32, 31).  q: int8 [N][K]; d: fp16 bits [N][K/32]. */
w4_status i8g32_quantize(const float* W, int N, int K, int8_t* q, uint16_t* d, w4_stream_t s);

/* ------------------------------------------------------------------------
 * Load time on the host: the same three quantizers as plain C++ over host
 * memory, for loaders that hold float weights on the host.  Outputs are
 * bit-identical to the device calls above (IEEE fp32 division,
 * round-half-to-even to an integer, fp16 round-to-nearest-even).  All
 * pointers are HOST pointers (no alignment rule); the call is synchronous,
 * makes no CUDA call and keeps no state, so it is safe from any thread.
 * Same shapes and checks as the device calls: N >= 0, K > 0, and K % 8 == 0
 * (w4_quantize_rows_host) or K % 32 == 0 (the group formats).
 * ------------------------------------------------------------------------ */
w4_status w4_quantize_rows_host(const float* W, int N, int K, uint32_t* packed, float* s_w);
w4_status q4_0_quantize_host(const float* W, int N, int K, uint8_t* blocks);
w4_status i8g32_quantize_host(const float* W, int N, int K, int8_t* q, uint16_t* d);

/* ------------------------------------------------------------------------
 * Load time: repack canonical weights into the device layout, fusing shards.
 * [310B-Gemma4] §3.1 (load-time reorder; q/k/v and gate/up concatenated by
 * rows into one matrix, one repack, one matmul per token).
 *
 * shard_* are HOST arrays of n_shards (1..W4_MAX_SHARDS) device pointers;
 * shard_rows is a HOST array of row counts.  The fused matrix has
 * N = sum(shard_rows) rows, shard 0 first.  `out` must hold *_repacked_bytes
 * (N, K) bytes (out_bytes is checked) and must not overlap the shards.
 * ------------------------------------------------------------------------ */
size_t w4_repacked_bytes(int N, int K);
w4_status w4_repack(const uint32_t* const* shard_packed, const int* shard_rows, int n_shards, int K,
                    void* out, size_t out_bytes, w4_stream_t s);

size_t q4_0_repacked_bytes(int N, int K);
w4_status q4_0_repack(const uint8_t* const* shard_blocks, const int* shard_rows, int n_shards, int K,
                      void* out, size_t out_bytes, w4_stream_t s);

size_t i8g32_repacked_bytes(int N, int K);
w4_status i8g32_repack(const int8_t* const* shard_q, const uint16_t* const* shard_d, const int* shard_rows,
                       int n_shards, int K, void* out, size_t out_bytes, w4_stream_t s);

/* Q6G32 from the I8G32 canonical format (codes must lie in [-32, 31], as
 * i8g32_quantize makes them; other codes are packed modulo 64). */
size_t q6g32_repacked_bytes(int N, int K);
w4_status q6g32_repack(const int8_t* const* shard_q, const uint16_t* const* shard_d, const int* shard_rows,
                       int n_shards, int K, void* out, size_t out_bytes, w4_stream_t s);

/* Gate/up weights of a gated MLP, paired for the GLU epilogue of the
 * *_linear_fused calls: row tile t holds gate rows 4t..4t+3 and then up rows
 * 4t..4t+3 (8 ceil(I/4) rows in all, padding past I zero), so one thread
 * block sees both halves of every output.  gate and up: canonical [I][..]
 * device arrays (W4: uint32 [I][K/8]; Q4_0: 18-byte blocks [I][K/32]; per-row
 * INT8, for the experts of w4_moe_experts: int8 [I][K]).
 * out: *_glu_repacked_bytes(I, K) bytes, 16-byte aligned. */
size_t w4_glu_repacked_bytes(int I, int K);
w4_status w4_repack_glu(const uint32_t* gate, const uint32_t* up, int I, int K, void* out, size_t out_bytes,
                        w4_stream_t s);
size_t w8_glu_repacked_bytes(int I, int K);
w4_status w8_repack_glu(const int8_t* gate, const int8_t* up, int I, int K, void* out, size_t out_bytes,
                        w4_stream_t s);
size_t q4_0_glu_repacked_bytes(int I, int K);
w4_status q4_0_repack_glu(const uint8_t* gate, const uint8_t* up, int I, int K, void* out, size_t out_bytes,
                          w4_stream_t s);

/* Concatenate per-shard float vectors (per-row scales s_w, bias) into `out`
 * in shard order.  parts: HOST array of device pointers; lens: HOST array. */
w4_status w4_concat_f32(const float* const* parts, const int* lens, int n_parts, float* out, w4_stream_t s);

/* ------------------------------------------------------------------------
 * Per token: activation quantization.
 * [Orin-INT4] §"从 FP 线性层到 INT4 DP4A 的数学推导":
 *   sx[m] = max_i |x[m][i]| / 127 (IEEE fp32 division),
 *   qx[m][i] = clip(rint(x[m][i] / sx[m]), -127, 127); an all-zero token gives
 *   sx = 0, qx = 0.  NaN/Inf inputs are undefined behaviour.
 * x: float [M][K]; qx: int8 [M][K]; sx: float [M].
 * ------------------------------------------------------------------------ */
w4_status a8_quantize(const float* x, int M, int K, int8_t* qx, float* sx, w4_stream_t s);

/* ------------------------------------------------------------------------
 * Per token: GEMV on INT8 activations.
 *
 * w4a8_gemv, [Orin-INT4] §"从 FP 线性层到 INT4 DP4A 的数学推导" and §"DP4A 做了什么":
 *   acc[m][j] = sum_i q_w[j][i] * qx[m][i]   (exact int32),
 *   y[m][j]   = fmaf(s_w[j] * sx[m], (float)acc, b[j])   (b = 0 if bias NULL).
 *   Up to two tokens the sums run on DP4A; from three tokens (see
 *   W4_TUNE_TC_MIN_M) on the tensor cores, with exact fp8 products and fp32
 *   partial sums.  y is bit-identical either way.
 * q4_0_gemv / i8g32_gemv / q6g32_gemv, [310B-Gemma4] §3.1 / §3.2:
 *   acc_g = exact int32 sum over 32-block g,
 *   y[m][j] = fmaf(sx[m], sum_g d_g * acc_g, b[j])  (fp32; group order unspecified).
 *   With more than 8 tokens these (and the *_linear calls of these formats)
 *   run as two launches of the eight-token kernel, tokens 0-7 and the rest,
 *   each reading the weights once.  Every step is per token: codes, scales
 *   and integer group sums are those of one launch; y may differ from a call
 *   of other token counts only in the fp32 group-sum order.
 * w: repacked weights; s_w: float [N]; bias: float [N] or NULL; qx: int8 [M][K];
 * sx: float [M]; y: float [M][N] (row m at y + m*N).
 * ------------------------------------------------------------------------ */
w4_status w4a8_gemv(const void* w, const float* s_w, const float* bias, const int8_t* qx, const float* sx,
                    int M, int N, int K, float* y, w4_stream_t s);
/* Device scratch a GEMV or linear call of this shape needs from its caller:
 * always 0.  Where K is split over several blocks (W4_PATH_* plans with
 * k_splits > 1) the partial sums merge on chip, in the shared memory of one
 * thread-block cluster, so no call takes a workspace. */
size_t w4_workspace_bytes(int M, int N, int K);
w4_status q4_0_gemv(const void* w, const float* bias, const int8_t* qx, const float* sx,
                    int M, int N, int K, float* y, w4_stream_t s);
w4_status i8g32_gemv(const void* w, const float* bias, const int8_t* qx, const float* sx,
                     int M, int N, int K, float* y, w4_stream_t s);
w4_status q6g32_gemv(const void* w, const float* bias, const int8_t* qx, const float* sx,
                     int M, int N, int K, float* y, w4_stream_t s);

/* ------------------------------------------------------------------------
 * Per token: the whole decode linear, quantization fused into the GEMV
 * ([Orin-INT4] §"后续还能继续优化什么" item 2 names fusing the activation
 * quantization with a neighbouring operator).  Each thread block quantizes x
 * into its shared memory; block 0 also writes qx and sx (caller buffers, same
 * shapes as a8_quantize) so that the caller sees the codes used.  When M*K
 * does not fit in shared memory the call runs a8_quantize into qx/sx and then
 * the *_gemv kernel; results are identical either way.
 * flags: 0 or W4_FLAG_PDL.
 * ------------------------------------------------------------------------ */
w4_status w4a8_linear(const void* w, const float* s_w, const float* bias, const float* x, int M, int N, int K,
                      float* y, int8_t* qx, float* sx, unsigned flags, w4_stream_t s);
w4_status q4_0_linear(const void* w, const float* bias, const float* x, int M, int N, int K,
                      float* y, int8_t* qx, float* sx, unsigned flags, w4_stream_t s);
w4_status i8g32_linear(const void* w, const float* bias, const float* x, int M, int N, int K,
                       float* y, int8_t* qx, float* sx, unsigned flags, w4_stream_t s);
w4_status q6g32_linear(const void* w, const float* bias, const float* x, int M, int N, int K,
                       float* y, int8_t* qx, float* sx, unsigned flags, w4_stream_t s);

/* ------------------------------------------------------------------------
 * The decode linear with its neighbouring operators fused in.
 * [Orin-INT4] §"后续还能继续优化什么" item 1 names the kernel boundaries
 * between RMSNorm, quantization, linear, SwiGLU and the residual add;
 * [310B-Gemma4] §4.2 names add+rmsnorm and gelu+mul fusions.  With f:
 *   - f->norm_weight != NULL: x is first normalized per token,
 *       r = 1 / sqrt(S / K + eps),  x'_i = (x_i * r) * g_i,
 *     with S = sum_i x_i^2 rounded once to fp32 and every other step an IEEE
 *     fp32 operation; x' is then quantized (qx, sx hold its codes).
 *     norm_weight: float [K], 16-byte aligned; norm_eps > 0 and finite.
 *   - f->glu = W4_GLU_SILU or W4_GLU_GELU_TANH: w comes from *_repack_glu
 *     (I = N gate rows and N up rows); s_w and bias hold 2N values, the gate
 *     rows' then the up rows'; the linear's gate and up outputs g, u (each
 *     exactly as the plain linear makes them) become
 *       SiLU:      y = fl(fl(g / fl(1 + expf(-g))) * u)
 *       GELU tanh: y = (g / 2)(1 + tanhf(sqrt(2/pi)(g + 0.044715 g^3))) u,
 *     y: float [M][N].  Only W4 and Q4_0 take a GLU.
 *   - f->residual != NULL: float [M][N], added last, y = residual + out (fp32);
 *     it may be y itself (the in-place residual update) but must not
 *     otherwise overlap y.
 * f = NULL or all fields zero is exactly the *_linear call.  x must not
 * overlap y.  Many tokens (the tensor-core path) or a long x run the
 * normalize+quantize as its own kernel (rms_a8_quantize) ahead of the GEMV;
 * the results are the same.
 * ------------------------------------------------------------------------ */
#define W4_GLU_NONE 0
#define W4_GLU_SILU 1
#define W4_GLU_GELU_TANH 2
typedef struct {
    const float* norm_weight;
    float norm_eps;
    int glu;
    const float* residual;
} w4_fusion;

w4_status w4a8_linear_fused(const void* w, const float* s_w, const float* bias, const float* x, int M, int N,
                            int K, float* y, int8_t* qx, float* sx, const w4_fusion* f, unsigned flags,
                            w4_stream_t s);
w4_status q4_0_linear_fused(const void* w, const float* bias, const float* x, int M, int N, int K, float* y,
                            int8_t* qx, float* sx, const w4_fusion* f, unsigned flags, w4_stream_t s);
w4_status i8g32_linear_fused(const void* w, const float* bias, const float* x, int M, int N, int K, float* y,
                             int8_t* qx, float* sx, const w4_fusion* f, unsigned flags, w4_stream_t s);
w4_status q6g32_linear_fused(const void* w, const float* bias, const float* x, int M, int N, int K, float* y,
                             int8_t* qx, float* sx, const w4_fusion* f, unsigned flags, w4_stream_t s);

/* RMSNorm (as above) then the activation quantizer, one kernel: qx, sx of
 * the normalized tokens.  x: float [M][K]; norm_weight: float [K]. */
w4_status rms_a8_quantize(const float* x, const float* norm_weight, float eps, int M, int K, int8_t* qx, float* sx,
                          unsigned flags, w4_stream_t s);

/* The same operators as separate kernels (what a decoder runs without the
 * fusions), fp32 in and out, flags 0 or W4_FLAG_PDL:
 *   w4_rmsnorm: out[M][K] = RMSNorm(x) exactly as above (out may not overlap x);
 *   w4_glu:     out[M][I] = act(gu[m][j]) * gu[m][I + j] for a [M][2I] gate|up
 *               output (kind W4_GLU_SILU or W4_GLU_GELU_TANH), as above;
 *   w4_add:     out[i] = a[i] + b[i], i < n (out may be a or b). */
w4_status w4_rmsnorm(const float* x, const float* norm_weight, float eps, int M, int K, float* out, unsigned flags,
                     w4_stream_t s);
w4_status w4_glu(const float* gu, int kind, int M, int I, float* out, unsigned flags, w4_stream_t s);
w4_status w4_add(const float* a, const float* b, long long n, float* out, unsigned flags, w4_stream_t s);

/* ------------------------------------------------------------------------
 * Weight-only paths on float activations: the two paths [Orin-INT4]
 * §"为什么 INT4 float 解包不快" measures INT4 DP4A against (weight-only INT8,
 * and INT4 unpacked to float).  The activations are not quantized:
 *   y[m][j] = fmaf(s_w[j], sum_i q_w[j][i] * x[m][i], b[j]),
 * every weight converted to fp32 and multiply-added in fp32 (summation order
 * unspecified).
 *   w4a32_gemv: per-row INT4 weights in the w4_repack layout (the bytes the
 *     DP4A path reads), unpacked to float.
 *   w8a32_gemv: per-row INT8 weights from w8_quantize_rows (s_w = max|W|/127,
 *     q = clip(rint(W / s_w), -127, 127), int8 [N][K]) in the w8_repack
 *     layout: 32-byte units holding a row's 32 int8 weights of a chunk in
 *     order, in the (t, c, r) order of the other formats, no scale plane.
 * x: float [M][K], 16-byte aligned; 1 <= M <= 4; flags: 0 or W4_FLAG_PDL.
 * x is staged in shared memory as fp32 beside a weight ring of at least two
 * stages, so M*K is limited to about 40000 values (W4_ERR_UNSUPPORTED_SHAPE
 * beyond: K = 18944 takes at most two tokens).
 * ------------------------------------------------------------------------ */
w4_status w8_quantize_rows(const float* W, int N, int K, int8_t* q, float* s_w, w4_stream_t s);
size_t w8_repacked_bytes(int N, int K);
w4_status w8_repack(const int8_t* const* shard_q, const int* shard_rows, int n_shards, int K, void* out,
                    size_t out_bytes, w4_stream_t s);
w4_status w4a32_gemv(const void* w, const float* s_w, const float* bias, const float* x, int M, int N, int K,
                     float* y, unsigned flags, w4_stream_t s);
w4_status w8a32_gemv(const void* w, const float* s_w, const float* bias, const float* x, int M, int N, int K,
                     float* y, unsigned flags, w4_stream_t s);

/* ------------------------------------------------------------------------
 * INT8 x INT8 linear with a scale for each token and each output channel, for
 * any number of tokens (a prompt as well as a decode step):
 *   acc[m][j] = sum_i q_w[j][i] * qx[m][i]   (exact int32),
 *   y[m][j]   = fmaf(s_w[j] * sx[m], (float)acc[m][j], b[j]) (+ residual),
 * rounded to y's type (to nearest even).  Weights: the per-row INT8 of
 * w8_quantize_rows in the w8_repack layout (any int8, -128 included).
 *   w8a8_matmul  takes codes and scales (as a8_quantize makes them);
 *   w8a8_linear  quantizes x first, with f->norm_weight normalized as in the
 *     *_linear_fused calls; the arithmetic of both is theirs, on x widened to
 *     fp32.  qx: int8 [M][K] receives the codes, or NULL; sx: float [M]
 *     receives the scales.
 * x: [M][K] of x_type, 16-byte aligned; y: [M][N] of y_type; residual: float
 * [M][N], added in fp32 before the rounding (it may be y itself where y is
 * W4_F32).  x must not overlap y.  f may be NULL; a GLU is refused.
 * 0 <= M <= W4_MAX_TOKENS, K % 32 == 0, any N.
 * workspace: device memory of w8a8_workspace_bytes(M, N, K) bytes (2 K for each
 * token and up to 192 of padding), 16-byte aligned, with no contents to keep; calls that
 * share one must not overlap on the GPU.  W4_FLAG_PDL as above: the weights
 * are fetched before the dependency wait.
 * The codes and the scale of a token given, its row is the same in every batch,
 * and so are the codes of an x that is not normalized.  With norm_weight the sum
 * of squares is added in an order that depends on M, to 2^-45 of it, and rounded
 * once: for a sum that close to a rounding boundary (one random token in some 10
 * million) r, and with it a few codes, may be a step off another batch's.
 * ------------------------------------------------------------------------ */
#define W4_F32 0
#define W4_F16 1
#define W4_BF16 2
#define W4_MAX_TOKENS (1 << 20)
size_t w8a8_workspace_bytes(int M, int N, int K); /* 0 for a shape the calls refuse */
w4_status w8a8_matmul(const void* w, const float* s_w, const float* bias, const int8_t* qx, const float* sx, int M,
                      int N, int K, void* y, int y_type, void* workspace, size_t ws_bytes, w4_stream_t s);
w4_status w8a8_linear(const void* w, const float* s_w, const float* bias, const void* x, int x_type, int M, int N,
                      int K, void* y, int y_type, int8_t* qx, float* sx, const w4_fusion* f, unsigned flags,
                      void* workspace, size_t ws_bytes, w4_stream_t s);

/* ------------------------------------------------------------------------
 * Mixture-of-experts layer for 1 to 16 tokens: a router and the experts' gated
 * MLP on per-row INT4 or INT8 weights and INT8 activations.
 *
 * w4_moe_route, one launch.  With x' = RMSNorm(x) as in the *_linear_fused
 * calls (or x, without norm_weight):
 *   l_e = sum_i x'_i w[e][i], rounded once to fp32 from a compensated sum;
 *   W4_ROUTE_SOFTMAX: the top_k experts by l; p = softmax(l) over all E;
 *   W4_ROUTE_SIGMOID: p_e = 1 / (1 + exp(-l_e)) rounded once to fp32 (subnormal
 *     values to half a step and 2^-24 of the value), the top_k experts by
 *     fp32(p_e + select_bias[e]);
 *   equal keys: the lowest index first.  weights = p of the chosen (divided by
 *   their sum with renormalize; 0 where that sum is 0) * scale.
 * ids: int [M][top_k], best first; weights: float [M][top_k]; qx, sx: the
 * codes and scales of x' (as rms_a8_quantize makes them), or both NULL.
 * x: [M][K] of x_type, 16-byte aligned; w: float [E][K], 16-byte aligned;
 * K % 32 == 0, 1 <= top_k <= min(E, 16), E <= 1024; K up to about 50000 (a
 * token is kept in shared memory as fp32).  A logit past fp32 is an infinity
 * of its sign (softmax then has NaN weights); a NaN logit is the last choice;
 * the ids are valid and distinct whatever x holds.  The order of the sums
 * depends on M: a logit within 2^-44 of its terms' magnitudes of a rounding
 * boundary may be a step off another batch's (and r, as for w8a8_linear).
 *
 * w4_moe_experts.  For every token m and slot s with expert e = ids[m][s]:
 *   g, u = linear(qx, sx) by e's gate and up rows, as the W4 / W8A8 linears,
 *   h    = act(g) u, evaluated to one fp32 rounding over the whole range of g
 *          and u (subnormal values to half a step and 2^-24 of the value),
 *   d    = linear of h's codes (quantized as a8_quantize does) by e's down rows,
 *   y[m] = sum over the slots in order of weights[m][s] * d (fp32), then the
 *          n_shared shared experts with weight 1, then + residual[m], rounded
 *          to y's type.
 * An id outside 0 .. E - 1 is an empty slot and contributes nothing; a token
 * with empty slots only gets the residual (or 0).  An expert may be named
 * twice.  The experts' weights are read once for all their tokens; for given
 * codes, ids and weights the results do not depend on the other tokens of the
 * call, nor on timing.
 *   experts: E + n_shared of them, the shared ones last, one behind the other:
 *     w_gu  *_repack_glu of gate and up [I][H] each, *_glu_repacked_bytes(I, H)
 *           apart;   s_gu (b_gu): float [E + n_shared][2 I], gate rows first;
 *     w_dn  *_repack of down [H][I], *_repacked_bytes(H, I) apart;
 *           s_dn (b_dn): float [E + n_shared][H].
 *     fmt: W4_FMT_W4 or W4_FMT_W8; glu: W4_GLU_SILU or W4_GLU_GELU_TANH;
 *     H % 32 == 0, I % 32 == 0; E + n_shared <= 1024, n_shared <= 4.
 *   residual: float [M][H] or NULL (may be y itself where y is W4_F32).
 *   workspace: w4_moe_workspace_bytes(..) bytes, 16-byte aligned, with no
 *     contents to keep; calls that share one must not overlap on the GPU.
 * Two launches (the first prepares the workspace).  The kernel waits
 * on its own blocks' progress with bounded waits (see w4_device_error), but
 * needs no co-resident grid: calls on several streams, each with its own
 * workspace, may run at once.
 *
 * w4_moe_layer: w4_moe_route, then w4_moe_experts on its choice, in two
 * launches, the second a programmatic dependent of the first; ids, weights,
 * qx and sx receive the choice and the codes (none may be NULL).
 * flags: 0 or W4_FLAG_PDL.  M = 0 is a valid empty call.
 * ------------------------------------------------------------------------ */
#define W4_FMT_W8 5 /* per-row INT8 (w8_quantize_rows); w4_experts only */
#define W4_ROUTE_SOFTMAX 0
#define W4_ROUTE_SIGMOID 1
#define W4_MAX_TOP_K 16
#define W4_MAX_EXPERTS 1024
#define W4_MAX_SHARED 4
typedef struct {
    const float* norm_weight; /* [K] or NULL */
    float norm_eps;
    const float* w;           /* [E][K] */
    const float* select_bias; /* [E] or NULL; W4_ROUTE_SIGMOID only */
    int E;
    int top_k;
    int score;
    int renormalize;
    float scale;
} w4_router;
typedef struct {
    int fmt;
    int E;
    int n_shared;
    int H;
    int I;
    int glu;
    const void* w_gu;
    const float* s_gu;
    const float* b_gu; /* or NULL */
    const void* w_dn;
    const float* s_dn;
    const float* b_dn; /* or NULL */
} w4_experts;
w4_status w4_moe_route(const w4_router* r, const void* x, int x_type, int M, int K, int* ids, float* weights,
                       int8_t* qx, float* sx, unsigned flags, w4_stream_t s);
size_t w4_moe_workspace_bytes(const w4_experts* e, int M, int top_k); /* 0 for what the calls refuse */
w4_status w4_moe_experts(const w4_experts* e, const int8_t* qx, const float* sx, const int* ids,
                         const float* weights, int M, int top_k, const float* residual, void* y, int y_type,
                         void* workspace, size_t ws_bytes, unsigned flags, w4_stream_t s);
w4_status w4_moe_layer(const w4_router* r, const w4_experts* e, const void* x, int x_type, int M, int* ids,
                       float* weights, int8_t* qx, float* sx, const float* residual, void* y, int y_type,
                       void* workspace, size_t ws_bytes, unsigned flags, w4_stream_t s);

/* ------------------------------------------------------------------------
 * Attention over a paged cache, for a decode step or the verification of a
 * tree of drafted tokens: the operators between the q/k/v and the output
 * projection.
 *
 * w4_kv_cache: one layer's cache, k and v [pages][Hkv][page_size][D] of
 *   W4_F16, W4_BF16 or W4_I8, 16-byte aligned.  INT8 codes have a scale for
 *   each token and head, k_scale and v_scale [pages][Hkv][page_size], 16-byte
 *   aligned (NULL for the 16-bit types).  D is 64, 128 or 256, page_size a
 *   power of two from 16 to 256.
 * w4_kv_batch: which rows of a call are whose.  Sequence b < B (at most
 *   W4_MAX_SEQUENCES) has rows q_start[b] .. q_start[b + 1] - 1 (q_start int
 *   [B + 1], ascending from 0) and ctx[b] places before them.  Row i of a
 *   sequence has place ctx[b] + i: entry (place % page_size) of page
 *   table[b][place / page_size] (table int [B][max_pages]).  Rows behind the
 *   last sequence are left as they are.  A page outside 0 .. pages - 1, or a
 *   place past the table, holds nothing: it is not written, and no row sees
 *   it.  The arrays live on the device, so a captured call follows them.
 *   max_tokens: the most rows of a sequence (rows past it get no attention);
 *   at most W4_MAX_DRAFTS for w4_tree_attention, any number for w4_kv_append.
 *
 * w4_rope_table: turns float [positions][rot / 2][2], 16-byte aligned,
 *   (cos, sin)(p * factor * inv_freq[i]) * scale: angles in 64 bits, each
 *   number rounded once; rot % 8 == 0, at most 256.  inv_freq: double
 *   [rot / 2] on the device.
 * w4_kv_append, one launch: rows qkv [T] of ld values of x_type (16-byte
 *   aligned, so is ld), Hq query heads, then Hkv key and Hkv value heads of D.
 *   RMSNorm of each query (q_norm float [D]) and key head (k_norm), either
 *   may be NULL; rotation of the first rot values of each query and key head
 *   (rope NULL: none) by row positions[t] of the table (NULL: the row's
 *   place), in pairs (i, i + rot / 2) (W4_ROPE_HALF) or (2 i, 2 i + 1)
 *   (W4_ROPE_INTERLEAVED): a' = a c - b s, b' = b c + a s.  A position that
 *   the table does not have gives NaN.  A head that holds a NaN has codes of 0
 *   and the scale NaN in an INT8 cache.  q [T][Hq][D] of q_type
 *   (W4_F16 or W4_BF16), 16-byte aligned; k and v go to the cache, rounded
 *   once (norms of what goes to 16 bits are plain fp32 sums), or as the codes
 *   and scale that a8_quantize gives for a head's values (the norm's steps
 *   then as in rms_a8_quantize, a rotated value of a key rounded once to
 *   fp32).  Two rows with the same place race.
 * w4_kv_values: out float [pages][Hkv][page_size][D], 16-byte aligned: the
 *   numbers that an INT8 cache's keys (W4_KEYS) or values (W4_VALUES) stand
 *   for, codes times scales, every page of the cache.
 * w4_tree_attention: y[t][h] = sum p v / sum p, p = exp(scale q.k) (0 < scale <
 *   2e38), over the
 *   places below ctx and the drafts of the row's own sequence (the rows of
 *   this call, already appended) whose bit the row's mask has: bit j of
 *   mask[t] (uint64, device) is row j of the sequence.  mask NULL: row i sees
 *   rows 0 .. i.  A row that sees nothing gets 0.  What a row does not see
 *   does not reach it, infinities and NaN included.  An infinite value (or
 *   scale of values) that it sees makes its outputs infinite, or NaN where the
 *   probability is 0 in 16 bits or, in two parts of fp16, below 2^-13 of the
 *   row's largest.  q [T][Hq][D] of the
 *   cache's type (either 16-bit type for W4_I8), y [T][Hq][D] of y_type, both
 *   16-byte aligned; query head h reads key head h / (Hq / Hkv).
 *   Sums in fp32, of which the tensor cores cut up to 2^-23 a step: 192 steps
 *   at most where y is W4_F32 (or W4_F16 of another cache), 1024 where it is
 *   W4_F16 over a W4_F16 cache, 8192 where it is W4_BF16.  A probability enters
 *   the second product in the 16-bit type of the values (bf16 for W4_I8) in two
 *   parts, in three where that is bf16 and y is W4_F32, in one where it is fp16
 *   and y W4_BF16.  In fp16 it is off by 2^-34 of the row's largest besides
 *   (fp16's least step).
 *   workspace: w4_tree_attention_workspace_bytes(..) bytes, 16-byte aligned,
 *   with no contents to keep; calls that share one must not overlap on the
 *   GPU.  Two launches.  For given inputs the result is the same in every
 *   call, but it depends on the other sequences of the call in its last bits
 *   (how a sequence is split).
 * flags: 0 or W4_FLAG_PDL (the same: these kernels touch no memory before
 * their dependency wait, so every launch is a programmatic dependent of the
 * one before it).  T = 0 or B = 0 is a valid empty call.
 * ------------------------------------------------------------------------ */
#define W4_I8 3
#define W4_ROPE_HALF 0
#define W4_ROPE_INTERLEAVED 1
#define W4_KEYS 0
#define W4_VALUES 1
#define W4_MAX_SEQUENCES 1024
#define W4_MAX_DRAFTS 64
typedef struct {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int type;
    int pages;
    int page_size;
    int Hkv;
    int D;
} w4_kv_cache;
typedef struct {
    const int* table;
    const int* ctx;
    const int* q_start;
    int B;
    int max_pages;
    int max_tokens;
} w4_kv_batch;
typedef struct {
    const float* turns;
    int positions;
    int rot;
    int layout;
} w4_rope;
w4_status w4_rope_table(const double* inv_freq, double factor, double scale, int positions, int rot, float* turns,
                        w4_stream_t s);
w4_status w4_kv_append(const w4_kv_cache* c, const w4_kv_batch* b, const w4_rope* rope, const void* qkv, int x_type,
                       long long ld, int T, int Hq, const int* positions, const float* q_norm, const float* k_norm,
                       float eps, void* q, int q_type, unsigned flags, w4_stream_t s);
w4_status w4_kv_values(const w4_kv_cache* c, int which, float* out, w4_stream_t s);
size_t w4_tree_attention_workspace_bytes(const w4_kv_cache* c, const w4_kv_batch* b, int T, int Hq); /* 0: refused or empty */
w4_status w4_tree_attention(const w4_kv_cache* c, const w4_kv_batch* b, const void* q, int q_type, int T, int Hq,
                            const unsigned long long* mask, float scale, void* y, int y_type, void* workspace,
                            size_t ws_bytes, unsigned flags, w4_stream_t s);

/* ------------------------------------------------------------------------
 * w4_logits_adjust, one or two launches: penalties for repeated tokens, biases and a
 * grammar's mask on rows of logits, behind the vocabulary projection.
 *   Sequence s < S has length[s] tokens ids[s][..] (ids int [S][cap]), the
 *   first prompt[s] of them the prompt (prompt NULL: none), the others
 *   generated.  Row r is sequence r's, or with row_start (int [S + 1],
 *   ascending from 0) row row_start[s] + i is sequence s's i-th; rows behind
 *   the last sequence are left as they are.  drafts int [R]: the token of each row in a
 *   drafted tree; row r's path (bit j of mask[r]: row j of its sequence, j <
 *   64; mask NULL: rows 0 .. i) counts as generated, r's own token with its own bit.
 *   For token v with n occurrences among the generated ones:
 *     l = l > 0 ? l / repetition[s] : l * repetition[s]   if n > 0 or v is in the prompt,
 *     l = l - frequency[s] * n - presence[s]              if n > 0,
 *     l = l + the sum of v's biases, added up from 0 in their order (bias_ids int [S][n_bias], bias float),
 *     l = -inf                                            if bit v % 32 of allowed[r][v / 32] is 0,
 *   each step an fp32 operation, rounded to the logits' type.  The arrays of
 *   factors float [S] may be NULL (1, 0 and 0), so may allowed (uint32 [R][ceil(V / 32)]).
 *   Ids outside 0 .. V - 1 are passed over.  logits: [R] rows of ld values of
 *   `type`, out the same with ld_out (it may be logits itself, with
 *   the same ld).  V <= 2^24, cap <= 2^28,
 *   n_bias <= W4_MAX_BIASES.  The rows must not overlap other than that.  flags:
 *   0 or W4_FLAG_PDL (the same, as above).
 * ------------------------------------------------------------------------ */
#define W4_MAX_BIASES 1024
typedef struct {
    int V;
    int S;
    const int* ids;          /* [S][cap], or NULL with cap 0 */
    int cap;
    const int* length;       /* [S] */
    const int* prompt;       /* [S] or NULL */
    const float* repetition; /* [S] or NULL */
    const float* frequency;  /* [S] or NULL */
    const float* presence;   /* [S] or NULL */
    const int* bias_ids;     /* [S][n_bias], or NULL with n_bias 0 */
    const float* bias;
    int n_bias;
} w4_logit_rules;
w4_status w4_logits_adjust(const w4_logit_rules* u, const void* logits, int type, long long ld, int R, const int* row_start,
                           const int* drafts, const unsigned long long* mask, const unsigned* allowed, void* out,
                           long long ld_out, unsigned flags, w4_stream_t s);

/* ------------------------------------------------------------------------
 * A chain of per-row INT4 decode linears in one launch (a decode step's
 * linear set).  Linear i computes exactly what w4a8_linear computes for
 * descs[i]; linear i+1 reads its x only after every output of linear i is
 * written, so descs[i+1].x may alias (part of) descs[i].y.  While a linear's
 * activations wait on that dependency, the weights of the following linears
 * keep streaming (one persistent block per SM, cooperative launch).
 *
 * descs: HOST array of n (1..W4_MAX_CHAIN) descriptors, all with the same
 * M tokens.  Per descriptor: w (repacked W4, 16-B aligned), s_w [N], bias [N]
 * or NULL, x [M][K] (16-B aligned), y [M][N], and qx [M][K] / sx [M] to
 * receive the activation codes, or NULL.
 * workspace: device memory of w4_chain_workspace_bytes() bytes, 16-B aligned,
 * zero-filled before its first use; each call leaves it zero again, ready for
 * the next.  Calls that share a workspace must not overlap on the GPU.  After
 * a call that reported W4_ERR_DEVICE_TIMEOUT, zero the workspace again.
 * Host threads may call the chain entry points at the same time, each with
 * its own workspace and stream: the launch parameters are staged per thread.
 * The chain runs its linears on DP4A whatever M is.  Per-row INT4 calls of
 * three or more tokens are faster through the per-linear entry points
 * (w4a8_linear with W4_FLAG_PDL, on the tensor cores), which need the qx / sx
 * buffers the chain may leave out.  On the 7B step the per-linear launches
 * chained with W4_FLAG_PDL are also faster at one token (0.872 against
 * 1.03-1.07 ms); the chain is the single-launch alternative. 
 * ------------------------------------------------------------------------ */
#define W4_MAX_CHAIN 128
typedef struct {
    const void* w;
    const float* s_w;
    const float* bias;
    const float* x;
    float* y;
    int8_t* qx;
    float* sx;
    int N;
    int K;
} w4_linear_desc;

size_t w4_chain_workspace_bytes(void);
w4_status w4a8_linear_chain(const w4_linear_desc* descs, int n, int M, void* workspace, size_t ws_bytes,
                            w4_stream_t s);

/* ------------------------------------------------------------------------
 * w4a8_linear_chain without caller-provided device memory.  The source pages
 * have no counterpart of this entry point: it exists for callers that cannot
 * allocate device memory at the point of the call -- for example code running
 * under an engine whose memory planner owns every device allocation, or code
 * that must not call cudaMalloc while a stream is being captured into a CUDA
 * graph -- and therefore cannot provide the chain's workspace.
 *
 * The grid-barrier state lives in a fixed array of
 * w4_chain_noalloc_scratch_bytes() (256) bytes inside the library; every GPU
 * that loads the library holds it until the process exits.  Each call clears
 * it (cudaMemsetAsync on `s`) and then runs exactly w4a8_linear_chain.  The
 * call allocates nothing and frees nothing.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress); make that first call before any stream capture.
 *   - All calls share the one array: calls that overlap on the GPU (other
 *     streams, other threads) race on it and must be serialised by the caller.
 *   - A workspace need above the array's size is rejected with
 *     W4_ERR_UNSUPPORTED_SHAPE; all other arguments are checked as in
 *     w4a8_linear_chain, before anything is enqueued: a call that fails a
 *     check does not touch the array (no clear), so it cannot disturb a
 *     chain already in flight.
 * ------------------------------------------------------------------------ */
size_t w4_chain_noalloc_scratch_bytes(void);
w4_status w4a8_linear_chain_noalloc(const w4_linear_desc* descs, int n, int M, w4_stream_t s);

/* ------------------------------------------------------------------------
 * Device error word.  Kernels that give up a bounded wait (about 0.25 s on an
 * mbarrier) record a nonzero code here and return early; their outputs are
 * then undefined.  w4_device_error synchronises the current device, reads the
 * word into *code (host pointer) and returns W4_ERR_DEVICE_TIMEOUT if it is
 * nonzero, else W4_OK.  w4_clear_device_error zeroes it (synchronous).
 * ------------------------------------------------------------------------ */
w4_status w4_device_error(unsigned* code);
w4_status w4_last_device_error(unsigned* code); /* the same call under a second name */
w4_status w4_clear_device_error(void);

/* Self-test of the timeout path: launches a kernel whose bounded wait nothing
 * completes (an mbarrier on which no thread arrives), so it gives up after
 * timeout_us microseconds (1..1000000) and sets the device error word to the
 * wait-timeout code (0x57414954, "WAIT"), as a GEMV's waits do.  cluster = 1
 * waits as the K-split leader does (two blocks in a cluster, cluster-scope
 * acquire, the other block leaving); 0 waits as every other ring does.  The
 * kernel always finishes and faults nothing; clear the word afterwards.
 * W4_ERR_INVALID_ARG for other arguments. */
w4_status w4_selftest_wait_timeout(int cluster, unsigned timeout_us, w4_stream_t s);

/* ------------------------------------------------------------------------
 * Pure-read HBM bandwidth probe: the roofline denominator for a kernel that
 * only reads.  [310B-Gemma4] §4.1 measures the device's pure read bandwidth
 * (distinct from a read+write copy) as the bound of a weight-streaming decode;
 * this is the same measurement on this device.  The kernel streams `bytes`
 * bytes of `buf` (16-byte aligned; bytes a multiple of 16) once through the
 * same per-warp bulk-copy rings as the GEMVs (one block per SM, evict-first)
 * and writes the XOR of all its 32-bit words to *sink (device, 4 bytes), so
 * that no read is dead.  bytes = 0 writes 0.  Time it with events on `s`.
 * ------------------------------------------------------------------------ */
w4_status w4_hbm_read(const void* buf, size_t bytes, unsigned* sink, w4_stream_t s);

#ifdef __cplusplus
}
#endif

#endif /* W4A8_H */
