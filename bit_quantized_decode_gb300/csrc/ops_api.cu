// C ABI of the INT8 x INT8 linear and the mixture-of-experts layer (declared
// in include/w4a8.h): argument checks, launch plan and dispatch.  No entry point allocates memory or
// synchronises.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/w4a8.h"
#include "operators.h"

using namespace w4k;

static_assert(W4_FMT_W8 == FMT_W8F && W4_FMT_W4 == FMT_W4, "public format codes");
static_assert(W4_MAX_EXPERTS == kMxMaxExperts && W4_MAX_TOP_K + W4_MAX_SHARED == kMxMaxSlots, "public limits");
static_assert(W4_F32 == T_F32 && W4_F16 == T_F16 && W4_BF16 == T_BF16, "public element types");

namespace {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline w4_status cuda_status(cudaError_t e) { return e == cudaSuccess ? W4_OK : W4_ERR_CUDA; }
inline bool elem_type(int t) { return t == W4_F32 || t == W4_F16 || t == W4_BF16; }

// Tokens that the fp16 codes of a call may take: M, and up to a tile's padding.
inline size_t padded_tokens(int M)
{
    return M <= 16 ? 16 : static_cast<size_t>(M) + kP8MaxTok;
}

w4_status check_w8_shape(int M, int N, int K)
{
    if (M < 0 || N < 0 || K <= 0) return W4_ERR_INVALID_ARG;
    if (K % 32 != 0 || K > W4_MAX_K || M > W4_MAX_TOKENS || N > (1 << 30) - 8) return W4_ERR_UNSUPPORTED_SHAPE;
    const long long tiles = static_cast<long long>((N + kG8Rows - 1) / kG8Rows) * ((M + 15) / 16);
    return tiles > (1 << 30) ? W4_ERR_UNSUPPORTED_SHAPE : W4_OK;
}

// Tiles of an M x N x K product: 128 rows by up to 128 tokens to a block, with
// K splits where tiles are few, or 256 rows by up to 192 tokens to a pair of
// blocks.  A stage of either takes about the same time (4096 tokens, 37888 x
// 3584: 868 us with blocks, 730 with pairs), so the one with fewer rounds of
// tiles over the SMs is taken.
bool plan_gemm8(const DeviceFacts& d, Gemm8Args& a, bool& pairs, int& grid, size_t& smem)
{
    auto tile = [&](int most, int step) {
        const int n = (a.M + most - 1) / most;
        return ((a.M + n - 1) / n + step - 1) / step * step;
    };
    a.C = a.K / 32;
    a.T = (a.N + kRows - 1) / kRows;
    const int nst = (a.C + kG8StageChunks - 1) / kG8StageChunks;
    int nt1 = tile(kG8MaxTok, 16);
    const int nt2 = tile(kP8MaxTok, 32);
    // several token tiles in one round: as many as there are SMs for
    const int n_g = (a.N + kG8Rows - 1) / kG8Rows;
    if (a.M > kG8MaxTok && n_g * ((a.M + nt1 - 1) / nt1) <= d.sms) {
        const int n = d.sms / n_g;
        const int nt = ((a.M + n - 1) / n + 15) / 16 * 16;
        if (nt >= 32 && nt < nt1) nt1 = nt;
    }
    const long long tiles1 = static_cast<long long>((a.N + kG8Rows - 1) / kG8Rows) * ((a.M + nt1 - 1) / nt1);
    const long long tiles2 = static_cast<long long>((a.N + 2 * kG8Rows - 1) / (2 * kG8Rows)) * ((a.M + nt2 - 1) / nt2);
    const int npairs = d.sms / 2;
    pairs = a.M > kG8MaxTok && npairs > 0 && (tiles2 + npairs - 1) / npairs < (tiles1 + d.sms - 1) / d.sms;
    a.splits = 1;
    if (pairs) {
        a.nt = nt2 / 2;
        a.n_g = (a.N + 2 * kG8Rows - 1) / (2 * kG8Rows);
        a.n_tt = (a.M + nt2 - 1) / nt2;
        a.stages = kP8MaxStages;
        while (a.stages > 2 && pair8_smem(a.stages, a.nt).total > d.smem_optin) --a.stages;
        smem = static_cast<size_t>(pair8_smem(a.stages, a.nt).total);
        grid = 2 * (tiles2 < npairs ? static_cast<int>(tiles2) : npairs);
    } else {
        a.nt = nt1;
        a.n_g = (a.N + kG8Rows - 1) / kG8Rows;
        a.n_tt = (a.M + nt1 - 1) / nt1;
        while (a.splits < kG8MaxSplit && tiles1 * 2 * a.splits <= d.sms && nst >= 4 * a.splits) a.splits *= 2;
        a.stages = gemm8_max_stages(a.nt) < kG8MaxStages ? gemm8_max_stages(a.nt) : kG8MaxStages;
        while (a.stages > 2 && gemm8_smem(a.stages, a.nt, a.splits).total > d.smem_optin) --a.stages;
        smem = static_cast<size_t>(gemm8_smem(a.stages, a.nt, a.splits).total);
        grid = a.splits > 1 ? static_cast<int>(tiles1) * a.splits : tiles1 < d.sms ? static_cast<int>(tiles1) : d.sms;
    }
    return smem <= static_cast<size_t>(d.smem_optin);
}

// The plan of a product: its tile arguments are needed before the codes are laid out.
struct Gemm8Plan {
    Gemm8Args a = {};
    bool pairs = false;
    int grid = 0;
    size_t smem = 0;
    bool make(const DeviceFacts& d, int M, int N, int K)
    {
        a.M = M;
        a.N = N;
        a.K = K;
        a.err = d.err;
        return plan_gemm8(d, a, pairs, grid, smem);
    }
};

// A product of up to eight tokens that the DP4A kernel takes; false where the
// codes leave no room for its rings.
bool plan_gemv8(const DeviceFacts& d, Gemv8Args& a, int& grid, size_t& smem)
{
    if (a.M > kV8MaxTok) return false;
    a.slot = 8192;
    while (a.slot > 4096 && gemv8_smem(a.slot, a.M, a.K) > d.smem_optin) a.slot /= 2;
    smem = static_cast<size_t>(gemv8_smem(a.slot, a.M, a.K));
    if (smem > static_cast<size_t>(d.smem_optin)) return false;
    // warps to a tile: as many as there are warps for, each with 1024 K or more
    const int T = (a.N + 7) / 8, C = a.K / 32;
    a.share = 1;
    while (a.share < 4 && 2 * a.share * static_cast<long long>(T) <= static_cast<long long>(d.sms) * kV8Warps && C >= 64 * a.share)
        a.share *= 2;
    grid = T < d.sms ? T : d.sms;
    return true;
}

w4_status run_gemm8(Gemm8Plan& p, const void* w, const float* s_w, const float* bias, const uint4* xh, const float* sx,
                    const float* residual, void* y, int y_type, cudaStream_t s)
{
    p.a.w = static_cast<const uint8_t*>(w);
    p.a.s_w = s_w;
    p.a.bias = bias;
    p.a.xh = xh;
    p.a.sx = sx;
    p.a.residual = residual;
    p.a.y = y;
    p.a.ytype = y_type;
    return cuda_status(p.pairs ? launch_gemm_w8_pair(p.a, p.grid, p.smem, true, s) : launch_gemm_w8(p.a, p.grid, p.smem, true, s));
}

w4_status check_w8_operands(const void* w, const float* s_w, const float* bias, const void* y, int y_type)
{
    if (!w || !s_w || !y) return W4_ERR_INVALID_ARG;
    if (!aligned(w, 16) || !aligned(s_w, 4) || (bias && !aligned(bias, 4)) ||
        !aligned(y, static_cast<size_t>(elem_bytes(y_type))))
        return W4_ERR_MISALIGNED;
    return W4_OK;
}

// ------------------------------------------------------ mixture of experts
w4_status check_router(const w4_router* r, int M, int K)
{
    if (!r || M < 0 || K <= 0) return W4_ERR_INVALID_ARG;
    if (r->E < 1 || r->top_k < 1 || (r->score != W4_ROUTE_SOFTMAX && r->score != W4_ROUTE_SIGMOID)) return W4_ERR_INVALID_ARG;
    if (r->select_bias != nullptr && r->score != W4_ROUTE_SIGMOID) return W4_ERR_INVALID_ARG;
    if (r->norm_weight != nullptr && (!(r->norm_eps > 0.0f) || !(r->norm_eps < 3.0e38f))) return W4_ERR_INVALID_ARG;
    if (r->top_k > r->E) return W4_ERR_INVALID_ARG;
    if (r->E > W4_MAX_EXPERTS || r->top_k > W4_MAX_TOP_K || M > W4_MAX_M || K % 32 != 0 || K > W4_MAX_K)
        return W4_ERR_UNSUPPORTED_SHAPE;
    return W4_OK;
}

// Blocks per cluster, tokens per cluster and warps per expert.  A token's
// logits spread over a cluster of 16 blocks up to eight tokens; more tokens take
// clusters of 8, all of which run at once.  256 experts of 1536, softmax scores,
// us in graph replays: 9 tokens 13.4 (clusters of 16: 10.3), 12 tokens 13.5
// (10.4), 16 tokens 14.4 (17.4); 64 experts of 3584: 9 tokens 9.9 (9.6), 16
// tokens 10.7 (14.6).  As few tokens to a cluster as two blocks per SM allow.
bool plan_route(const DeviceFacts& d, RouteArgs& a)
{
    const int most = a.M <= 8 ? kRtMaxCluster : 8;
    a.cluster = 1;
    while (a.cluster < most && 2 * a.cluster <= a.E) a.cluster *= 2;
    a.tok = 1;
    while (a.tok < kRtMaxTok && (a.M + a.tok - 1) / a.tok * a.cluster > 2 * d.sms) a.tok *= 2;
    while (a.tok > 1 && route_smem(a.tok, a.K, a.E) > d.smem_optin) a.tok /= 2;
    if (route_smem(a.tok, a.K, a.E) > d.smem_optin) return false;
    a.parts = 1;
    while (a.parts < kRtWarps && kRtWarps / (2 * a.parts) * a.cluster >= a.E) a.parts *= 2;
    return true;
}

w4_status run_route(const w4_router* r, const void* x, int x_type, int M, int K, int* ids, float* weights, int8_t* qx,
                    float* sx, const MoeFill& fill, bool pdl, cudaStream_t s)
{
    DeviceFacts d;
    if (!device_facts(&d)) return W4_ERR_CUDA;
    RouteArgs a = {};
    a.x = x;
    a.gamma = r->norm_weight;
    a.eps = r->norm_weight != nullptr ? r->norm_eps : 0.0f;
    a.w = r->w;
    a.sel = r->select_bias;
    a.E = r->E;
    a.top_k = r->top_k;
    a.sigmoid = r->score == W4_ROUTE_SIGMOID;
    a.renorm = r->renormalize != 0;
    a.scale = r->scale;
    a.M = M;
    a.K = K;
    a.ids = ids;
    a.weights = weights;
    a.qx = qx;
    a.sx = sx;
    a.fill = fill;
    if (!plan_route(d, a)) return W4_ERR_UNSUPPORTED_SHAPE;
    return cuda_status(launch_moe_route(a, x_type, pdl, s));
}

// Pointers of a router call (after check_router).
w4_status check_route_pointers(const w4_router* r, const void* x, const int* ids, const float* weights,
                               const int8_t* qx, const float* sx)
{
    if (!r->w || !x || !ids || !weights || (qx == nullptr) != (sx == nullptr)) return W4_ERR_INVALID_ARG;
    if (!aligned(r->w, 16) || !aligned(x, 16) || !aligned(ids, 4) || !aligned(weights, 4) || (qx && !aligned(qx, 16)) ||
        (sx && !aligned(sx, 4)) || (r->norm_weight && !aligned(r->norm_weight, 16)) ||
        (r->select_bias && !aligned(r->select_bias, 4)))
        return W4_ERR_MISALIGNED;
    return W4_OK;
}

w4_status check_experts(const w4_experts* e, int M, int top_k)
{
    if (!e || M < 0 || top_k < 1 || e->E < 1 || e->n_shared < 0 || e->H <= 0 || e->I <= 0) return W4_ERR_INVALID_ARG;
    if (e->fmt != W4_FMT_W4 && e->fmt != W4_FMT_W8) return W4_ERR_INVALID_ARG;
    if (e->glu != W4_GLU_SILU && e->glu != W4_GLU_GELU_TANH) return W4_ERR_INVALID_ARG;
    if (M > W4_MAX_M || top_k > W4_MAX_TOP_K || e->n_shared > W4_MAX_SHARED || e->E > W4_MAX_EXPERTS - e->n_shared ||
        e->H % 32 != 0 || e->I % 32 != 0 || e->H > W4_MAX_K || e->I > W4_MAX_K)
        return W4_ERR_UNSUPPORTED_SHAPE;
    return W4_OK;
}

w4_status check_expert_pointers(const w4_experts* e, const float* residual, const void* y, int y_type)
{
    if (!e->w_gu || !e->s_gu || !e->w_dn || !e->s_dn || !y) return W4_ERR_INVALID_ARG;
    if (!aligned(e->w_gu, 16) || !aligned(e->w_dn, 16) || !aligned(e->s_gu, 4) || !aligned(e->s_dn, 4) ||
        (e->b_gu && !aligned(e->b_gu, 4)) || (e->b_dn && !aligned(e->b_dn, 4)) || (residual && !aligned(residual, 4)) ||
        !aligned(y, static_cast<size_t>(elem_bytes(y_type))))
        return W4_ERR_MISALIGNED;
    return W4_OK;
}

// Parts of the workspace: the ticket counter, then (prepared) h, the slots'
// outputs and the quantizing tasks' results, then the codes of h.
struct MoeSpace {
    size_t h, part, qdone, qh, total;
};
MoeSpace moe_space(const w4_experts* e, int M, int top_k)
{
    const size_t P = static_cast<size_t>(M) * (top_k + e->n_shared);
    const size_t nseg = static_cast<size_t>((e->I + kMxSeg - 1) / kMxSeg);
    MoeSpace w;
    w.h = kMxHead * 4;
    w.part = w.h + P * e->I * 4;
    w.qdone = w.part + P * e->H * 4;
    w.qh = w.qdone + (P * nseg * 8 + 127) / 128 * 128;
    w.total = w.qh + P * e->I * (e->fmt == W4_FMT_W4 ? 2 : 1);       // (INT4 on the tensor cores: as fp16)
    return w;
}
MoeFill moe_fill_of(const MoeSpace& w, void* ws)
{
    return MoeFill{static_cast<uint4*>(ws), static_cast<unsigned>((w.qh - kMxHead * 4) / 16)};
}

// Pairs per entry (an expert and some of its tokens, whose weights are read
// once).  Where an expert that is reached at all has one token as a rule, the
// DP4A entries of two are ahead, elsewhere the tensor cores' eight.  64 experts
// of 2368 x 3584 in INT4, top 8: 6 tokens (1.36 tokens per expert) 101 us by
// two, 108 by eight; 8 tokens (1.52) 129 and 123, 16 tokens 213 and 178.  128
// experts of 768 x 1536 and a shared one in INT8, top 6: 5 tokens (1.25) 38 us
// by two, 47 by eight; 12 tokens (1.47) 63 and 55.
int moe_entry_pairs(const DeviceFacts& d, const w4_experts* e, int M, int top_k, MoePlan& p)
{
    const size_t most = static_cast<size_t>(d.smem_optin);
    if (M > 2) {
        const double reached = e->E * (1.0 - pow(1.0 - static_cast<double>(top_k < e->E ? top_k : e->E) / e->E, M)) + e->n_shared;
        if (static_cast<double>(M) * (top_k + e->n_shared) > 1.4 * reached) {
            p = moe_plan(e->fmt, kMxTok, M, e->H, most);
            if (p.fits) return kMxTok;
        }
    }
    const int tok = M <= 1 ? 1 : 2;
    p = moe_plan(e->fmt, tok, M, e->H, most);
    return tok;
}

w4_status run_experts(const w4_experts* e, const int8_t* qx, const float* sx, const int* ids, const float* weights, int M,
                      int top_k, const float* residual, void* y, int y_type, void* ws, cudaStream_t s)
{
    DeviceFacts d;
    if (!device_facts(&d)) return W4_ERR_CUDA;
    const MoeSpace w = moe_space(e, M, top_k);
    uint8_t* base = static_cast<uint8_t*>(ws);
    MoeArgs a = {};
    a.w_gu = static_cast<const uint8_t*>(e->w_gu);
    a.w_dn = static_cast<const uint8_t*>(e->w_dn);
    a.s_gu = e->s_gu;
    a.b_gu = e->b_gu;
    a.s_dn = e->s_dn;
    a.b_dn = e->b_dn;
    a.qx = qx;
    a.sx = sx;
    a.ids = ids;
    a.weights = weights;
    a.residual = residual;
    a.y = y;
    a.ytype = y_type;
    a.glu = e->glu;
    a.M = M;
    a.H = e->H;
    a.I = e->I;
    a.E = e->E;
    a.S = e->n_shared;
    a.top_k = top_k;
    a.ticket = reinterpret_cast<unsigned*>(base);
    a.h = reinterpret_cast<float*>(base + w.h);
    a.part = reinterpret_cast<float*>(base + w.part);
    a.qdone = reinterpret_cast<unsigned long long*>(base + w.qdone);
    a.qh = reinterpret_cast<int8_t*>(base + w.qh);
    a.err = d.err;
    MoePlan plan;
    const int tok = moe_entry_pairs(d, e, M, top_k, plan);
    if (!plan.fits) return W4_ERR_UNSUPPORTED_SHAPE;
    a.inv_x16 = 16.0f / static_cast<float>(e->H);
    const int u = plan.tiles;
    const int u1 = ((e->I + 3) / 4 + u - 1) / u, u2 = ((e->H + 7) / 8 + u - 1) / u;
    a.inv_t1 = 1.0f / static_cast<float>(u1);
    a.inv_t2 = 1.0f / static_cast<float>(u2);
    a.inv_seg = 1.0f / static_cast<float>((e->I + kMxSeg - 1) / kMxSeg);
    a.inv_add = 1.0f / static_cast<float>((e->H + mx_add(tok) - 1) / mx_add(tok));
    a.stage_x = plan.staged;
    // every SM a share of the gate/up tiles: a ticket for each warp at the start
    // (or fewer), then a few at a time, two batches ahead (a batch takes a
    // microsecond to fetch, a ticket some ten to work off)
    const long long work = static_cast<long long>(M) * (top_k + e->n_shared) * u1;
    const int grid = work < d.sms ? static_cast<int>(work) : d.sms;
    const long long share = work / grid;
    a.batch0 = share < plan.warps ? static_cast<int>(share) : plan.warps;
    a.batch = share >= 8 ? 4 : share >= 4 ? 2 : 1;
    return cuda_status(launch_moe_experts(e->fmt, tok, a, grid, plan.warps, plan.smem, true, s));
}

}  // namespace

extern "C" {

size_t w8a8_workspace_bytes(int M, int N, int K)
{
    if (check_w8_shape(M, N, K) != W4_OK) return 0;
    return M > 0 ? padded_tokens(M) * K * 2 : 0;
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
    DeviceFacts d;
    if (!device_facts(&d)) return W4_ERR_CUDA;
    int grid = 0;
    size_t smem = 0;
    Gemv8Args v = {};
    v.M = M;
    v.N = N;
    v.K = K;
    if (plan_gemv8(d, v, grid, smem)) {
        v.w = static_cast<const uint8_t*>(w);
        v.s_w = s_w;
        v.bias = bias;
        v.qx_in = qx;
        v.sx_in = sx;
        v.y = y;
        v.ytype = y_type;
        v.err = d.err;
        return cuda_status(launch_gemv_w8(v, grid, smem, false, s));
    }
    uint4* xh = static_cast<uint4*>(workspace);
    Gemm8Plan p;
    if (!p.make(d, M, N, K)) return W4_ERR_UNSUPPORTED_SHAPE;
    r = cuda_status(launch_expand_codes(qx, M, K, xh, p.a.nt, false, s));
    if (r != W4_OK) return r;
    return run_gemm8(p, w, s_w, bias, xh, sx, nullptr, y, y_type, s);
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
    const bool pdl = (flags & W4_FLAG_PDL) != 0;
    DeviceFacts d;
    if (!device_facts(&d)) return W4_ERR_CUDA;
    int grid = 0;
    size_t smem = 0;
    Gemv8Args v = {};
    v.M = M;
    v.N = N;
    v.K = K;
    const bool few = N > 0 && plan_gemv8(d, v, grid, smem);
    if (few) {
        v.w = static_cast<const uint8_t*>(w);
        v.s_w = s_w;
        v.bias = bias;
        v.residual = residual;
        v.y = y;
        v.ytype = y_type;
        v.err = d.err;
        if (M == 1 || (M <= kV8FusedTok && M * K <= kV8FusedValues)) {
            v.x = x;
            v.xtype = x_type;
            v.gamma = gamma;
            v.eps = gamma != nullptr ? f->norm_eps : 0.0f;
            v.qx_out = qx;
            v.sx_out = sx;
            return cuda_status(launch_gemv_w8(v, grid, smem, pdl, s));
        }
        v.qx_in = qx != nullptr ? qx : static_cast<int8_t*>(workspace);
        v.sx_in = sx;
    }
    QuantRowsArgs q = {};
    q.x = x;
    q.gamma = gamma;
    q.eps = gamma != nullptr ? f->norm_eps : 0.0f;
    q.M = M;
    q.K = K;
    q.qx = few ? const_cast<int8_t*>(v.qx_in) : qx;
    q.sx = sx;
    q.xh = N > 0 && !few ? static_cast<uint4*>(workspace) : nullptr;
    Gemm8Plan p;
    if (q.xh != nullptr && !p.make(d, M, N, K)) return W4_ERR_UNSUPPORTED_SHAPE;
    q.nt = p.a.nt;
    r = cuda_status(launch_quant_rows(q, x_type, pdl, s));
    if (r != W4_OK || N == 0) return r;
    if (few) return cuda_status(launch_gemv_w8(v, grid, smem, true, s));
    return run_gemm8(p, w, s_w, bias, q.xh, sx, residual, y, y_type, s);
}

w4_status w4_moe_route(const w4_router* r, const void* x, int x_type, int M, int K, int* ids, float* weights,
                       int8_t* qx, float* sx, unsigned flags, w4_stream_t s)
{
    w4_status st = check_router(r, M, K);
    if (st != W4_OK) return st;
    if (!elem_type(x_type) || (flags & ~W4_FLAG_PDL) != 0) return W4_ERR_INVALID_ARG;
    if (M == 0) return W4_OK;
    st = check_route_pointers(r, x, ids, weights, qx, sx);
    if (st != W4_OK) return st;
    return run_route(r, x, x_type, M, K, ids, weights, qx, sx, MoeFill{}, (flags & W4_FLAG_PDL) != 0,
                     reinterpret_cast<cudaStream_t>(s));
}

size_t w4_moe_workspace_bytes(const w4_experts* e, int M, int top_k)
{
    if (check_experts(e, M, top_k) != W4_OK || M == 0) return 0;
    return moe_space(e, M, top_k).total;
}

w4_status w4_moe_experts(const w4_experts* e, const int8_t* qx, const float* sx, const int* ids,
                         const float* weights, int M, int top_k, const float* residual, void* y, int y_type,
                         void* workspace, size_t ws_bytes, unsigned flags, w4_stream_t st)
{
    w4_status r = check_experts(e, M, top_k);
    if (r != W4_OK) return r;
    if (!elem_type(y_type) || (flags & ~W4_FLAG_PDL) != 0) return W4_ERR_INVALID_ARG;
    if (M == 0) return W4_OK;
    r = check_expert_pointers(e, residual, y, y_type);
    if (r == W4_ERR_INVALID_ARG || !qx || !sx || !ids || !weights || !workspace) return W4_ERR_INVALID_ARG;
    if (ws_bytes < w4_moe_workspace_bytes(e, M, top_k)) return W4_ERR_UNSUPPORTED_SHAPE;
    if (r != W4_OK || !aligned(qx, 16) || !aligned(sx, 4) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(workspace, 16))
        return W4_ERR_MISALIGNED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(st);
    r = cuda_status(launch_moe_fill(moe_fill_of(moe_space(e, M, top_k), workspace), (flags & W4_FLAG_PDL) != 0, s));
    if (r != W4_OK) return r;
    return run_experts(e, qx, sx, ids, weights, M, top_k, residual, y, y_type, workspace, s);
}

w4_status w4_moe_layer(const w4_router* r, const w4_experts* e, const void* x, int x_type, int M, int* ids,
                       float* weights, int8_t* qx, float* sx, const float* residual, void* y, int y_type,
                       void* workspace, size_t ws_bytes, unsigned flags, w4_stream_t s)
{
    if (!r || !e) return W4_ERR_INVALID_ARG;
    w4_status st = check_router(r, M, e->H);
    if (st == W4_OK) st = check_experts(e, M, r->top_k);
    if (st != W4_OK) return st;
    if (r->E != e->E || !elem_type(x_type) || !elem_type(y_type) || (flags & ~W4_FLAG_PDL) != 0) return W4_ERR_INVALID_ARG;
    if (M == 0) return W4_OK;
    st = check_route_pointers(r, x, ids, weights, qx, sx);
    const w4_status se = check_expert_pointers(e, residual, y, y_type);
    if (st == W4_ERR_INVALID_ARG || se == W4_ERR_INVALID_ARG || !qx || !workspace) return W4_ERR_INVALID_ARG;
    if (ws_bytes < w4_moe_workspace_bytes(e, M, r->top_k)) return W4_ERR_UNSUPPORTED_SHAPE;
    if (st != W4_OK || se != W4_OK || !aligned(workspace, 16)) return W4_ERR_MISALIGNED;
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(s);
    st = run_route(r, x, x_type, M, e->H, ids, weights, qx, sx, moe_fill_of(moe_space(e, M, r->top_k), workspace),
                   (flags & W4_FLAG_PDL) != 0, cs);
    if (st != W4_OK) return st;
    return run_experts(e, qx, sx, ids, weights, M, r->top_k, residual, y, y_type, workspace, cs);
}

}  // extern "C"
