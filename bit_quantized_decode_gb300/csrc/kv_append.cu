// Cache append: RMSNorm of each query and key head, their rotation by
// position, and the way of keys and values into a paged cache, in one pass
// over the q/k/v projection's output.
//
//   x' = (x r) g, r = 1 / sqrt(fp32(sum x^2) / D + eps)         (q and k, optional)
//   a' = a c - b s, b' = b c + a s   over pairs of the first `rot` values
//   16-bit cache: rounded once; INT8: s = max|x'| / 127, q = clip(rint(x' / s)).
//
// D / 8 lanes take a head, eight values to a lane, pairs within a lane: a
// rotation needs no exchange, and a pair's (cos, sin) is read once for all heads of a warp.  A warp takes 4, 2 or
// 1 heads of a token at a time (D 64, 128, 256).  An INT8 code hangs on the last bit of a
// value, so a key for an INT8 cache is rotated with exact products and a compensated
// sum (rounded once), and its squares are summed in compensated pairs as in the other
// fused norms; numbers that are rounded to 16 bits take plain fp32 sums and rsqrtf
// (2^-20 of the value at most).  A few tokens are bound by the launch and the chain of
// loads (row's sequence and length, then page and rotation, beside the values): one token 2.2 us,
// 16 drafts to INT8 2.5.  Prompts (12,300 rows of 2560 bf16 values with norms to fp16, 136 MB): 45 us, 3.0 TB/s,
// without norms 37: the same chain at the start of each warp, then instructions (issue slots 57% taken).
#include "attention.h"
#include "fusion.cuh"
#include "ptx.cuh"
#include "typed_io.cuh"

namespace w4k {
namespace {

// Four consecutive fp32 values.
__device__ __forceinline__ void load4(const float* p, float* v)
{
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}

// Four values as they lie in memory, and widened.
template <int T>
struct Raw4 {
    uint2 v;
    __device__ __forceinline__ void load(const void* base, size_t at) { v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at)); }
    __device__ __forceinline__ void widen(float* f) const
    {
        const uint32_t w[2] = {v.x, v.y};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if constexpr (T == T_F16) {
                const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                f[2 * k] = h.x;
                f[2 * k + 1] = h.y;
            } else {                                          // bf16: the upper half of an fp32
                f[2 * k] = __uint_as_float(w[k] << 16);
                f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            }
        }
    }
};
template <>
struct Raw4<T_F32> {
    float4 v;
    __device__ __forceinline__ void load(const void* base, size_t at) { v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + at)); }
    __device__ __forceinline__ void widen(float* f) const { f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w; }
};

__device__ __forceinline__ uint32_t pack16(int type, float a, float b)
{
    if (type == T_F16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// a c + b d rounded once (but for sums within some 2^-46 of a rounding boundary).
__device__ __forceinline__ float dot2_once(float a, float c, float b, float d)
{
    const float p = __fmul_rn(a, c), pe = __fmaf_rn(a, c, -p);
    const float q = __fmul_rn(b, d), qe = __fmaf_rn(b, d, -q);
    float s, e;
    two_sum(p, q, s, e);
    return __fadd_rn(s, __fadd_rn(e, __fadd_rn(pe, qe)));
}

__device__ __forceinline__ float max_or_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Blocks to an SM that the registers leave room for: 80 a thread of fp32 values (90 without the bound: 12,300 rows of 36 heads of
// 128 71 -> 77 us), 72 of 16-bit ones.
template <int XT, int D>
constexpr int kv_blocks() { return XT != T_F32 ? 7 : D == 256 ? 5 : 6; }

template <int XT, int D>
__global__ void __launch_bounds__(kKaThreads, kv_blocks<XT, D>()) kv_append_kernel(const AppendArgs A)
{
    constexpr int kLanes = D / 8;               // lanes of a head
    constexpr int kHeads = 32 / kLanes;         // heads of a warp
    const int lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    const int H = A.Hq + 2 * A.c.Hkv;
    const int groups = (H + kHeads - 1) / kHeads;             // warps' loads of a token's heads
    const int parts = (groups + A.per - 1) / A.per;           // warps of a token
    const long long task = (static_cast<long long>(blockIdx.x) * kKaThreads + threadIdx.x) >> 5;
    if (task >= static_cast<long long>(A.T) * parts) return;
    const int t = static_cast<int>(task / parts);
    const int g0 = static_cast<int>(task - static_cast<long long>(t) * parts) * A.per, g1 = min(g0 + A.per, groups);
    const int u = lane % kLanes;                // eight values of the head

    // A lane's eight values are two fours, half of a part of the head apart (the rotated part, the rest, or a value head's
    // whole), so that lanes beside each other read and write beside each other: whole sectors in every access.  In the half
    // layout the second four are the partners of the first; interleaved pairs lie within a four.
    const int rotated = A.Hq + A.c.Hkv;
    const bool turns = 8 * u < A.rot;           // (this lane's values of a query or key head)
    const int at0 = turns ? 4 * u : A.rot / 2 + 4 * u, at1 = at0 + (turns ? A.rot : D - A.rot) / 2;
    const size_t row0 = static_cast<size_t>(t) * A.ld, row = row0 + (lane / kLanes) * D;
    constexpr int kAhead = 2;                   // heads whose loads are in flight
    Raw4<XT> lo[kAhead], hi[kAhead];
    auto load = [&](int g) {
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            const int head = (g + e) * kHeads + lane / kLanes;
            if (g + e < g1) {
                const size_t base = head < H ? row + (g + e) * (kHeads * D) : row0;   // (lanes without a head read the first one's)
                const bool plain = head >= rotated;
                lo[e].load(A.x, base + (plain ? 4 * u : at0));
                hi[e].load(A.x, base + (plain ? D / 2 + 4 * u : at1));
            }
        }
    };
    load(g0);

    // the row's sequence: with up to 32 of them everything about them is asked for at once (a round of loads is a third of a
    // few tokens' time)
    const int told = A.pos != nullptr ? __ldg(A.pos + t) : 0;
    int b, i, before;
    if (A.b.B <= 32) {
        const bool is = lane < A.b.B;
        const int q0 = is ? __ldg(A.b.q_start + lane) : 0, q1 = is ? __ldg(A.b.q_start + lane + 1) : 0;
        before = is ? __ldg(A.b.ctx + lane) : 0;
        b = __popc(__ballot_sync(0xffffffffu, is && q1 <= t));
        i = t - __shfl_sync(0xffffffffu, q0, b & 31);
        before = __shfl_sync(0xffffffffu, before, b & 31);
    } else {
        b = row_sequence(A.b.q_start, A.b.B, t, lane);
        i = b < A.b.B ? t - __ldg(A.b.q_start + b) : 0;
        before = b < A.b.B ? __ldg(A.b.ctx + b) : 0;
    }
    if (b >= A.b.B || i < 0) return;            // behind the last sequence
    const long long place = static_cast<long long>(max(before, 0)) + i;
    const bool i8 = A.c.type == T_I8;
    float cs[8];                                // (cos, sin) of this lane's four pairs
    if (A.rot > 0) {
        const long long p = A.pos != nullptr ? told : place;
        const bool lost = p < 0 || p >= A.positions;              // a position that the table does not have
        if (turns) {
            const float* cp = A.turns + static_cast<size_t>(lost ? 0 : p) * A.rot;
            load4(cp + (A.interleaved ? 4 * u : 8 * u), cs);
            load4(cp + (A.interleaved ? A.rot / 2 + 4 * u : 8 * u + 4), cs + 4);
            if (lost)
#pragma unroll
                for (int k = 0; k < 8; k += 2) cs[k] = __int_as_float(0x7fc00000);
        }
    }
    // the page; a place past the table, or a page that the cache does not have, is not written
    const long long pi = place >> A.c.lg;
    const int page = pi < A.b.max_pages ? __ldg(A.b.table + static_cast<size_t>(b) * A.b.max_pages + pi) : -1;
    const bool stored = page >= 0 && page < A.c.pages;
    const size_t slot0 = static_cast<size_t>(stored ? page : 0) * A.c.Hkv * A.c.page + static_cast<size_t>(place & (A.c.page - 1));

    const bool normed = A.q_norm != nullptr || A.k_norm != nullptr;
    const float* w_of = nullptr;                // the norm weights at hand
    float w[8];
    uint16_t* const q_row = static_cast<uint16_t*>(A.q) + static_cast<size_t>(t) * A.Hq * D;
    auto one = [&](int g, const Raw4<XT>& l, const Raw4<XT>& h4) {
        float x[8];
        l.widen(x);
        h4.widen(x + 4);
        const int head = g * kHeads + lane / kLanes;
        const bool have = head < H, is_q = head < A.Hq, is_k = !is_q && head < rotated;
        // codes hang on the last bit of an INT8 cache's keys; what is rounded to 16 bits takes plain fp32 sums
        const bool coded = i8 && g * kHeads < rotated && (g + 1) * kHeads > A.Hq;     // (of the whole warp)
        if (normed && g * kHeads < rotated) {
            const float* const w_n = is_q ? A.q_norm : is_k ? A.k_norm : nullptr;
            if (w_n != w_of && w_n != nullptr) {
                w_of = w_n;
                load4(w_n + at0, w);
                load4(w_n + at1, w + 4);
            }
            float r;
            if (coded) {
                float sh = 0.0f, sl = 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k) sq_acc(x[k], sh, sl);
#pragma unroll
                for (int off = kLanes / 2; off > 0; off >>= 1) {
                    const float h2 = __shfl_xor_sync(0xffffffffu, sh, off), l2 = __shfl_xor_sync(0xffffffffu, sl, off);
                    pair_merge(sh, sl, h2, l2);
                }
                sh = __shfl_sync(0xffffffffu, sh, lane - u);  // (the same sum in every lane of the head)
                sl = __shfl_sync(0xffffffffu, sl, lane - u);
                r = rms_scale(sh, sl, D, A.eps);
            } else {
                float sum = 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k) sum = __fmaf_rn(x[k], x[k], sum);
#pragma unroll
                for (int off = kLanes / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                r = rsqrtf(__fmaf_rn(sum, 1.0f / D, A.eps));
            }
            if (w_n != nullptr) {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = __fmul_rn(__fmul_rn(x[k], r), w[k]);
            }
        }
        if (turns && head < rotated) {
            auto turn = [&](float& a, float& v, float c, float s) {
                const float p = a, q = v;
                if (coded) {
                    a = dot2_once(p, c, -q, s);
                    v = dot2_once(q, c, p, s);
                } else {
                    a = __fmaf_rn(p, c, -__fmul_rn(q, s));
                    v = __fmaf_rn(q, c, __fmul_rn(p, s));
                }
            };
            if (A.interleaved) {
#pragma unroll
                for (int k = 0; k < 4; ++k) turn(x[2 * k], x[2 * k + 1], cs[2 * k], cs[2 * k + 1]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) turn(x[k], x[4 + k], cs[2 * k], cs[2 * k + 1]);
            }
        }
        const bool plain = head >= rotated;
        const int o0 = plain ? 4 * u : at0, o1 = plain ? D / 2 + 4 * u : at1;
        const int hk = is_k ? head - A.Hq : head - rotated;
        const size_t slot = slot0 + static_cast<size_t>(is_q || !have ? 0 : hk) * A.c.page;
        const bool store = have && !is_q && stored;
        if (is_q || (store && !i8)) {
            uint16_t* d = is_q ? q_row + head * D : static_cast<uint16_t*>(is_k ? A.c.k : A.c.v) + slot * D;
            uint4 h;
            if ((is_q ? A.qtype : A.c.type) == T_F16)
                h = make_uint4(pack16(T_F16, x[0], x[1]), pack16(T_F16, x[2], x[3]), pack16(T_F16, x[4], x[5]), pack16(T_F16, x[6], x[7]));
            else
                h = make_uint4(pack16(T_BF16, x[0], x[1]), pack16(T_BF16, x[2], x[3]), pack16(T_BF16, x[4], x[5]), pack16(T_BF16, x[6], x[7]));
            *reinterpret_cast<uint2*>(d + o0) = make_uint2(h.x, h.y);
            *reinterpret_cast<uint2*>(d + o1) = make_uint2(h.z, h.w);
        }
        if (!i8 || (g + 1) * kHeads <= A.Hq) return;          // (of the whole warp)
        float top = 0.0f;                       // (a NaN stays one: of the head's values, and of a position the table does not have)
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max_or_nan(top, fabsf(x[k]));
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) top = max_or_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
        if (store) {
            const A8Scale ks = a8_scale(top);
            uint2 q = quant8(x, ks);
            const bool nan = top != top;        // codes of 0 with the scale NaN
            if (nan) q = make_uint2(0u, 0u);
            int8_t* d = static_cast<int8_t*>(is_k ? A.c.k : A.c.v) + slot * D;
            *reinterpret_cast<uint32_t*>(d + o0) = q.x;
            *reinterpret_cast<uint32_t*>(d + o1) = q.y;
            if (u == 0) (is_k ? A.c.ks : A.c.vs)[slot] = nan ? __int_as_float(0x7fc00000) : ks.s;
        }
        __syncwarp();
    };
#pragma unroll 1
    for (int g = g0; g < g1; g += kAhead) {
        if (g > g0) load(g);
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
            if (g + e < g1) one(g + e, lo[e], hi[e]);
    }
}

template <int XT, int D>
cudaError_t launch(AppendArgs& a, cudaStream_t s)
{
    // Few tokens: a warp for every load of heads.  Many: a warp takes more of a token's heads (the token's lookups once),
    // as long as the SMs keep some 32 warps each.
    constexpr int kHeads = 32 / (D / 8), kWarps = 152 * 32;
    const long long groups = (a.Hq + 2 * a.c.Hkv + kHeads - 1) / kHeads;
    const long long per = static_cast<long long>(a.T) * groups / kWarps;
    a.per = static_cast<int>(per < 1 ? 1 : per < groups ? per : groups);
    const long long tasks = static_cast<long long>(a.T) * ((groups + a.per - 1) / a.per);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((tasks * 32 + kKaThreads - 1) / kKaThreads));
    cfg.blockDim = dim3(kKaThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_append_kernel<XT, D>, a);
}

template <int XT>
cudaError_t launch_d(AppendArgs& a, cudaStream_t s)
{
    return a.c.D == 64 ? launch<XT, 64>(a, s) : a.c.D == 128 ? launch<XT, 128>(a, s) : launch<XT, 256>(a, s);
}

// (cos, sin) of position * factor * inv_freq, times scale: angles of far positions
// need the product and its reduction in 64 bits; each number is rounded once.
__global__ void rope_table_kernel(const double* inv_freq, double factor, double scale, long long n, int half, float2* turns)
{
    const long long e = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (e >= n) return;
    const long long p = e / half;
    double s, c;
    sincos(static_cast<double>(p) * factor * inv_freq[e - p * half], &s, &c);
    turns[e] = make_float2(static_cast<float>(c * scale), static_cast<float>(s * scale));
}

// An INT8 cache's codes times their scales, eight to a thread.
__global__ void __launch_bounds__(256) kv_values_kernel(const int8_t* codes, const float* scale, long long words, int lg_words, float* out)
{
    pdl_launch_dependents();
    pdl_wait();
    const long long w = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (w >= words) return;
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(codes) + w);
    const float s = __ldg(scale + (w >> lg_words));
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __fmul_rn(static_cast<float>(static_cast<int8_t>((k < 4 ? q.x : q.y) >> (8 * (k & 3)))), s);
    float4* d = reinterpret_cast<float4*>(out) + 2 * w;
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
}

}  // namespace

cudaError_t launch_kv_values(const KvView& c, bool values, float* out, cudaStream_t s)
{
    const int lg_words = c.D == 64 ? 3 : c.D == 128 ? 4 : 5;  // of eight codes, in a token
    const long long words = static_cast<long long>(c.pages) * c.Hkv * c.page << lg_words;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((words + 255) / 256));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_values_kernel, static_cast<const int8_t*>(values ? c.v : c.k),
                              static_cast<const float*>(values ? c.vs : c.ks), words, lg_words, out);
}

cudaError_t launch_kv_append(AppendArgs& a, int xtype, cudaStream_t s)
{
    return xtype == T_F32 ? launch_d<T_F32>(a, s) : xtype == T_F16 ? launch_d<T_F16>(a, s) : launch_d<T_BF16>(a, s);
}

cudaError_t launch_rope_table(const double* inv_freq, double factor, double scale, int positions, int half, float* turns,
                              cudaStream_t s)
{
    const long long n = static_cast<long long>(positions) * half;
    rope_table_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(inv_freq, factor, scale, n, half,
                                                                            reinterpret_cast<float2*>(turns));
    return cudaGetLastError();
}

}  // namespace w4k
