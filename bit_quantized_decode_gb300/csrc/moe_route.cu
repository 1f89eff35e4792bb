// Expert router of a mixture-of-experts layer for a few tokens: RMSNorm, the
// scores of E experts, the top_k of them and their weights, and the INT8 codes
// that the experts' kernel reads, in one launch.
//
//   x' = RMSNorm(x) (or x), l_e = fp32(sum_i x'_i w_ei),
//   softmax: the largest l;  p = softmax(l) over all experts;
//   sigmoid: the largest fp32(p_e + bias_e), p_e = fp32(1 / (1 + exp(-l_e)));
//   ties go to the lowest index; weight = p (/ the chosen experts' sum) * scale.
//
// A choice hangs on the last bit of a logit, so the sums are compensated
// (products split exactly by an FMA, error-free additions; about 2^-44 of the
// sum of magnitudes) and rounded once, and the sigmoid is evaluated in pairs
// of fp32 (exact_act.cuh).
//
// One thread-block cluster of up to 16 blocks serves up to four tokens: every
// block normalizes them (a few tens of KB from L2, cheaper than a second
// hop), its warps take experts (several warps to one where experts are few,
// each a share of K), the logits go to the cluster's first block through
// distributed shared memory, and one warp per token picks the experts there,
// while the last block writes the codes.  No global scratch, no flags; the
// launch is bound by latency (weights, two block barriers, one cluster
// barrier, top_k warp reductions).  One token over 64 experts of 3584: 7.8 us;
// 16 tokens over 256 experts of 1536: 14.4 us with softmax scores, 17.5 us with
// sigmoid ones (a token's 256 are evaluated by one warp, eight to a lane).
#include "exact_act.cuh"
#include "fusion.cuh"
#include "operators.h"
#include "ptx.cuh"
#include "quant_a8.cuh"
#include "typed_io.cuh"

namespace w4k {
namespace {

// (hi, lo) += a b, the product exact, the sum compensated.
__device__ __forceinline__ void dot_acc(float a, float b, float& hi, float& lo)
{
    const float p = __fmul_rn(a, b);
    const float pe = __fmaf_rn(a, b, -p);
    float s, e;
    two_sum(hi, p, s, e);
    hi = s;
    lo = __fadd_rn(lo, __fadd_rn(e, pe));
}

// Ascending unsigned order of floats; NaN below all, never 0.
__device__ __forceinline__ uint32_t order_key(float v)
{
    if (!(v == v)) return 1u;
    const uint32_t u = __float_as_uint(__fadd_rn(v, 0.0f));          // -0 as +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kRtAhead = 4;                     // float4 of router weights that a lane holds before the wait

template <int XT, int TG>
__global__ void __launch_bounds__(kRtThreads, 2) moe_route_kernel(const RouteArgs a)
{
    extern __shared__ __align__(16) float rsm[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cs = a.cluster;
    const int rank = static_cast<int>(blockIdx.x) % cs;
    const int m0 = static_cast<int>(blockIdx.x) / cs * TG;
    const int nt = min(TG, a.M - m0);
    const int K = a.K, K4 = K >> 2, K8 = K >> 3;
    const int Epad = (a.E + 3) & ~3;
    float* xs = rsm;                                      // [TG][K]
    float* part_s = xs + TG * K;                          // [warps][TG][2]
    float* key_s = part_s + kRtWarps * kRtMaxTok * 2;     // [TG][Epad], the leader's
    uint32_t* ord_s = reinterpret_cast<uint32_t*>(key_s + TG * Epad);   // [TG][Epad] selection keys, the leader's
    float* red_s = key_s + 2 * TG * Epad;                 // [TG][warps][2]

    pdl_launch_dependents();
    // this block's experts: the slot of warp group g in pass p is (p * groups + g) * cs + rank
    const int groups = kRtWarps / a.parts;
    const int grp = warp / a.parts, sub = warp % a.parts;
    const int k0 = static_cast<int>(static_cast<long long>(sub) * K4 / a.parts);
    const int k1 = static_cast<int>(static_cast<long long>(sub + 1) * K4 / a.parts);
    // the router's weights do not depend on the previous kernel: the first
    // pieces of this warp's first expert into registers, the rest towards L2
    float4 w0[kRtAhead];
    {
        const int e = grp * cs + rank;
        const float4* wr = reinterpret_cast<const float4*>(a.w + static_cast<size_t>(e) * K);
#pragma unroll
        for (int u = 0; u < kRtAhead; ++u) {
            const int i = k0 + lane + 32 * u;
            w0[u] = e < a.E && i < k1 ? __ldg(wr + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    for (int e = grp * cs + rank; e < a.E; e += groups * cs) {
        const char* row = reinterpret_cast<const char*>(a.w + static_cast<size_t>(e) * K);
        for (int o = (sub * 32 + lane) * 128; o < 4 * K; o += a.parts * 32 * 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(row + o));
    }
    pdl_wait();
    moe_fill(a.fill);

    // ---- the tokens as fp32 in shared memory, normalized
    float hi[TG], lo[TG];
#pragma unroll
    for (int t = 0; t < TG; ++t) {
        hi[t] = lo[t] = 0.0f;
        if (t < nt)
            for (int i = tid; i < K8; i += kRtThreads) {
                float v[8];
                load8<XT>(a.x, static_cast<size_t>(m0 + t) * K + 8 * i, v);
                float4* d = reinterpret_cast<float4*>(xs + t * K) + 2 * i;
                d[0] = make_float4(v[0], v[1], v[2], v[3]);
                d[1] = make_float4(v[4], v[5], v[6], v[7]);
                if (a.gamma != nullptr)
#pragma unroll
                    for (int k = 0; k < 8; ++k) sq_acc(v[k], hi[t], lo[t]);
            }
    }
    if (a.gamma != nullptr) {
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            warp_pair_sum(hi[t], lo[t]);
            if (lane == 0) {
                red_s[(t * kRtWarps + warp) * 2] = hi[t];
                red_s[(t * kRtWarps + warp) * 2 + 1] = lo[t];
            }
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            // the 16 warps' pairs, by every warp (both halves of it alike)
            static_assert(kRtWarps == 16, "a half warp holds the block's pairs");
            float h = red_s[(t * kRtWarps + (lane & 15)) * 2], l = red_s[(t * kRtWarps + (lane & 15)) * 2 + 1];
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) {
                const float h2 = __shfl_xor_sync(0xffffffffu, h, off), l2 = __shfl_xor_sync(0xffffffffu, l, off);
                // (both partners add the same way round: the same result in every lane)
                const bool up = (lane & off) != 0;
                float a0 = up ? h2 : h, a1 = up ? l2 : l;
                pair_merge(a0, a1, up ? h : h2, up ? l : l2);
                h = a0;
                l = a1;
            }
            const float r = rms_scale(h, l, K, a.eps);
            if (t < nt)
                for (int i = tid; i < K8; i += kRtThreads) {          // the same places as above: no barrier
                    float4* d = reinterpret_cast<float4*>(xs + t * K) + 2 * i;
                    const float4* g = reinterpret_cast<const float4*>(a.gamma) + 2 * i;
                    d[0] = rms_apply(d[0], r, __ldg(g));
                    d[1] = rms_apply(d[1], r, __ldg(g + 1));
                }
        }
    }
    __syncthreads();

    // ---- logits
    if (cs > 1) cluster_sync();                       // the leader's shared memory is there
    for (int e0 = 0; e0 < a.E; e0 += groups * cs) {
        const int e = e0 + grp * cs + rank;
        float ah[TG][4], al[TG][4];
#pragma unroll
        for (int t = 0; t < TG; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) ah[t][k] = al[t][k] = 0.0f;
        if (e < a.E) {
            const float4* wr = reinterpret_cast<const float4*>(a.w + static_cast<size_t>(e) * K);
            auto piece = [&](const float4& w, int i) {
#pragma unroll
                for (int t = 0; t < TG; ++t) {
                    const float4 x = reinterpret_cast<const float4*>(xs + t * K)[i];
                    if (t < nt) {
                        dot_acc(x.x, w.x, ah[t][0], al[t][0]);
                        dot_acc(x.y, w.y, ah[t][1], al[t][1]);
                        dot_acc(x.z, w.z, ah[t][2], al[t][2]);
                        dot_acc(x.w, w.w, ah[t][3], al[t][3]);
                    }
                }
            };
            if (e0 == 0) {
#pragma unroll
                for (int u = 0; u < kRtAhead; ++u)
                    if (k0 + lane + 32 * u < k1) piece(w0[u], k0 + lane + 32 * u);
            }
#pragma unroll 4
            for (int i = k0 + lane + (e0 == 0 ? 32 * kRtAhead : 0); i < k1; i += 32) piece(__ldg(wr + i), i);
        }
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            pair_merge(ah[t][0], al[t][0], ah[t][1], al[t][1]);
            pair_merge(ah[t][2], al[t][2], ah[t][3], al[t][3]);
            pair_merge(ah[t][0], al[t][0], ah[t][2], al[t][2]);
            warp_pair_sum(ah[t][0], al[t][0]);
            if (lane == 0) {
                part_s[(warp * TG + t) * 2] = ah[t][0];
                part_s[(warp * TG + t) * 2 + 1] = al[t][0];
            }
        }
        __syncthreads();
        if (tid < groups * TG) {
            const int g = tid / TG, t = tid % TG;
            const int ee = e0 + g * cs + rank;
            if (ee < a.E && t < nt) {
                const float* p = part_s + (g * a.parts * TG + t) * 2;
                float h = p[0], l = p[1];
                for (int s = 1; s < a.parts; ++s) pair_merge(h, l, p[s * TG * 2], p[s * TG * 2 + 1]);
                // (past fp32 the errors of the sum are NaN)
                const float logit = fabsf(h) <= 0x1.fffffep+127f ? __fadd_rn(h, l) : h;
                if (cs > 1) st_cluster_u32(mapa_shared(smem_u32(key_s + t * Epad + ee), 0u), __float_as_uint(logit));
                else key_s[t * Epad + ee] = logit;
            }
        }
        __syncthreads();
    }
    if (cs > 1) cluster_sync();

    // ---- the codes (the last block) and the choice (the first)
    if (rank == cs - 1 && a.qx != nullptr) {
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            float mx = 0.0f;
            if (t < nt)
                for (int i = tid; i < K4; i += kRtThreads) {
                    const float4 v = reinterpret_cast<const float4*>(xs + t * K)[i];
                    mx = fmaxf(mx, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
                }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            if (lane == 0) red_s[warp * TG + t] = mx;
        }
        __syncthreads();
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            if (t >= nt) break;
            float amax = red_s[t];
#pragma unroll
            for (int w = 1; w < kRtWarps; ++w) amax = fmaxf(amax, red_s[w * TG + t]);
            const A8Scale ks = a8_scale(amax);
            if (tid == 0) a.sx[m0 + t] = ks.s;
            uint2* q = reinterpret_cast<uint2*>(a.qx + static_cast<size_t>(m0 + t) * K);
            for (int i = tid; i < K8; i += kRtThreads) {
                const float4* d = reinterpret_cast<const float4*>(xs + t * K) + 2 * i;
                const float v[8] = {d[0].x, d[0].y, d[0].z, d[0].w, d[1].x, d[1].y, d[1].z, d[1].w};
                q[i] = quant8(v, ks);
            }
        }
    }
    if (rank == 0 && warp < nt) {
        float* key = key_s + warp * Epad;                 // logits, then (sigmoid) scores and the selection key
        const int m = m0 + warp;
        // each lane's keys are its own places of the array
        auto key_of = [&](int e) -> uint32_t {
            float v = key[e];
            if (a.sigmoid) {
                v = xa_logistic(v);
                key[e] = v;
                if (a.sel != nullptr) v = __fadd_rn(v, __ldg(a.sel + e));
            }
            return order_key(v);
        };
        uint32_t mine0 = 0u, mine1 = 0u;                  // up to 64 experts: the keys stay in registers
        const bool small = a.E <= 64;
        float sum_all = 0.0f, top = 0.0f;
        int my_id = 0;
        float my_val = 0.0f;
        if (small) {
            if (lane < a.E) mine0 = key_of(lane);
            if (lane + 32 < a.E) mine1 = key_of(lane + 32);
        } else {
            for (int e = lane; e < a.E; e += 32) ord_s[warp * Epad + e] = key_of(e);
        }
        __syncwarp();
        for (int k = 0; k < a.top_k; ++k) {
            uint32_t best = 0u;
            int at = 0x7fffffff;
            if (small) {
                if (mine0 != 0u) {
                    best = mine0;
                    at = lane;
                }
                if (mine1 > best) {
                    best = mine1;
                    at = lane + 32;
                }
            } else {
                // (taken ones are 0)
                for (int e = lane; e < a.E; e += 32) {
                    const uint32_t u = ord_s[warp * Epad + e];
                    if (u > best) {
                        best = u;
                        at = e;
                    }
                }
            }
            const uint32_t win = __reduce_max_sync(0xffffffffu, best);
            const int id = static_cast<int>(__reduce_min_sync(0xffffffffu, best == win ? static_cast<unsigned>(at) : 0x7fffffffu));
            if (at == id) {
                if (!small) ord_s[warp * Epad + id] = 0u;
                else if (id < 32) mine0 = 0u;
                else mine1 = 0u;
            }
            const float v = key[id];
            if (k == 0) top = v;
            if (lane == k) {
                my_id = id;
                my_val = v;
            }
        }
        if (!a.sigmoid) {
            if (!a.renorm) {
                for (int e = lane; e < a.E; e += 32) sum_all += expf(__fsub_rn(key[e], top));
            }
            my_val = lane < a.top_k ? expf(__fsub_rn(my_val, top)) : 0.0f;
        }
        if (lane >= a.top_k) my_val = 0.0f;
        float sum = a.renorm ? my_val : sum_all;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, off));
        if (lane < a.top_k) {
            float w = my_val;
            if (a.renorm || !a.sigmoid) w = sum != 0.0f ? __fdiv_rn(w, sum) : 0.0f;
            a.ids[static_cast<size_t>(m) * a.top_k + lane] = my_id;
            a.weights[static_cast<size_t>(m) * a.top_k + lane] = __fmul_rn(w, a.scale);
        }
    }
}

template <int XT, int TG>
cudaError_t launch_route_t(const RouteArgs& a, bool pdl, cudaStream_t s)
{
    auto kern = moe_route_kernel<XT, TG>;
    const size_t smem = static_cast<size_t>(route_smem(TG, a.K, a.E));
    static SmemLimit limit, wide;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), limit, smem);
    if (e != cudaSuccess) return e;
    if (a.cluster > 8) {
        int dev = 0;
        e = cudaGetDevice(&dev);
        if (e == cudaSuccess && wide.bytes[dev].load(std::memory_order_acquire) == 0) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e == cudaSuccess) wide.bytes[dev].store(1, std::memory_order_release);
        }
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.M + TG - 1) / TG * a.cluster));
    cfg.blockDim = dim3(kRtThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (pdl) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    if (a.cluster > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = static_cast<unsigned>(a.cluster);
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    cfg.attrs = na > 0 ? attr : nullptr;
    cfg.numAttrs = static_cast<unsigned>(na);
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int XT>
cudaError_t launch_route_x(const RouteArgs& a, bool pdl, cudaStream_t s)
{
    if (a.tok == 1) return launch_route_t<XT, 1>(a, pdl, s);
    if (a.tok == 2) return launch_route_t<XT, 2>(a, pdl, s);
    return launch_route_t<XT, 4>(a, pdl, s);
}

}  // namespace

cudaError_t launch_moe_route(const RouteArgs& a, int xtype, bool pdl, cudaStream_t s)
{
    if (xtype == T_F32) return launch_route_x<T_F32>(a, pdl, s);
    if (xtype == T_F16) return launch_route_x<T_F16>(a, pdl, s);
    return launch_route_x<T_BF16>(a, pdl, s);
}

}  // namespace w4k
