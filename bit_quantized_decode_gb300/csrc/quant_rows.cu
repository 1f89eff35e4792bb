// Per-token INT8 activation codes for any number of tokens and for fp32, fp16
// or bf16 activations, with RMSNorm in front where asked: the codes and scales
// of a8_quantize / rms_a8_quantize (every step an IEEE fp32 operation on the
// activations widened to fp32, see quant_a8.cuh and fusion.cuh).
//
// One block per token, or a cluster of up to eight where tokens are few and
// long: each block then has a part of the row, and they exchange their sums and
// maxima through distributed shared memory (64 tokens of 18944: 6.5 -> 4 us).
// The row stays in registers between the norm, the maximum and the rounding
// (up to 20480 values a block; longer ones are read again).  Besides
// the int8 codes it writes them as fp16 in the layout that the tensor-core
// product copies tiles of (f16_word): a stage of a token tile is one
// contiguous run in the MMA's core-matrix order.  It moves the activations once and the codes once (2 bytes each); its
// time is HBM traffic for long prompts and one launch's latency for few tokens.
// Short rows on as many blocks per SM as registers allow: 1000 tokens of 1536 in
// one wave of blocks instead of two (22.5 -> 22.0 us with their product).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fusion.cuh"
#include "operators.h"
#include "ptx.cuh"
#include "quant_a8.cuh"
#include "typed_io.cuh"

namespace w4k {
namespace {

constexpr int kQrThreads = 256;
constexpr int kQrWarps = kQrThreads / 32;
constexpr int kQrMaxCluster = 8;

template <int XT, int NIT, bool kNorm>
__global__ void __launch_bounds__(kQrThreads, NIT == 1 ? 7 : NIT == 2 ? 5 : 1) quant_rows_kernel(const QuantRowsArgs a)
{
    __shared__ float red_s[2 * kQrWarps];
    __shared__ float all_s[3 * kQrMaxCluster];                  // the cluster's blocks: sums (hi, lo), maxima
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cs = a.cluster;
    const int rank = cs > 1 ? static_cast<int>(blockIdx.x) % cs : 0;
    const int m = static_cast<int>(blockIdx.x) / cs;
    const int K8_all = a.K >> 3;
    const int k0 = static_cast<int>(static_cast<long long>(rank) * K8_all / cs);
    const int K8 = static_cast<int>(static_cast<long long>(rank + 1) * K8_all / cs) - k0;    // this block's groups of eight
    constexpr int kN = NIT > 0 ? NIT : 1;
    pdl_launch_dependents();
    if (cs > 1) cluster_arrive_release();                       // waited for before the first store to another block
    pdl_wait();
    const size_t row = static_cast<size_t>(m) * a.K + 8 * static_cast<size_t>(k0);
    float v[kN][8];
    if constexpr (NIT > 0) {
#pragma unroll
        for (int it = 0; it < NIT; ++it) {
            const int i = tid + it * kQrThreads;
            if (i < K8) load8<XT>(a.x, row + 8 * static_cast<size_t>(i), v[it]);
            else zero8(v[it]);
        }
    }
    auto each = [&](auto&& f) {
        if constexpr (NIT > 0) {
#pragma unroll
            for (int it = 0; it < NIT; ++it) {
                const int i = tid + it * kQrThreads;
                if (i < K8) f(i, v[it]);
            }
        } else {
            for (int i = tid; i < K8; i += kQrThreads) {
                load8<XT>(a.x, row + 8 * static_cast<size_t>(i), v[0]);
                f(i, v[0]);
            }
        }
    };
    float r = 1.0f;
    auto normed = [&](int i, float (&t)[8]) {
        if constexpr (kNorm) {
            float g[8];
            load8<T_F32>(a.gamma, 8 * static_cast<size_t>(k0 + i), g);
#pragma unroll
            for (int k = 0; k < 8; ++k) t[k] = __fmul_rn(__fmul_rn(t[k], r), g[k]);
        }
    };
    if constexpr (kNorm) {
        float hi = 0.0f, lo = 0.0f;
        each([&](int, float (&t)[8]) {
#pragma unroll
            for (int k = 0; k < 8; ++k) sq_acc(t[k], hi, lo);
        });
        warp_pair_sum(hi, lo);
        if (lane == 0) {
            red_s[2 * warp] = hi;
            red_s[2 * warp + 1] = lo;
        }
        __syncthreads();
        hi = red_s[0];
        lo = red_s[1];
#pragma unroll
        for (int w = 1; w < kQrWarps; ++w) pair_merge(hi, lo, red_s[2 * w], red_s[2 * w + 1]);
        if (cs > 1) {
            cluster_wait_acquire();
            if (tid < cs) {
                st_cluster_u32(mapa_shared(smem_u32(all_s + 2 * rank), static_cast<uint32_t>(tid)), __float_as_uint(hi));
                st_cluster_u32(mapa_shared(smem_u32(all_s + 2 * rank + 1), static_cast<uint32_t>(tid)), __float_as_uint(lo));
            }
            cluster_sync();
            hi = all_s[0];
            lo = all_s[1];
            for (int b = 1; b < cs; ++b) pair_merge(hi, lo, all_s[2 * b], all_s[2 * b + 1]);
        }
        r = rms_scale(hi, lo, a.K, a.eps);
        __syncthreads();
    }
    float mx = 0.0f;
    each([&](int i, float (&t)[8]) {
        normed(i, t);
#pragma unroll
        for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(t[k]));
    });
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    if (lane == 0) red_s[warp] = mx;
    __syncthreads();
    float amax = red_s[0];
#pragma unroll
    for (int w = 1; w < kQrWarps; ++w) amax = fmaxf(amax, red_s[w]);
    if (cs > 1) {
        float* max_s = all_s + 2 * kQrMaxCluster;
        if (!kNorm) cluster_wait_acquire();
        if (tid < cs) st_cluster_u32(mapa_shared(smem_u32(max_s + rank), static_cast<uint32_t>(tid)), __float_as_uint(amax));
        cluster_sync();
        for (int b = 0; b < cs; ++b) amax = fmaxf(amax, max_s[b]);
    }
    const A8Scale ks = a8_scale(amax);
    if (tid == 0 && rank == 0) a.sx[m] = ks.s;
    uint2* q8 = a.qx != nullptr ? reinterpret_cast<uint2*>(a.qx + row) : nullptr;
    each([&](int i, float (&t)[8]) {
        if constexpr (NIT == 0) normed(i, t);
        const uint2 q = quant8(t, ks);
        if (q8 != nullptr) q8[i] = q;
        if (a.xh != nullptr) a.xh[f16_word(m, k0 + i, K8_all, a.nt)] = codes_f16(q);
    });
}

__global__ void __launch_bounds__(256) expand_codes_kernel(const int8_t* __restrict__ qx, int M, int K8,
                                                           uint4* __restrict__ xh, int nt)
{
    pdl_launch_dependents();
    pdl_wait();
    const int m = blockIdx.x;
    const uint2* q = reinterpret_cast<const uint2*>(qx) + static_cast<size_t>(m) * K8;
    for (int i = threadIdx.x; i < K8; i += 256) xh[f16_word(m, i, K8, nt)] = codes_f16(__ldg(q + i));
}

cudaLaunchConfig_t row_launch(int blocks, int threads, bool pdl, cudaStream_t s, cudaLaunchAttribute* attr)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cfg;
}

template <int XT, bool kNorm>
cudaError_t launch_rows(const QuantRowsArgs& a, const cudaLaunchConfig_t& cfg)
{
    const int nit = ((a.K / 8 + a.cluster - 1) / a.cluster + kQrThreads - 1) / kQrThreads;
    if (nit <= 1) return cudaLaunchKernelEx(&cfg, quant_rows_kernel<XT, 1, kNorm>, a);
    if (nit <= 2) return cudaLaunchKernelEx(&cfg, quant_rows_kernel<XT, 2, kNorm>, a);
    if (nit <= 4) return cudaLaunchKernelEx(&cfg, quant_rows_kernel<XT, 4, kNorm>, a);
    if (nit <= 10) return cudaLaunchKernelEx(&cfg, quant_rows_kernel<XT, 10, kNorm>, a);
    return cudaLaunchKernelEx(&cfg, quant_rows_kernel<XT, 0, kNorm>, a);
}

template <int XT>
cudaError_t launch_typed(const QuantRowsArgs& a, const cudaLaunchConfig_t& cfg)
{
    return a.gamma != nullptr ? launch_rows<XT, true>(a, cfg) : launch_rows<XT, false>(a, cfg);
}

}  // namespace

cudaError_t launch_quant_rows(const QuantRowsArgs& args, int xtype, bool pdl, cudaStream_t s)
{
    // a block for about 4096 values, while there are few blocks
    QuantRowsArgs a = args;
    a.cluster = 1;
    while (a.cluster < kQrMaxCluster && a.K >= 8192 * a.cluster && a.M * a.cluster <= 256) a.cluster *= 2;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = row_launch(a.M * a.cluster, kQrThreads, pdl, s, attr);
    if (a.cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = static_cast<unsigned>(a.cluster);
        attr[cfg.numAttrs].val.clusterDim.y = 1;
        attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
        cfg.attrs = attr;
    }
    if (xtype == T_F32) return launch_typed<T_F32>(a, cfg);
    if (xtype == T_F16) return launch_typed<T_F16>(a, cfg);
    return launch_typed<T_BF16>(a, cfg);
}

cudaError_t launch_expand_codes(const int8_t* qx, int M, int K, uint4* xh, int nt, bool pdl, cudaStream_t s)
{
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = row_launch(M, 256, pdl, s, attr);
    return cudaLaunchKernelEx(&cfg, expand_codes_kernel, qx, M, K / 8, xh, nt);
}

}  // namespace w4k
