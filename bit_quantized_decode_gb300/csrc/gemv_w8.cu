// INT8 x INT8 linear of one to eight tokens: the weights are streamed once at
// HBM speed and the products formed with DP4A, exactly,
//   y = fma(fp32(s_w s_x), fp32(acc), b) (+ residual), rounded to y's type.
//
// Bound by the weights' bytes for long matrices and by latency for short ones.
//   * Every warp streams its row tiles (8 rows) through a ring of two slots fed
//     by bulk copies; the first are asked for before the dependency wait.  A
//     slot costs a wait and a copy however large it is, so it is 8 KB where the
//     codes leave room.  Few tiles: two or four warps share one, each a part of
//     K, and add their integer sums in shared memory.
//   * One or two tokens: every block normalizes and quantizes them itself (a
//     launch less); more come as codes from the row quantizer.
//   * A weight word meets four codes in one DP4A, with no unpacking; past eight
//     tokens the tensor cores' product (gemm_w8.cu) takes over.  Both are exact,
//     so the results agree bit for bit.  us in graph replays, quantizer included
//     (the tensor cores' product at the same tokens), 152064 x 3584: one token
//     80.7 (6.77 TB/s), two 83.6 (91.5), four 87.5 (91.0), seven 90.4 (92.1),
//     eight 95.5 (92.0); 4608 x 3584: two 6.6 (11.3), eight 9.6 (11.4).  At eight
//     a long matrix would gain from changing over and a short one would lose more.
// 4608 x 3584 with its norm, one token: 6.3 us.
#include "fusion.cuh"
#include "operators.h"
#include "ptx.cuh"
#include "quant_a8.cuh"
#include "typed_io.cuh"

namespace w4k {
namespace {

constexpr uint64_t kV8WaitNs = 250ull * 1000ull * 1000ull;

__device__ __forceinline__ void load8_typed(int type, const void* base, size_t at, float (&v)[8])
{
    if (type == T_F32) load8<T_F32>(base, at, v);
    else if (type == T_F16) load8<T_F16>(base, at, v);
    else load8<T_BF16>(base, at, v);
}

// Codes of the block's tokens into xs (and, from block 0, to the caller):
// kV8Warps / M warps to a token.
template <int TK>
__device__ __forceinline__ void quantize_tokens(const Gemv8Args& A, int8_t* xs, float* sx_s, float* red_s)
{
    constexpr int kPer = kV8Warps / TK;                    // warps per token
    constexpr int kKeep = 5;                               // groups of eight values that a thread keeps
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int m = warp / kPer, t = threadIdx.x - m * kPer * 32;
    const int K8 = A.K >> 3;
    const bool have = m < A.M;
    const size_t row = static_cast<size_t>(m) * A.K;
    float v[kKeep][8];
    float hi = 0.0f, lo = 0.0f, mx = 0.0f, r = 1.0f;
    if (have) {
#pragma unroll
        for (int u = 0; u < kKeep; ++u)
            if (t + u * kPer * 32 < K8) load8_typed(A.xtype, A.x, row + 8 * static_cast<size_t>(t + u * kPer * 32), v[u]);
            else zero8(v[u]);
    }
    // f(group, values) over this thread's groups, the kept ones first
    auto each = [&](auto&& f) {
        if (!have) return;
#pragma unroll
        for (int u = 0; u < kKeep; ++u)
            if (t + u * kPer * 32 < K8) f(t + u * kPer * 32, v[u], true);
        for (int i = t + kKeep * kPer * 32; i < K8; i += kPer * 32) {
            float w[8];
            load8_typed(A.xtype, A.x, row + 8 * static_cast<size_t>(i), w);
            f(i, w, false);
        }
    };
    auto scaled = [&](int i, float (&w)[8]) {
        float g[8];
        load8<T_F32>(A.gamma, 8 * static_cast<size_t>(i), g);
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = __fmul_rn(__fmul_rn(w[k], r), g[k]);
    };
    if (A.gamma != nullptr) {
        each([&](int, float (&w)[8], bool) {
#pragma unroll
            for (int k = 0; k < 8; ++k) sq_acc(w[k], hi, lo);
        });
        warp_pair_sum(hi, lo);
        if (lane == 0) {
            red_s[2 * warp] = hi;
            red_s[2 * warp + 1] = lo;
        }
        __syncthreads();
        if (have) {
            hi = red_s[2 * m * kPer];
            lo = red_s[2 * m * kPer + 1];
#pragma unroll
            for (int w = 1; w < kPer; ++w) pair_merge(hi, lo, red_s[2 * (m * kPer + w)], red_s[2 * (m * kPer + w) + 1]);
            r = rms_scale(hi, lo, A.K, A.eps);
        }
        __syncthreads();
    }
    each([&](int i, float (&w)[8], bool) {
        if (A.gamma != nullptr) scaled(i, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(w[k]));
    });
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    if (lane == 0) red_s[warp] = mx;
    __syncthreads();
    float amax = 0.0f;
    if (have) {
#pragma unroll
        for (int w = 0; w < kPer; ++w) amax = fmaxf(amax, red_s[m * kPer + w]);
    }
    const A8Scale ks = a8_scale(amax);
    if (have && t == 0) {
        sx_s[m] = ks.s;
        if (blockIdx.x == 0) A.sx_out[m] = ks.s;
    }
    uint2* out = have ? reinterpret_cast<uint2*>(xs + row) : nullptr;
    uint2* gout = have && blockIdx.x == 0 && A.qx_out != nullptr ? reinterpret_cast<uint2*>(A.qx_out + row) : nullptr;
    each([&](int i, float (&w)[8], bool kept) {
        if (!kept && A.gamma != nullptr) scaled(i, w);
        const uint2 q = quant8(w, ks);
        out[i] = q;
        if (gout != nullptr) gout[i] = q;
    });
}

template <int TK, bool kFused>
__global__ void __launch_bounds__(kV8Threads, 1) gemv_w8_kernel(const __grid_constant__ Gemv8Args A)
{
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slot = A.slot;
    uint8_t* ring = smem + static_cast<size_t>(warp) * 2 * slot;
    int8_t* xs = reinterpret_cast<int8_t*>(smem + kV8Warps * 2 * slot);
    int* part_s = reinterpret_cast<int*>(xs + A.M * A.K);                 // [warp][8 rows][kV8MaxTok]
    float* sx_s = reinterpret_cast<float*>(part_s + kV8Warps * 8 * kV8MaxTok);
    float* red_s = sx_s + 4 * kV8MaxTok;
    uint64_t* bars = reinterpret_cast<uint64_t*>(red_s + 4 * kV8Warps);
    const uint32_t my_bar = smem_u32(bars + 2 * warp), xbar = smem_u32(bars + 2 * kV8Warps);
    if (lane == 0) {
        mbar_init(my_bar, 1);
        mbar_init(my_bar + 8, 1);
        if (warp == 0) mbar_init(xbar, 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_launch_dependents();

    // ---- this warp's tiles: group `grp` of the block, of whose K this warp has [c0, c1)
    const int share = A.share, groups = kV8Warps / share;
    const int grp = warp / share, sub = warp - grp * share;
    const int C = A.K >> 5, T = (A.N + 7) >> 3;
    const int c0 = sub * C / share & ~15, c1 = sub == share - 1 ? C : (sub + 1) * C / share & ~15;
    const int lines = slot >> 8;                                          // 256 bytes: 8 rows x 32 weights
    const int step = groups * static_cast<int>(gridDim.x);
    const int t_first = grp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    const uint64_t pol = l2_policy_evict_first();
    int it = t_first, ic = c0, issued = 0, consumed = 0;                  // the slice to issue next
    const uint32_t ring_u = smem_u32(ring);
    auto issue_one = [&]() {
        if (it >= T) return;
        const int n = min(lines, c1 - ic);
        if (elect_one()) {
            const uint32_t bar = my_bar + 8 * (issued & 1);
            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(n) << 8);
            bulk_g2s(ring_u + static_cast<uint32_t>((issued & 1) * slot), A.w + ((static_cast<size_t>(it) * C + ic) << 8),
                     static_cast<uint32_t>(n) << 8, bar, pol);
        }
        __syncwarp();
        ++issued;
        ic += n;
        if (ic >= c1) {
            ic = c0;
            it += step;
        }
    };
    issue_one();
    issue_one();
    pdl_wait();

    // ---- the tokens' codes
    if constexpr (kFused) {
        quantize_tokens<TK>(A, xs, sx_s, red_s);
    } else {
        if (warp == 0 && elect_one()) {
            mbar_arrive_expect_tx(xbar, static_cast<uint32_t>(A.M * A.K));
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             smem_u32(xs)),
                         "l"(A.qx_in), "r"(static_cast<uint32_t>(A.M * A.K)), "r"(xbar)
                         : "memory");
        }
        if (tid < A.M) sx_s[tid] = __ldg(A.sx_in + tid);
        if (warp == 0 && !__all_sync(0xffffffffu, mbar_wait_bounded(xbar, 0u, kV8WaitNs)) && lane == 0 && A.err != nullptr)
            atomicExch(A.err, kErrWaitTimeout);
    }
    __syncthreads();

    const int hb = lane & 1, pl = lane >> 1, pp = pl & 3, my_row = 4 * hb + pp, qd = lane >> 3;
    int perm[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) perm[j] = ((j ^ pp) << 5) + (hb << 4);
    uint32_t ph = 0u;
    bool dead = false;
    for (int tile = t_first; tile < T; tile += step) {
        const int row = 8 * tile + my_row;
        float sw = 0.0f, bv = 0.0f;
        if (sub == 0 && row < A.N) {
            sw = __ldg(A.s_w + row);
            if (A.bias != nullptr) bv = __ldg(A.bias + row);
        }
        int acc[TK][4], acc2[TK][4];
#pragma unroll
        for (int m = 0; m < TK; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[m][j] = acc2[m][j] = 0;
        const int8_t* codes = xs + (c0 + pl) * 32;
        for (int c = c0; c < c1 && !dead; c += lines) {
            const uint32_t bar = my_bar + 8 * (consumed & 1);
            bool ok = __all_sync(0xffffffffu, mbar_test_wait(bar, ph));
            if (!ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, ph, kV8WaitNs));
            if (!ok) {
                dead = true;                       // stop computing, keep the groups' barriers
                if (lane == 0 && A.err != nullptr) atomicExch(A.err, kErrWaitTimeout);
                break;
            }
            const uint8_t* ub = ring + (consumed & 1) * slot + (pl * kRows + 4 * hb) * 32;
            const int n = min(lines, c1 - c) - pl;
#pragma unroll 2
            for (int l = 0; l < n; l += 16) {
                uint4 w0[4], w1[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // the halves are read in a lane-dependent order to spread the banks
                    const uint4 first = *reinterpret_cast<const uint4*>(ub + perm[j]);
                    const uint4 second = *reinterpret_cast<const uint4*>(ub + (perm[j] ^ 16));
                    w0[j] = hb ? second : first;
                    w1[j] = hb ? first : second;
                }
#pragma unroll
                for (int m = 0; m < TK; ++m) {
                    if (m == 0 || m < A.M) {
                        const uint4* xp = reinterpret_cast<const uint4*>(codes + m * A.K);
                        const uint4 x0 = xp[0], x1 = xp[1];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            int a = acc[m][j], b = TK <= 4 ? acc2[m][j] : 0;
                            a = dp4a_ss(w0[j].x, x0.x, a);
                            b = dp4a_ss(w1[j].x, x1.x, b);
                            a = dp4a_ss(w0[j].y, x0.y, a);
                            b = dp4a_ss(w1[j].y, x1.y, b);
                            a = dp4a_ss(w0[j].z, x0.z, a);
                            b = dp4a_ss(w1[j].z, x1.z, b);
                            a = dp4a_ss(w0[j].w, x0.w, a);
                            b = dp4a_ss(w1[j].w, x1.w, b);
                            if (TK <= 4) {
                                acc[m][j] = a;
                                acc2[m][j] = b;
                            } else {
                                acc[m][j] = a + b;
                            }
                        }
                    }
                }
                ub += 16 * kRows * 32;
                codes += 16 * 32;
            }
            ph ^= static_cast<uint32_t>(consumed & 1);
            ++consumed;
            __syncwarp();
            issue_one();
        }
        // lanes of equal (hb, pp) add up, then the read permutation is undone
#pragma unroll
        for (int m = 0; m < TK; ++m) {
            if (m == 0 || m < A.M) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (TK <= 4) acc[m][j] += acc2[m][j];
                    acc[m][j] += __shfl_xor_sync(0xffffffffu, acc[m][j], 8);
                    acc[m][j] += __shfl_xor_sync(0xffffffffu, acc[m][j], 16);
                }
                acc[m][0] += __shfl_xor_sync(0xffffffffu, acc[m][2], 4);
                acc[m][1] += __shfl_xor_sync(0xffffffffu, acc[m][3], 4);
                acc[m][0] += __shfl_xor_sync(0xffffffffu, acc[m][1], 2);
            }
        }
        if (share > 1) {
            // the warps of a group: sums through shared memory, the first one on
            int* mine = part_s + warp * 8 * kV8MaxTok;
            if (sub > 0 && lane < 8) {
#pragma unroll
                for (int m = 0; m < TK; ++m) mine[my_row * kV8MaxTok + m] = acc[m][0];
            }
            named_sync(1 + grp, static_cast<uint32_t>(32 * share));
            if (sub == 0) {
                for (int s = 1; s < share; ++s)
#pragma unroll
                    for (int m = 0; m < TK; ++m) acc[m][0] += part_s[((warp + s) * 8 + my_row) * kV8MaxTok + m];
            }
            named_sync(1 + grp, static_cast<uint32_t>(32 * share));
        }
        if (sub == 0 && !dead) {
#pragma unroll
            for (int i = 0; i < (TK + 3) / 4; ++i) {
                const int m = 4 * i + qd;
                if (4 * i >= A.M) break;
                int a = acc[4 * i][0];
#pragma unroll
                for (int q = 1; q < 4; ++q)
                    if (4 * i + q < TK && qd == q) a = acc[4 * i + q < TK ? 4 * i + q : 0][0];
                if (m < A.M && row < A.N) {
                    float v = __fmaf_rn(__fmul_rn(sw, sx_s[m]), __int2float_rn(a), bv);
                    const size_t o = static_cast<size_t>(m) * A.N + row;
                    if (A.residual != nullptr) v = __fadd_rn(A.residual[o], v);
                    store_typed(A.y, A.ytype, o, v);
                }
            }
        }
    }
    // after a wait that ran out: the copies in flight land before the block ends
    if (dead)
        for (int k = consumed; k < issued; ++k)
            if (!mbar_wait_bounded(my_bar + 8 * (k & 1), static_cast<uint32_t>(k >> 1) & 1u, kV8WaitNs)) break;
}

template <int TK, bool kFused>
cudaError_t launch_t(const Gemv8Args& a, int grid, size_t smem, bool pdl, cudaStream_t s)
{
    auto kern = gemv_w8_kernel<TK, kFused>;
    static SmemLimit limit;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), limit, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kV8Threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_gemv_w8(const Gemv8Args& a, int grid, size_t smem, bool pdl, cudaStream_t s)
{
    if (a.x != nullptr) return a.M <= 1 ? launch_t<1, true>(a, grid, smem, pdl, s) : launch_t<2, true>(a, grid, smem, pdl, s);
    if (a.M <= 1) return launch_t<1, false>(a, grid, smem, pdl, s);
    if (a.M <= 2) return launch_t<2, false>(a, grid, smem, pdl, s);
    if (a.M <= 4) return launch_t<4, false>(a, grid, smem, pdl, s);
    return launch_t<8, false>(a, grid, smem, pdl, s);
}

}  // namespace w4k
