// INT8 x INT8 matrix product of many tokens: the arithmetic of gemm_w8.cu
// (weights converted to fp16 in tensor memory, sums exact in fp32 over 1024 K,
// then int32) on tiles of 256 weight rows by up to 192 tokens, each computed by
// a pair of thread blocks with cta_group::2.
//
// Against one block per 128 x 128 tile: a block holds its own 128 rows of A and
// half of the tokens of B, so the codes move through L2 and shared memory once
// for 256 rows, and an MMA has 1.5 times the columns (a small one is bound by
// its issue).  Per 128 K and block: 16 KB of weights and 24 KB of codes for 768
// cycles of MMA.
//   * The MMA warp of the pair's first block issues for both; converted weights
//     and landed codes are announced to its barriers by both blocks' converting
//     warps (remote arrivals, cluster scope), and its commits arrive in both.
//   * Tensor memory: two accumulators of the tile's columns and four half
//     stages (64 K) of A.  Group g of the converting warps takes half g of every
//     stage, so a half is converted while the others are multiplied.
//   * The epilogue's two warpgroups hold 96 columns of int32 each; registers are
//     moved to them from the others (setmaxnreg; 5 x 128 threads start with 96,
//     then 40 + 72 + 72 + 144 + 144 of 480).
// 4096 tokens, 37888 x 3584 in bf16, with the quantizer: 728 to 734 us in graph
// replays, 1.52 PFLOP/s (the library's bf16 product sustains 1.73 on this chip),
// 760 us as single calls on changing inputs; the tensor pipe is active for two
// thirds of the time.
#include "gemm_w8.cuh"

namespace w4k {
namespace {

constexpr int kP8Epi = 12, kP8Conv = 4;                 // first warps of the epilogue and of the converting groups

__device__ __forceinline__ void pair_alloc(uint32_t dst_smem, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// One arrival on the barrier at this offset in both blocks once the MMAs issued so far have completed.
__device__ __forceinline__ void pair_commit(uint32_t bar)
{
    asm volatile("{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
                 "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(bar)
                 : "memory");
}
// Four MMAs: 64 K of A (eight columns to a slice) against B descriptors `bstep` apart.
__device__ __forceinline__ void pair_mma_x4(uint32_t d, uint32_t a, uint64_t b, uint64_t bstep, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 a1;\n\t.reg .b64 b1;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 q, %5, %5;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %4, p;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u64 b1, %2, %3;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], [a1], b1, %4, q;\n\t"
        "add.u32 a1, a1, 8;\n\tadd.u64 b1, b1, %3;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], [a1], b1, %4, q;\n\t"
        "add.u32 a1, a1, 8;\n\tadd.u64 b1, b1, %3;\n\ttcgen05.mma.cta_group::2.kind::f16 [%0], [a1], b1, %4, q;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "l"(bstep), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrival on a barrier of either block (address from mapa).  What it announces
// are tensor-memory accesses, complete and ordered by the tcgen05 fence in front;
// the cluster-scope release of mbar_arrive_remote_release would order all of the
// thread's memory traffic as well and took 800 cycles a stage.
__device__ __forceinline__ void pair_arrive(uint32_t addr)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// Wait of a whole warp for arrivals that may come from the other block; the
// lanes leave together, as in warp_wait.
__device__ __forceinline__ bool pair_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool pair_wait(uint32_t bar, uint32_t parity)
{
    bool ok = __all_sync(0xffffffffu, pair_try(bar, parity));
    if (!ok) {
        uint64_t t0 = 0;
#pragma unroll 1
        for (uint32_t i = 1; !ok; ++i) {
            ok = __all_sync(0xffffffffu, pair_try(bar, parity));
            if (!ok && (i & 31u) == 0u) {
                const uint64_t now = globaltimer_ns();
                if (i == 32u) t0 = now;
                else if (__any_sync(0xffffffffu, now - t0 > kG8WaitNs)) break;
            }
        }
    }
    __syncwarp();
    return ok;
}

// Outputs of one weight row and the tokens m0 + 16 b + i (16 b < cols); clears acc.
// sx: lane l holds the scales of tokens m0 + 32 j + l.
template <int YT>
__device__ __forceinline__ void pair_emit(const Gemm8Args& A, int (&acc)[6][16], int m0, int cols, int row, float sw, float bv,
                                          const float (&sx)[3])
{
    const bool have = row < A.N;
#pragma unroll
    for (int b = 0; b < 6; ++b) {
        if (16 * b < cols) {
            const int mb = m0 + 16 * b;
            const size_t at = static_cast<size_t>(mb) * A.N + row;
            if (A.residual != nullptr) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    // the residuals before their stores: y may be the residual itself
                    float r[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        r[i] = have && mb + 8 * g + i < A.M ? A.residual[at + static_cast<size_t>(8 * g + i) * A.N] : 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float s = __shfl_sync(0xffffffffu, sx[b >> 1], 16 * (b & 1) + 8 * g + i);
                        const float v = __fadd_rn(r[i], __fmaf_rn(__fmul_rn(sw, s), __int2float_rn(acc[b][8 * g + i]), bv));
                        if (have && mb + 8 * g + i < A.M) store_typed(A.y, YT, at + static_cast<size_t>(8 * g + i) * A.N, v);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float s = __shfl_sync(0xffffffffu, sx[b >> 1], 16 * (b & 1) + i);
                    const float v = __fmaf_rn(__fmul_rn(sw, s), __int2float_rn(acc[b][i]), bv);
                    if (have && mb + i < A.M) store_typed(A.y, YT, at + static_cast<size_t>(i) * A.N, v);
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[b][i] = 0;
        }
    }
}

__global__ void __launch_bounds__(kP8Threads, 1) gemm_w8_pair_kernel(const __grid_constant__ Gemm8Args A)
{
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = A.stages, nt = A.nt;                            // nt: this block's tokens, half of the tile's
    const Pair8Smem L = pair8_smem(S, nt);
    const int slot_bytes = kG8WBytes + nt * 64 * kG8StageChunks;
    const uint32_t bars = smem_u32(smem + L.bars);
    const uint32_t full_b = bars;                                  // [S] this block's stage landed
    const uint32_t empty_b = full_b + 8 * kP8MaxStages;            // [S] read by the MMAs (both blocks)
    const uint32_t ready_b = empty_b + 8 * kP8MaxStages;           // [kP8ABufs] in the first block: half converted in both
    const uint32_t free_b = ready_b + 8 * kP8ABufs;                // [kP8ABufs] half read by the MMAs (both blocks)
    const uint32_t accf_b = free_b + 8 * kP8ABufs;                 // [2] accumulator complete (both blocks)
    const uint32_t acce_b = accf_b + 16;                           // [2] in the first block: accumulator read in both
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L.tmem);
    const uint32_t rank = cluster_ctarank();
    const int pair = static_cast<int>(blockIdx.x) >> 1, pairs = static_cast<int>(gridDim.x) >> 1;
    const int ntiles = A.n_g * A.n_tt;                             // n_g: groups of 256 rows
    const int nst = (A.C + kG8StageChunks - 1) / kG8StageChunks;

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_b + 8 * s, 1);
            mbar_init(empty_b + 8 * s, 1);
        }
        for (int j = 0; j < kP8ABufs; ++j) {
            mbar_init(ready_b + 8 * j, 8);
            mbar_init(free_b + 8 * j, 1);
        }
        for (int j = 0; j < 2; ++j) {
            mbar_init(accf_b + 8 * j, 1);
            mbar_init(acce_b + 8 * j, 16);
        }
        fence_mbar_init();
    }
    __syncwarp();
    if (warp == 1) pair_alloc(smem_u32(tmem_slot), kG8TmemCols);
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                                // both blocks' barriers and tensor memory are there
    tc_fence_after();
    // the next kernel's blocks may come only once this one holds its tensor memory
    pdl_launch_dependents();
    const uint32_t tbase = *tmem_slot;
    const uint32_t col_a = 4u * static_cast<uint32_t>(nt);         // two accumulators of 2 nt columns, then A
    auto fail = [&]() {
        if (lane == 0 && A.err != nullptr) atomicExch(A.err, kErrWaitTimeout);
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0) {
            // --------------------------------------------------- copy warp
            const uint64_t pol = l2_policy_evict_first(), pol_b = l2_policy_evict_last();
            auto copy_w = [&](int row_tile, int st, int slot) {
                if (elect_one()) {
                    const uint32_t bar = full_b + 8 * slot;
                    const int k8 = 4 * min(kG8StageChunks, A.C - st * kG8StageChunks);
                    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(kG8WBytes + k8 * nt * 16));
                    tma_load_2d(smem_u32(smem + L.ring) + static_cast<uint32_t>(slot * slot_bytes), &A.wmap,
                                st * kG8StageChunks * 32, row_tile, bar, pol);
                }
                __syncwarp();
            };
            // the first tile's weights do not depend on the previous kernel
            int ahead = 0;
            if (pair < ntiles)
                for (; ahead < S && ahead < nst; ++ahead)
                    copy_w((2 * (pair / A.n_tt) + static_cast<int>(rank)) * (kG8Rows / kRows), ahead, ahead);
            pdl_wait();
            int it = 0, slot = 0;
            uint32_t ph = 1u;
            bool ok = true;
            for (int tile = pair; tile < ntiles && ok; tile += pairs) {
                const int g = tile / A.n_tt;
                const int row_tile = (2 * g + static_cast<int>(rank)) * (kG8Rows / kRows);
                const uint4* codes = A.xh + static_cast<size_t>(2 * (tile - g * A.n_tt) + static_cast<int>(rank)) * (A.K >> 3) * nt;
                for (int st = 0; st < nst; ++st, ++it) {
                    if (it >= S) {
                        ok = pair_wait(empty_b + 8 * slot, ph);
                        if (!ok) {
                            fail();
                            break;
                        }
                    }
                    if (it >= ahead) copy_w(row_tile, st, slot);
                    if (elect_one()) {
                        const int k8 = 4 * min(kG8StageChunks, A.C - st * kG8StageChunks);
                        bulk_g2s(smem_u32(smem + L.ring) + static_cast<uint32_t>(slot * slot_bytes + kG8WBytes),
                                 codes + static_cast<size_t>(st * kG8StageChunks * 4) * nt, static_cast<uint32_t>(k8 * nt * 16),
                                 full_b + 8 * slot, pol_b);
                    }
                    __syncwarp();
                    if (++slot == S) {
                        slot = 0;
                        ph ^= 1u;
                    }
                }
            }
            // every copy has landed before the block ends (also after a failure)
            for (int k = max(0, it - S); k < it; ++k)
                if (!warp_wait(full_b + 8 * (k % S), static_cast<uint32_t>(k / S) & 1u)) break;
        } else if (warp == 1 && rank == 0) {
            // ---------------------------------------------------- MMA warp
            const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(2 * nt >> 3) << 17) | (16u << 24);   // M = 256
            // core matrices of 8 tokens x 8 K (128 B): token groups 128 B apart, K groups nt * 16 B
            const uint64_t bdesc0 = smem_desc_noswizzle(smem_u32(smem + L.ring) + kG8WBytes, static_cast<uint32_t>(nt * 16), 128u);
            const uint64_t bstep = static_cast<uint64_t>(2 * nt), bslot = static_cast<uint64_t>(slot_bytes >> 4);
            uint64_t bdesc = bdesc0;
            int it = 0, ac = 0, slot = 0;
            bool ok = true;
            for (int tile = pair; tile < ntiles && ok; tile += pairs) {
                int run = 0;
                for (int st = 0; st < nst && ok; ++st, ++it) {
                    const bool last = st + 1 == nst || run == kG8AccStages - 1;
                    const uint32_t dcol = tbase + static_cast<uint32_t>((ac & 1) * 2 * nt);
                    const int k16 = 2 * min(kG8StageChunks, A.C - st * kG8StageChunks);
                    if (run == 0 && ac >= 2) ok = pair_wait(acce_b + 8 * (ac & 1), static_cast<uint32_t>((ac >> 1) - 1) & 1u);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int j = (2 * it + h) & (kP8ABufs - 1);
                        // converted in both blocks, so the codes have landed in both
                        ok = ok && pair_wait(ready_b + 8 * j, static_cast<uint32_t>((2 * it + h) / kP8ABufs) & 1u);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint32_t acol = tbase + col_a + static_cast<uint32_t>(j * kP8ACols);
                            const uint64_t bd = bdesc + static_cast<uint64_t>(4 * h) * bstep;
                            const uint32_t more = run == 0 && h == 0 ? 0u : 1u;
                            if (k16 >= 4 * h + 4) {
                                pair_mma_x4(dcol, acol, bd, bstep, idesc, more);
                            } else {
                                for (int kk = 0; kk < k16 - 4 * h; ++kk)
                                    pair_mma(dcol, acol + 8 * kk, bd + static_cast<uint64_t>(kk) * bstep, idesc, kk == 0 ? more : 1u);
                            }
                            pair_commit(free_b + 8 * j);
                            if (h == 1) {
                                pair_commit(empty_b + 8 * slot);
                                if (last) pair_commit(accf_b + 8 * (ac & 1));
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) {
                        fail();
                        break;
                    }
                    ++run;
                    if (last) {
                        ++ac;
                        run = 0;
                    }
                    bdesc += bslot;
                    if (++slot == S) {
                        slot = 0;
                        bdesc = bdesc0;
                    }
                }
            }
            // every MMA has completed before the tensor memory is freed
            if (it > 0) pair_wait(empty_b + 8 * ((it - 1) % S), static_cast<uint32_t>((it - 1) / S) & 1u);
        }
    } else if (warp < kP8Epi) {
        // ------------------------------------------------ converting warps
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const int grp = (warp - kP8Conv) >> 2;
        const int row = (warp & 3) * 32 + lane;                    // tensor-memory lane and weight row of the block
        const uint32_t tlane = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint8_t* units = smem + L.ring + (row >> 3) * (256 * kG8StageChunks) + (row & 7) * 32 + grp * 512;
        const uint32_t ready0 = mapa_shared(ready_b, 0);
        int it = 0, slot = 0;
        uint32_t sph = 0u;
        bool ok = true;
        for (int tile = pair; tile < ntiles && ok; tile += pairs) {
            for (int st = 0; st < nst; ++st, ++it) {
                const int nch = min(2, A.C - st * kG8StageChunks - 2 * grp);    // chunks of this half
                const int q = 2 * it + grp, j = q & (kP8ABufs - 1);
                ok = warp_wait(full_b + 8 * slot, sph);
                ok = ok && (q < kP8ABufs || pair_wait(free_b + 8 * j, static_cast<uint32_t>(q / kP8ABufs - 1) & 1u));
                if (!ok) {
                    fail();
                    break;
                }
                tc_fence_after();
                const uint8_t* u = units + slot * slot_bytes;
                uint4 a[2], b[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    a[e] = *reinterpret_cast<const uint4*>(u + e * 256);          // (two lanes to a bank, as in gemm_w8.cu)
                    b[e] = *reinterpret_cast<const uint4*>(u + e * 256 + 16);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (e < nch) {
                        uint32_t h[16];
                        unit_f16(a[e], b[e], h);
                        tmem_st16(tbase + tlane + col_a + static_cast<uint32_t>(kP8ACols * j + 16 * e), h);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) pair_arrive(ready0 + 8 * j);
                __syncwarp();
                if (++slot == S) {
                    slot = 0;
                    sph ^= 1u;
                }
            }
        }
    } else {
        // -------------------------------------------------- epilogue warps
        asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
        const int half = (warp - kP8Epi) >> 2;                     // columns half * nt ..
        const uint32_t tlane = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t acce0 = mapa_shared(acce_b, 0);
        int acc[6][16];                                            // columns half * nt + 16 b + i of this thread's row
#pragma unroll
        for (int b = 0; b < 6; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[b][i] = 0;
        int ac = 0;
        bool ok = true;
        pdl_wait();
        for (int tile = pair; tile < ntiles && ok; tile += pairs) {
            const int g = tile / A.n_tt;
            const int row = (2 * g + static_cast<int>(rank)) * kG8Rows + (warp & 3) * 32 + lane;
            const float sw = row < A.N ? __ldg(A.s_w + row) : 0.0f;
            const float bv = row < A.N && A.bias != nullptr ? __ldg(A.bias + row) : 0.0f;
            const int m0 = (2 * (tile - g * A.n_tt) + half) * nt;
            float sx[3];
#pragma unroll
            for (int j = 0; j < 3; ++j) sx[j] = m0 + 32 * j + lane < A.M ? __ldg(A.sx + m0 + 32 * j + lane) : 0.0f;
            for (int st = 0; st < nst; st += kG8AccStages, ++ac) {
                ok = pair_wait(accf_b + 8 * (ac & 1), static_cast<uint32_t>(ac >> 1) & 1u);
                if (!ok) {
                    fail();
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < 6; ++b) {
                    if (16 * b < nt) {
                        uint32_t d[16];
                        tmem_ld16(tbase + tlane + static_cast<uint32_t>((ac & 1) * 2 * nt + half * nt + 16 * b), d);
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[b][i] += __float2int_rn(__uint_as_float(d[i]));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) pair_arrive(acce0 + 8 * (ac & 1));
                __syncwarp();
            }
            if (!ok) break;
            if (A.ytype == T_F32) pair_emit<T_F32>(A, acc, m0, nt, row, sw, bv, sx);
            else if (A.ytype == T_F16) pair_emit<T_F16>(A, acc, m0, nt, row, sw, bv, sx);
            else pair_emit<T_BF16>(A, acc, m0, nt, row, sw, bv, sx);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                                // no arrival comes to a block that has left
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        pair_dealloc(tbase, kG8TmemCols);
    }
}

}  // namespace

cudaError_t launch_gemm_w8_pair(Gemm8Args& a, int grid, size_t smem, bool pdl, cudaStream_t s)
{
    auto kern = gemm_w8_pair_kernel;
    static SmemLimit limit;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), limit, smem);
    if (e == cudaSuccess) e = encode_w8_map(a);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kP8Threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (pdl) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = 2;
    attr[na].val.clusterDim.y = 1;
    attr[na].val.clusterDim.z = 1;
    ++na;
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(na);
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace w4k
