// INT8 x INT8 matrix product with a scale for each token and each output
// channel, for any number of tokens, on the 5th-generation tensor cores:
//   acc[m][j] = sum_i q_w[j][i] q_x[m][i]   (exact),
//   y[m][j]   = fma(fp32(s_w[j] s_x[m]), fp32(acc), b[j]) (+ residual), rounded to y's type.
//
// The chip's integer tensor rate is far below its fp16 rate, and an int8 value
// is an fp16 value exactly, so the product runs on tcgen05.mma kind::f16: a
// product is at most 2^14, 1024 of them at most 2^24, so an fp32 accumulator
// over 1024 K holds the integer sum exactly; each accumulator is then added
// into int32 registers while the tensor cores fill the other one.
//   * A (128 weight rows) streams as int8, is converted by eight warps (XOR,
//     byte permute, one fp16 subtraction) and stored into tensor memory, so a
//     weight costs one byte of HBM, L2 and shared-memory traffic.  The
//     repacked layout (8-row tiles of 32-byte units) is read as it is: the
//     same bytes serve every path of the format.
//   * B (up to 128 tokens) comes as fp16 codes in the layout that the row
//     quantizer writes: a K group of eight of a token tile is one contiguous
//     run, copied by a 1-D bulk copy into the core-matrix layout without
//     swizzle.
//   * Persistent blocks, one per SM: a copy warp, an MMA warp, eight
//     converting warps (two groups on alternate slots of 128 K) and eight
//     epilogue warps, joined by mbarriers only.
//   * Few tiles: K is split over a thread-block cluster; the splits exchange
//     their integer sums through distributed shared memory (split r owns the
//     tokens c with c % splits = r), so every block writes a share of y.
// A stage of 128 K takes some 400 ns whatever the tokens of the tile: a group's
// way from the landing over the conversion to the arrival, twice as long, more
// than the MMAs.  16 tokens, 152064 x 3584: 92 us (6.03 TB/s, measured copy rate
// 6.79); 64 tokens, 3584 x 18944: 26.1 us with the quantizer; 333 tokens, 3584 x
// 3584: 22.9 us with it.
#include <cuda_fp16.h>

#include <atomic>

#include "gemm_w8.cuh"

namespace w4k {
namespace {

constexpr int kWarpMma = 1, kWarpConv = 2, kWarpEpi = 10;

// kind::f16 MMAs of one stage's K slices (A in tensor memory, eight columns to
// a slice; B from shared-memory descriptors `bstep` apart in the address
// field): eight in one statement, or one.
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tc_mma_f16_ts_x8(uint32_t d, uint32_t a, uint64_t b, uint64_t bstep, uint32_t idesc,
                                                 uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 a1;\n\t.reg .b64 b1;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 q, %5, %5;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u64 b1, %2, %3;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, q;\n\t"
        "add.u32 a1, a1, 8;\n\tadd.u64 b1, b1, %3;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, q;\n\t"
        "add.u32 a1, a1, 8;\n\tadd.u64 b1, b1, %3;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, q;\n\t"
        "add.u32 a1, a1, 8;\n\tadd.u64 b1, b1, %3;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, q;\n\t"
        "add.u32 a1, a1, 8;\n\tadd.u64 b1, b1, %3;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, q;\n\t"
        "add.u32 a1, a1, 8;\n\tadd.u64 b1, b1, %3;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, q;\n\t"
        "add.u32 a1, a1, 8;\n\tadd.u64 b1, b1, %3;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %4, q;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "l"(bstep), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Scales of a warp's tokens m + 32 b + i (b < 2, i < 16), token 16 b + i in lane 16 b + i.
__device__ __forceinline__ float sx_of(const Gemm8Args& A, int m, int lane)
{
    m += lane + (lane & 16);
    return m < A.M ? __ldg(A.sx + m) : 0.0f;
}

// Outputs of one weight row and the tokens m0 + 32 b + i (32 b < cols); clears acc.
template <int YT>
__device__ __forceinline__ void emit_tile(const Gemm8Args& A, int (&acc)[4][16], int m0, int cols, int row, float sw,
                                          float bv, float sx0, float sx1)
{
    const bool have = row < A.N;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        if (32 * b < cols) {
            const int mb = m0 + 32 * b;
            const size_t at = static_cast<size_t>(mb) * A.N + row;
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float sx = __shfl_sync(0xffffffffu, b < 2 ? sx0 : sx1, 16 * (b & 1) + i);
                v[i] = __fmaf_rn(__fmul_rn(sw, sx), __int2float_rn(acc[b][i]), bv);
                acc[b][i] = 0;
            }
            if (A.residual != nullptr) {
                // every residual before the first store: y may be the residual itself
                float r[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    r[i] = have && mb + i < A.M ? A.residual[at + static_cast<size_t>(i) * A.N] : 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __fadd_rn(r[i], v[i]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (have && mb + i < A.M) store_typed(A.y, YT, at + static_cast<size_t>(i) * A.N, v[i]);
        }
    }
}

__global__ void __launch_bounds__(kG8Threads, 1) gemm_w8_kernel(const __grid_constant__ Gemm8Args A)
{
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = A.stages, nt = A.nt, ks = A.splits;
    const Gemm8Smem L = gemm8_smem(S, nt, ks);
    const int slot_bytes = kG8WBytes + nt * 64 * kG8StageChunks;
    const uint32_t col_a = 2u * static_cast<uint32_t>(nt);        // two accumulators, then a converted stage per slot
    const uint32_t bars = smem_u32(smem + L.bars);
    const uint32_t full_b = bars;                                  // [S] stage landed
    const uint32_t empty_b = full_b + 8 * kG8MaxStages;            // [S] slot and converted stage read: MMA commit
    const uint32_t ready_b = empty_b + 8 * kG8MaxStages;           // [S] converted (four warps)
    const uint32_t accf_b = ready_b + 8 * kG8MaxStages;            // [2] accumulator complete
    const uint32_t acce_b = accf_b + 16;                           // [2] accumulator read (eight warps)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L.tmem);
    volatile uint32_t* dead_s = tmem_slot + 1;

    const int rank = ks > 1 ? static_cast<int>(blockIdx.x) % ks : 0;
    const int tile_first = static_cast<int>(blockIdx.x) / ks;
    const int tile_step = static_cast<int>(gridDim.x) / ks;
    const int ntiles = A.n_g * A.n_tt;
    const int nst = (A.C + kG8StageChunks - 1) / kG8StageChunks;
    const int st0 = static_cast<int>(static_cast<long long>(rank) * nst / ks);
    const int st1 = static_cast<int>(static_cast<long long>(rank + 1) * nst / ks);

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full_b + 8 * s, 1);
            mbar_init(empty_b + 8 * s, 1);
            mbar_init(ready_b + 8 * s, 4);
        }
        for (int j = 0; j < 2; ++j) {
            mbar_init(accf_b + 8 * j, 1);
            mbar_init(acce_b + 8 * j, 8);
        }
        fence_mbar_init();
        *dead_s = 0u;
    }
    __syncwarp();
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(tmem_slot), kG8TmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // The next kernel's blocks may come only once this one holds its tensor memory.  (All of it: blocks that wait for tensor
    // memory on an SM wait for this one to end.  None of the library's is beside it there: 143 KB of shared memory at
    // least here, 106 KB at least in gemv_tc.cu, of 228 KB.)
    pdl_launch_dependents();
    if (ks > 1) cluster_sync();          // the other splits' shared memory is there
    const uint32_t tbase = *tmem_slot;
    auto fail = [&]() {
        *dead_s = 1u;
        if (A.err != nullptr) atomicExch(A.err, kErrWaitTimeout);
    };
    if (warp == 0) {
        // ------------------------------------------------------- copy warp
        const uint64_t pol = l2_policy_evict_first(), pol_b = l2_policy_evict_last();
        auto copy_w = [&](int row_tile, int st, int slot) {
            if (elect_one()) {
                const uint32_t bar = full_b + 8 * slot;
                const int k8 = 4 * min(kG8StageChunks, A.C - st * kG8StageChunks);
                mbar_arrive_expect_tx(bar, static_cast<uint32_t>(kG8WBytes + k8 * nt * 16));
                // 16 row tiles x 128 K; tiles past T and chunks past C arrive as zeros
                tma_load_2d(smem_u32(smem + L.ring) + static_cast<uint32_t>(slot * slot_bytes), &A.wmap,
                            st * kG8StageChunks * 32, row_tile, bar, pol);
            }
            __syncwarp();
        };
        auto copy_b = [&](const uint4* codes, int st, int slot) {
            if (elect_one()) {
                const int k8 = 4 * min(kG8StageChunks, A.C - st * kG8StageChunks);
                bulk_g2s(smem_u32(smem + L.ring) + static_cast<uint32_t>(slot * slot_bytes + kG8WBytes),
                         codes + static_cast<size_t>(st * kG8StageChunks * 4) * nt, static_cast<uint32_t>(k8 * nt * 16),
                         full_b + 8 * slot, pol_b);
            }
            __syncwarp();
        };
        // the first tile's weights do not depend on the previous kernel
        int ahead = 0;
        if (tile_first < ntiles)
            for (; ahead < S && st0 + ahead < st1; ++ahead)
                copy_w((tile_first / A.n_tt) * (kG8Rows / kRows), st0 + ahead, ahead);
        pdl_wait();
        int it = 0, slot = 0;
        uint32_t ph = 1u;                // parity of the slot's previous release
        bool ok = true;
        for (int tile = tile_first; tile < ntiles && ok; tile += tile_step) {
            const int g = tile / A.n_tt;
            const int row_tile = g * (kG8Rows / kRows);
            const uint4* codes = A.xh + static_cast<size_t>(tile - g * A.n_tt) * (A.K >> 3) * nt;
            for (int st = st0; st < st1; ++st, ++it) {
                if (it >= ahead) {
                    if (it >= S) {
                        ok = warp_wait(empty_b + 8 * slot, ph);
                        if (!ok) {
                            if (lane == 0) fail();
                            break;
                        }
                    }
                    copy_w(row_tile, st, slot);
                }
                copy_b(codes, st, slot);
                if (++slot == S) {
                    slot = 0;
                    ph ^= 1u;
                }
            }
        }
        // every copy has landed before the block ends (also after a failure)
        for (int k = max(0, it - S); k < it; ++k)
            if (!warp_wait(full_b + 8 * (k % S), static_cast<uint32_t>(k / S) & 1u)) break;
    } else if (warp == kWarpMma) {
        // -------------------------------------------------------- MMA warp
        const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(nt >> 3) << 17) | (static_cast<uint32_t>(kG8Rows >> 4) << 24);
        int it = 0, ac = 0, slot = 0;
        uint32_t sph = 0u;
        bool ok = true;
        // core matrices of 8 tokens x 8 K (128 B): token groups 128 B apart, K groups nt * 16 B
        const uint64_t bdesc0 = smem_desc_noswizzle(smem_u32(smem + L.ring) + kG8WBytes, static_cast<uint32_t>(nt * 16), 128u);
        const uint64_t bstep = static_cast<uint64_t>(2 * nt);          // 16 K in the descriptor's address field
        const uint64_t bslot = static_cast<uint64_t>(slot_bytes >> 4);
        uint64_t bdesc = bdesc0;
        uint32_t acol = tbase + col_a;
        for (int tile = tile_first; tile < ntiles && ok; tile += tile_step) {
            int run = 0;                 // stages in the current accumulator
            for (int st = st0; st < st1; ++st, ++it) {
                const bool last = st + 1 == st1 || run == kG8AccStages - 1;
                const uint32_t dcol = tbase + static_cast<uint32_t>((ac & 1) * nt);
                if (run == 0 && ac >= 2) ok = warp_wait(acce_b + 8 * (ac & 1), static_cast<uint32_t>((ac >> 1) - 1) & 1u);
                // converted, so landed: the converting warps saw the codes land with the weights (a wait of this warp for
                // them as well took 8% of the 16-token lm_head)
                ok = ok && warp_wait(ready_b + 8 * slot, sph);
                if (!ok) {
                    if (lane == 0) fail();
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t more = run == 0 ? 0u : 1u;
                    if ((st + 1) * kG8StageChunks <= A.C) {
                        tc_mma_f16_ts_x8(dcol, acol, bdesc, bstep, idesc, more);
                    } else {
                        const int k16 = 2 * (A.C - st * kG8StageChunks);
                        for (int kk = 0; kk < k16; ++kk)
                            tc_mma_f16_ts(dcol, acol + 8 * kk, bdesc + static_cast<uint64_t>(kk) * bstep, idesc, kk == 0 ? more : 1u);
                    }
                    tc_commit(empty_b + 8 * slot);
                    if (last) tc_commit(accf_b + 8 * (ac & 1));
                }
                __syncwarp();
                ++run;
                if (last) {
                    ++ac;
                    run = 0;
                }
                bdesc += bslot;
                acol += kG8ACols;
                if (++slot == S) {
                    slot = 0;
                    sph ^= 1u;
                    bdesc = bdesc0;
                    acol = tbase + col_a;
                }
            }
        }
        // every MMA has completed before the tensor memory is freed
        if (it > 0) warp_wait(empty_b + 8 * ((it - 1) % S), static_cast<uint32_t>((it - 1) / S) & 1u);
    } else if (warp >= kWarpConv && warp < kWarpEpi) {
        // ------------------------------------------------ converting warps
        const int grp = (warp - kWarpConv) >> 2;
        const int row = (warp & 3) * 32 + lane;                    // tensor-memory lane and weight row of the tile
        const uint32_t tlane = static_cast<uint32_t>((warp & 3) * 32) << 16;
        int it = 0, slot = 0;
        uint32_t sph = 0u;
        bool ok = true;
        for (int tile = tile_first; tile < ntiles && ok; tile += tile_step) {
            for (int st = st0; st < st1; ++st, ++it) {
                // A group has its slots to itself (not every other stage: with an odd number of slots the groups would
                // take turns on a slot, and the one that is ahead could take a landing of the turn before last, whose
                // parity is the same, for its own)
                if ((slot & 1) == grp) {
                    // the slot's refill follows the MMAs that read its last converted
                    // stage, so a landed stage also has its tensor-memory columns free
                    const int nch = min(kG8StageChunks, A.C - st * kG8StageChunks);
                    ok = warp_wait(full_b + 8 * slot, sph);
                    if (!ok) {
                        if (lane == 0) fail();
                        break;
                    }
                    tc_fence_after();
                    const uint8_t* u = smem + L.ring + slot * slot_bytes + (row >> 3) * (256 * kG8StageChunks) + (row & 7) * 32;
                    uint4 a[kG8StageChunks], b[kG8StageChunks];
#pragma unroll
                    for (int e = 0; e < kG8StageChunks; ++e) {
                        // (two lanes to a bank; reading every other row's halves the other way round would spread them, but the
                        // selects that put the halves back took more: 16-token lm_head 93.6 against 91.5 us)
                        a[e] = *reinterpret_cast<const uint4*>(u + e * 256);
                        b[e] = *reinterpret_cast<const uint4*>(u + e * 256 + 16);
                    }
#pragma unroll
                    for (int e = 0; e < kG8StageChunks; ++e) {
                        if (e < nch) {
                            uint32_t h[16];
                            unit_f16(a[e], b[e], h);
                            tmem_st16(tbase + tlane + col_a + static_cast<uint32_t>(kG8ACols * slot + 16 * e), h);
                        }
                    }
                    // (the reads of the slot are ordered before the copy that refills it)
                    fence_proxy_async_smem();
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ready_b + 8 * slot);
                    __syncwarp();
                }
                if (++slot == S) {
                    slot = 0;
                    sph ^= 1u;
                }
            }
        }
    } else if (warp >= kWarpEpi) {
        // -------------------------------------------------- epilogue warps
        const int half = (warp - kWarpEpi) >> 2;
        const uint32_t tlane = static_cast<uint32_t>((warp & 3) * 32) << 16;
        int acc[4][16];                  // token columns 32 b + 16 half + i of this thread's row
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[b][i] = 0;
        int ac = 0;
        bool ok = true;
        pdl_wait();
        for (int tile = tile_first; tile < ntiles && ok; tile += tile_step) {
            const int g = tile / A.n_tt;
            const int row = g * kG8Rows + (warp & 3) * 32 + lane;
            const float sw = row < A.N ? __ldg(A.s_w + row) : 0.0f;
            const float bv = row < A.N && A.bias != nullptr ? __ldg(A.bias + row) : 0.0f;
            for (int st = st0; st < st1; st += kG8AccStages, ++ac) {
                ok = warp_wait(accf_b + 8 * (ac & 1), static_cast<uint32_t>(ac >> 1) & 1u);
                if (!ok) {
                    if (lane == 0) fail();
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (32 * b + 16 * half < nt) {
                        uint32_t d[16];
                        tmem_ld16(tbase + tlane + static_cast<uint32_t>((ac & 1) * nt + 32 * b + 16 * half), d);
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[b][i] += __float2int_rn(__uint_as_float(d[i]));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(acce_b + 8 * (ac & 1));
                __syncwarp();
            }
            if (ks > 1 || !ok) break;
            const int m0 = (tile - g * A.n_tt) * nt + 16 * half;
            const float sx0 = sx_of(A, m0, lane), sx1 = sx_of(A, m0 + 64, lane);
            if (A.ytype == T_F32) emit_tile<T_F32>(A, acc, m0, nt - 16 * half, row, sw, bv, sx0, sx1);
            else if (A.ytype == T_F16) emit_tile<T_F16>(A, acc, m0, nt - 16 * half, row, sw, bv, sx0, sx1);
            else emit_tile<T_BF16>(A, acc, m0, nt - 16 * half, row, sw, bv, sx0, sx1);
        }
        if (ks > 1) {
            // token column c of the tile belongs to split c % ks: its sums go there
            const int lg = 31 - __clz(ks), per = nt >> lg;              // (a power of two)
            const uint32_t red_u = smem_u32(smem + L.red);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (32 * b + 16 * half < nt) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int c = 32 * b + 16 * half + i;
                        const int o = (rank * per + (c >> lg)) * kG8Rows + (warp & 3) * 32 + lane;
                        st_cluster_u32(mapa_shared(red_u + 4u * static_cast<uint32_t>(o), static_cast<uint32_t>(c & (ks - 1))),
                                       static_cast<uint32_t>(acc[b][i]));
                    }
                }
            }
        }
    }
    __syncwarp();

    // ---- K splits: this split's columns, summed in order of the splits
    if (ks > 1) {
        const int per = nt / ks;
        const int* red = reinterpret_cast<const int*>(smem + L.red);
        // a row and every fourth of the columns to a thread
        static_assert(kG8Rows == 128 && kG8Threads >= 512, "threads for the exchange");
        const int r = tid & (kG8Rows - 1), c0 = tid >> 7;
        const int row = (tile_first / A.n_tt) * kG8Rows + r;
        const int m0 = (tile_first % A.n_tt) * nt + rank;
        const bool mine = tid < 512 && row < A.N;
        pdl_wait();
        const float sw = mine ? __ldg(A.s_w + row) : 0.0f;
        const float bv = mine && A.bias != nullptr ? __ldg(A.bias + row) : 0.0f;
        cluster_sync();
        const bool dead = *dead_s != 0u;
#pragma unroll 4
        for (int c = c0; c < per; c += 4) {
            const int m = m0 + c * ks;
            if (mine && m < A.M && !dead) {
                int s = 0;
                for (int q = 0; q < ks; ++q) s += red[(q * per + c) * kG8Rows + r];
                float v = __fmaf_rn(__fmul_rn(sw, __ldg(A.sx + m)), __int2float_rn(s), bv);
                const size_t o = static_cast<size_t>(m) * A.N + row;
                if (A.residual != nullptr) v = __fadd_rn(A.residual[o], v);
                store_typed(A.y, A.ytype, o, v);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tbase, kG8TmemCols);
    }
}

}  // namespace

// The weights as a 2-D array of 8-byte elements: a row per 8-row tile (C
// chunks of 256 bytes), a box of 16 tiles x one stage.
cudaError_t encode_w8_map(Gemm8Args& a)
{
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<void*> cached{nullptr};
    void* fn = cached.load(std::memory_order_acquire);
    if (fn == nullptr) {
        cudaDriverEntryPointQueryResult got;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &got);
        if (e != cudaSuccess) return e;
        if (got != cudaDriverEntryPointSuccess || fn == nullptr) return cudaErrorNotSupported;
        cached.store(fn, std::memory_order_release);
    }
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.C) * 32, static_cast<cuuint64_t>(a.T)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.C) * 256};
    const cuuint32_t box[2] = {32 * kG8StageChunks, kG8Rows / kRows};
    const cuuint32_t ones[2] = {1, 1};
    const CUresult r = reinterpret_cast<Encode>(fn)(
        &a.wmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, 2, const_cast<uint8_t*>(a.w), dims, strides, box, ones,
        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_gemm_w8(Gemm8Args& a, int grid, size_t smem, bool pdl, cudaStream_t s)
{
    auto kern = gemm_w8_kernel;
    static SmemLimit limit;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), limit, smem);
    if (e == cudaSuccess) e = encode_w8_map(a);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kG8Threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (pdl) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    if (a.splits > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = static_cast<unsigned>(a.splits);
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    cfg.attrs = na > 0 ? attr : nullptr;
    cfg.numAttrs = static_cast<unsigned>(na);
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace w4k
