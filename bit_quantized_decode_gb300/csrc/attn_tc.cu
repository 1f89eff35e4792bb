// Attention of many rows over a paged cache on the 5th-generation tensor
// cores: a wide draft tree times a key head's group gives up to some hundred
// rows for the same keys, more than mma.sync keeps up with while the cache
// streams (see attn_tree.cu, which takes calls of few rows and defines the
// operation and the layout of the work).
//
// A block takes a tile of 128 rows of one (sequence, key head) over 64 cached
// tokens at a time:
//   S = Q K^T   tcgen05.mma 128 x 64 x D: K in shared memory as TMA's 128-byte
//               swizzle lays it, Q in tensor memory (heads of 256 with an fp32
//               output, for which that has no room, in shared memory: an MMA of 128 x 64 x 16 then takes 62 cycles,
//               bound by reading Q), S in tensor memory (the next product runs
//               during the softmax, into a second buffer or, heads of 256, when the first is read);
//   softmax     two threads per row (tensor-memory lane), 32 tokens each; they
//               exchange their maxima.  The maximum in use is raised only when it
//               is passed by more than 2^12 (fp16 values: 2^6): probabilities are then at most
//               4096 (exact scaling, the sums stay in fp32), and the output, which
//               lies in tensor memory, is rescaled a few times per segment
//               instead of once per tile;
//   O += P V    P goes back to tensor memory in 16 bits (in parts, as there)
//               and is the A operand; V as it lies, 64 values of a token in a
//               row, is an operand with its columns contiguous.  Over long
//               contexts O is taken out now and then and summed in fp32: see kFlushParts.
// Warps: one orders copies, one issues MMAs, eight take the softmax; for an INT8
// cache eight widen codes to 16 bits (exact) in shared memory.  All
// are joined by mbarriers with bounded waits.
//
// A tile of 128 rows by 64 tokens takes 1330 cycles with one part to a probability, the softmax's time (maximum and exchange 400,
// exponentials 400, the way from the scores' arrival to P's 1100 in all); its MMAs take 530, its bytes 1470 at the SM's share of
// the memory rate (bf16, heads of 128).  Three parts (fp32 outputs) take 1850.  16 drafts of 28 heads over 4096 bf16 places, fp32
// outputs: 16.9 us, over 131071 73 (70 if sums stay in tensor memory); 8 x 64 drafts over 2800 to 4000 places, two parts: 60 (52
// with one, tensor pipe 28% active then).  INT8 with heads of 256, one part: 2700 cycles a tile (its bytes take 1480) with no
// resource full (issue slots 50%, tensor pipe 25%, DRAM 26% of the time): a tile's way from codes to 16 bits, scores, softmax and
// product, of which two 16-bit tiles and one place for scores let little overlap; warps wait for loads most.  5 drafts of 8 heads
// over 120001 places, two parts: 41 us, over a bf16 cache 40.
#include "attn_tree.cuh"
#include "gemm_w8.cuh"

namespace w4k {
namespace {

constexpr int kTcRows = kAtTcRows, kTcUnit = kAtTcUnit;
constexpr int kConvWarps = 8;                   // warps 2, 3, 12 .. 17: four for keys, four for values
// Tiles whose products add up in tensor memory before the sum is taken out, so that the error stops growing with the context: the
// tensor cores cut a sum's low bits at every step, always towards zero.  Values that are all positive, fp32 outputs (12 steps a
// tile of three parts), 25 to 100 tiles to a block: 0.9e-6 to 3.2e-6 off with 8, 1.4e-6 to 6.6e-6 with 16, 2.9e-6 to 13e-6 with 32.
// 16 drafts over 131071 places: 78, 73, 72 us, 70 without; over 65536 48, 45, 43, 43, INT8 68, 56, 54, 54.
constexpr int kFlushParts = 16;
// 16-bit outputs: 0.4e-6 a tile and part.  One part, 2048 tiles to a block: 8.3e-4 (3.4 half steps of fp16); 1.0e-4 with 256,
// 0.2e-4 with 64.  16 drafts of 8 sequences over 131071 places, 431 tiles to a block, one part of bf16: 322 us without, 328 with
// 256, 347 with 64, INT8 420, 440, 486.  The code alone costs 8 x 64 drafts over 4096 places 52.5 -> 53.8, so calls in which no
// block can have more than 128 tiles of a segment do without.
constexpr int kFlushLate = 128;

template <int D, int CT, int kParts>
struct Tc {
    static constexpr bool kI8 = CT == T_I8;
    static constexpr int kBoxes = D / 64;                     // 128-byte column groups of 16-bit values
    static constexpr bool kQInT = D <= 128 || kParts < 3;     // queries in tensor memory
    static constexpr int kSBufs = D == 256 && kQInT ? 1 : 2;  // places for the scores
    static constexpr int kQ = kQInT ? 0 : kTcRows * D * 2;
    static constexpr int kHalf = kTcUnit * D * 2;             // a tile's keys (or values) in 16 bits
    static constexpr int kRaw = kTcUnit * D;                  // the same in codes
    static constexpr int kStages = kI8 ? (D == 64 ? 14 : D == 128 ? 7 : 2) : (D == 64 ? 10 : D == 128 ? 6 : kQInT ? 3 : 2);   // copies
    static constexpr int kConv = kI8 ? (D == 256 && !kQInT ? 1 : 2) : kStages;   // 16-bit tiles
    static constexpr int kMeta = kStages + kConv + 2;         // tiles between the order of a tile's keys and the end of its softmax, at most
    static constexpr int kThreads = kI8 ? 384 + 32 * (kConvWarps - 2) : 384;
    static constexpr int kPBufs = D == 256 ? (kParts == 1 ? 2 : 1) : kParts < 3 ? 3 : 2;              // places for P
    static constexpr int kCols = 512;
    static constexpr int cS = D, cP = D + kSBufs * kTcUnit, cQ = D == 256 ? 384 : cP + 192;   // tensor-memory columns of S, P and Q; O begins at 0
    static_assert(!kQInT || cQ + D / 2 <= kCols, "tensor memory");
    static_assert(cP + kPBufs * 32 * kParts <= (kQInT ? cQ : kCols), "tensor memory");
    // shared memory
    static constexpr int oQ = 0;
    static constexpr int oKv = kQ;                            // [kConv] keys, values
    static constexpr int oRaw = oKv + kConv * 2 * kHalf;
    static constexpr int oScale = oRaw + (kI8 ? kStages * 2 * kRaw : 0);    // [kMeta][2][64]
    static constexpr int oMeta = oScale + (kI8 ? kMeta * 2 * kTcUnit * 4 : 0);   // [kMeta]: which sixteenths of a tile have a page; 16: a vast scale
    static constexpr int oTop = (oMeta + kMeta * 4 + 7) / 8 * 8;       // [2][2][128]: numbers of a row's halves with their turn, even and odd
    static constexpr int oBars = oTop + 4 * kTcRows * 8;
    static constexpr int nBars = 4 * kStages + 4 * kConv + 9;
    static constexpr int oMisc = oBars + nBars * 8;           // tensor memory's base, failure flag, odd values flag
    static constexpr int oWarpSum = oMisc + 16;
    static constexpr int oPre = oWarpSum + kThreads / 32 * 4;
    static constexpr int smem(int B) { return oPre + (B + 1) * 4 + 1024; }
    static_assert(smem(kAtMaxSeq) <= 232448, "shared memory of a block");
    // (all of tensor memory: no other block of this library that takes some may be on the SM; the least of them has 106 KB)
    static_assert(smem(1) > 123 * 1024, "alone with its tensor memory on an SM");
};

// Shared-memory matrix descriptors with the 128-byte swizzle.  Rows of 128 bytes
// (64 values of K): groups of eight rows are 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_rows(uint32_t a)
{
    return static_cast<uint64_t>((a & 0x3FFFFu) >> 4) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}
// Rows of 128 bytes that run along N: groups of eight K are 1024 bytes apart, groups of 64 N `lbo`.
__device__ __forceinline__ uint64_t desc_cols(uint32_t a, uint32_t lbo)
{
    return static_cast<uint64_t>((a & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// Four MMAs of 16 K each in one statement (the operands in uniform registers once): both operands in shared memory, 32 bytes
// of a row to a step; the first overwrites unless `accumulate`.
__device__ __forceinline__ void mma_ss_x4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a1, b1;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, %4, %4;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "add.u64 a1, %1, 2;\n\tadd.u64 b1, %2, 2;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, q;\n\t"
        "add.u64 a1, %1, 4;\n\tadd.u64 b1, %2, 4;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, q;\n\t"
        "add.u64 a1, %1, 6;\n\tadd.u64 b1, %2, 6;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, q;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// The same with A in tensor memory, eight columns to a step.
__device__ __forceinline__ void mma_ts_rows_x4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 a1;\n\t.reg .b64 b1;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 q, %4, %4;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u64 b1, %2, 2;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n\t"
        "add.u32 a1, %1, 16;\n\tadd.u64 b1, %2, 4;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n\t"
        "add.u32 a1, %1, 24;\n\tadd.u64 b1, %2, 6;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// The same with A in tensor memory (eight columns to a step) and B's rows along N (16 rows of 128 bytes to a step).
__device__ __forceinline__ void mma_ts_x4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\t.reg .b32 a1;\n\t.reg .b64 b1;\n\tsetp.eq.b32 q, %0, %0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, q;\n\t"
        "add.u32 a1, %1, 8;\n\tadd.u64 b1, %2, 128;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n\t"
        "add.u32 a1, %1, 16;\n\tadd.u64 b1, %2, 256;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n\t"
        "add.u32 a1, %1, 24;\n\tadd.u64 b1, %2, 384;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc)
        : "memory");
}

// A warp's half of the columns out of tensor memory, onto f times what the rows' place in the workspace holds (if it holds
// something; row null: none).
template <int D>
__device__ __forceinline__ void take_out(uint32_t tl, int half, float4* row, int part_rows, bool holds, float f)
{
#pragma unroll 1
    for (int k = 0; k < D / 32; ++k) {
        const int j = half * (D / 32) + k;
        uint32_t r[16];
        tmem_ld16(tl + 16 * j, r);
        if (row != nullptr) {
            float4* d = row + 4 * j * part_rows;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float4 v = make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]), __uint_as_float(r[4 * e + 2]),
                                       __uint_as_float(r[4 * e + 3]));
                if (holds && f == 1.0f) {       // nothing to wait for (the thread's own place: one order)
                    atomicAdd(d + e * part_rows, v);
                    continue;
                }
                if (holds) {
                    const float4 o = __ldcg(d + e * part_rows);
                    v = make_float4(v.x + f * o.x, v.y + f * o.y, v.z + f * o.z, v.w + f * o.w);
                }
                __stcg(d + e * part_rows, v);
            }
        }
        __syncwarp();
        const uint32_t zero[16] = {};
        tmem_st16(tl + 16 * j, zero);
    }
    tmem_wait_st();
}

// Out of line for the loop that comes here once in many tiles.
template <int D>
__device__ __noinline__ void take_out_seldom(uint32_t tl, int half, float4* row, int part_rows, bool holds, float f)
{
    take_out<D>(tl, half, row, part_rows, holds, f);
}

// kFlush: the tiles after which a sum is taken out, 0: never.
template <int D, int CT, int QT, int kParts, int kFlush>
__global__ void __launch_bounds__(Tc<D, CT, kParts>::kThreads, 1) attn_tc_kernel(const __grid_constant__ AttnArgs A)
{
    using C = Tc<D, CT, kParts>;
    constexpr bool kI8 = C::kI8;
    constexpr int PT = CT == T_F16 ? T_F16 : T_BF16;          // type of the second product
    constexpr int S = C::kStages, NC = C::kConv;
    // log2 of what a probability may reach before the maximum in use is raised; in fp16 that is lost from the range below: a
    // probability is off by 2^-34 of the row's largest.  (8 x 64 drafts over an fp16 cache, scores of 1.5 nats about their
    // mean, fp32 outputs: 63.2 us with 2^12, 63.6 with 2^7, 65.3 with 2^6, 69.9 with 2^5, 74 with 2^4; fp16 outputs 52.2, 52.3,
    // 52.4, 53.9 and 57.6)
    constexpr float kRaise = PT == T_F16 ? 6.0f : 12.0f, kLift = prob_lift(PT, kRaise);
    extern __shared__ uint8_t raw_s[];
    uint8_t* smem = raw_s + ((1024u - (smem_u32(raw_s) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t bars = smem_u32(smem + C::oBars);
    const uint32_t raw_full = bars, raw_empty = raw_full + 16 * S;                   // codes (INT8): keys, then values
    const uint32_t k_full = raw_empty + 16 * S, k_empty = k_full + 8 * NC;            // 16-bit keys
    const uint32_t v_full = k_empty + 8 * NC, v_empty = v_full + 8 * NC;             // and values
    const uint32_t s_full = v_empty + 8 * NC, p_full = s_full + 16, pv_done = p_full + 16, q_full = pv_done + 16, wg_bar = q_full + 8, s_empty = wg_bar + 8;
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::oMisc);
    volatile uint32_t* dead_s = misc + 1;
    volatile uint32_t* odd_s = misc + 2;
    volatile uint32_t* meta_s = reinterpret_cast<volatile uint32_t*>(smem + C::oMeta);
    float* scale_s = reinterpret_cast<float*>(smem + C::oScale);
    int* pre_s = reinterpret_cast<int*>(smem + C::oPre);

    if (tid == 0) {
        for (int k = 0; k < 2 * S; ++k) {
            mbar_init(raw_full + 8 * k, 1);
            mbar_init(raw_empty + 8 * k, kConvWarps / 2);
        }
        for (int k = 0; k < NC; ++k) {
            mbar_init(k_full + 8 * k, kI8 ? kConvWarps / 2 : 1);
            mbar_init(k_empty + 8 * k, 1);
            mbar_init(v_full + 8 * k, kI8 ? kConvWarps / 2 : 1);
            mbar_init(v_empty + 8 * k, 1);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(s_full + 8 * k, 1);
            mbar_init(p_full + 8 * k, 8);
            mbar_init(pv_done + 8 * k, 1);
        }
        mbar_init(q_full, 8);
        mbar_init(wg_bar, 8);
        mbar_init(s_empty, 8);
        fence_mbar_init();
        *dead_s = 0u;
        *odd_s = 0u;
    }
    for (int k = tid; k < 4 * kTcRows; k += C::kThreads) reinterpret_cast<unsigned long long*>(smem + C::oTop)[k] = 0ull;   // (turns begin at 1)
    if (tid == 32 && !kI8) {
        prefetch_map(&A.kmap);
        prefetch_map(&A.vmap);
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc(smem_u32(misc), C::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = misc[0];
    pdl_wait();
    pdl_launch_dependents();                    // (this block holds its tensor memory; the joining launch reads this one's inputs early)
    const Layout lay = block_layout<C::kThreads>(A, kTcRows, kTcUnit, pre_s, reinterpret_cast<int*>(smem + C::oWarpSum));
    if (blockIdx.x == 0 && A.b.B > 32)          // for the joining launch
        for (int b = tid; b <= A.b.B; b += C::kThreads) A.head[b] = pre_s[b];
    const int2 range = block_units(lay, A, static_cast<int>(blockIdx.x), kTcUnit);
    const int us = range.x, ue = range.y;
    if (us >= ue) {
        if (warp == 1) tmem_dealloc(tb, C::kCols);
        return;
    }
    auto fail = [&]() {
        *dead_s = 1u;
        if (A.err != nullptr) atomicExch(A.err, kErrWaitTimeout);
    };

    if (warp == 0) {
        // ---------------------------------------------------------- copies
        const int per = min(A.c.page, kTcUnit), boxes = kTcUnit / per;       // tokens of a copy, copies of a tile
        int it = 0;
        bool ok = true;
        for (int begin = us; begin < ue && ok;) {
            const Segment sg = find_segment(A, lay, begin, kTcRows, kTcUnit);
            const int end = min(sg.u0 + sg.units, ue);
            for (int u = begin; u < end; ++u, ++it) {
                const int t0 = (u - sg.u0) * kTcUnit;
                int page = -1;
                const int t = t0 + lane * per;
                if (lane < boxes && t < sg.f.len)
                    page = __ldg(A.b.table + static_cast<size_t>(sg.b) * A.b.max_pages + (t >> A.c.lg));
                const bool there = page >= 0 && page < A.c.pages;
                const uint32_t have = __ballot_sync(0xffffffffu, there);
                const int z = there ? page * A.c.Hkv + sg.h : 0, y = t & (A.c.page - 1);
                const int n = __popc(have);
                uint32_t sixteenths = 0;
                for (int k = 0; k < boxes; ++k)
                    if (have >> k & 1u) sixteenths |= ((1u << (per / 16)) - 1u) << (k * (per / 16));
                const int st = it % S;
                const uint32_t ph = static_cast<uint32_t>(it / S - 1) & 1u;
                if constexpr (kI8) {
                    // The softmax reads both scales behind the scores, which wait for the keys alone: so the values' scales
                    // come with the keys, too.
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t bar = raw_full + 8 * (half * S + st);
                        if (it >= S) ok = warp_wait(raw_empty + 8 * (half * S + st), ph);
                        if (!ok) break;
                        if (lane == 0) {
                            if (half == 0) meta_s[it % C::kMeta] = sixteenths;
                            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(n * per * (half ? D : D + 8)));
                        }
                        __syncwarp();
                        if (there) {
                            const size_t at = static_cast<size_t>(z) * A.c.page + y;
                            bulk_copy(smem_u32(smem + C::oRaw) + (2 * st + half) * C::kRaw + lane * per * D,
                                      static_cast<const uint8_t*>(half ? A.c.v : A.c.k) + at * D, per * D, bar);
                            if (half == 0) {
                                const uint32_t to = smem_u32(scale_s + (it % C::kMeta) * 2 * kTcUnit + lane * per);
                                bulk_copy(to, A.c.ks + at, per * 4, bar);
                                bulk_copy(to + kTcUnit * 4, A.c.vs + at, per * 4, bar);
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) {                  // (a tile whose keys alone were ordered: they land, too)
                        warp_wait(raw_full + 8 * st, static_cast<uint32_t>(it / S) & 1u);
                        break;
                    }
                } else {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t bar = (half ? v_full : k_full) + 8 * st;
                        if (it >= S) ok = warp_wait((half ? v_empty : k_empty) + 8 * st, ph);
                        if (!ok) break;
                        if (lane == 0) {
                            if (half == 0) meta_s[it % C::kMeta] = sixteenths;
                            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(n * per * D * 2));
                        }
                        __syncwarp();
                        if (there) {
                            const uint32_t dst = smem_u32(smem + C::oKv) + st * 2 * C::kHalf + half * C::kHalf + lane * per * 128;
#pragma unroll
                            for (int x = 0; x < C::kBoxes; ++x)
                                tma_load_3d(dst + x * kTcUnit * 128, half ? &A.vmap : &A.kmap, 64 * x, y, z, bar);
                        }
                        __syncwarp();
                    }
                    if (!ok) {                  // (a tile whose keys alone were ordered: they land, too)
                        warp_wait(k_full + 8 * st, static_cast<uint32_t>(it / S) & 1u);
                        break;
                    }
                }
                __syncwarp();
            }
            begin = end;
        }
        if (!ok && lane == 0) fail();
        // every copy has landed before the block ends (also after a failure)
        for (int k = max(0, it - S); k < it; ++k) {
            const uint32_t ph = static_cast<uint32_t>(k / S) & 1u;
            if constexpr (kI8) {
                if (!warp_wait(raw_full + 8 * (k % S), ph) || !warp_wait(raw_full + 8 * (S + k % S), ph)) break;
            } else {
                if (!warp_wait(k_full + 8 * (k % S), ph) || !warp_wait(v_full + 8 * (k % S), ph)) break;
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        constexpr uint32_t qf = QT == T_BF16 ? 1u : 0u, pf = PT == T_BF16 ? 1u : 0u;
        constexpr uint32_t iqk = (1u << 4) | (qf << 7) | (qf << 10) | (static_cast<uint32_t>(kTcUnit >> 3) << 17) | (static_cast<uint32_t>(kTcRows >> 4) << 24);
        constexpr uint32_t ipv = (1u << 4) | (pf << 7) | (pf << 10) | (1u << 16) | (static_cast<uint32_t>(D >> 3) << 17) | (static_cast<uint32_t>(kTcRows >> 4) << 24);
        const uint64_t q_desc = desc_rows(smem_u32(smem + C::oQ)), k_desc = desc_rows(smem_u32(smem + C::oKv));
        const uint64_t v_desc = desc_cols(smem_u32(smem + C::oKv) + C::kHalf, kTcUnit * 128);
        int it = 0, pieces = 0;
        bool ok = true;
        auto scores = [&](int i) {              // S of tile i, whose keys are there
            tc_fence_after();
            if (elect_one()) {
                const uint64_t k = k_desc + static_cast<uint64_t>((i % NC) * (2 * C::kHalf >> 4));
                const uint32_t d = tb + C::cS + (i % C::kSBufs) * kTcUnit;
#pragma unroll
                for (int x = 0; x < C::kBoxes; ++x) {
                    if constexpr (C::kQInT) mma_ts_rows_x4(d, tb + C::cQ + 32 * x, k + x * (kTcUnit * 128 >> 4), iqk, x > 0);
                    else mma_ss_x4(d, q_desc + x * (kTcRows * 128 >> 4), k + x * (kTcUnit * 128 >> 4), iqk, x > 0);
                }
                tc_commit(k_empty + 8 * (i % NC));
                tc_commit(s_full + 8 * (i & 1));
            }
            __syncwarp();
        };
        auto product = [&](int i) {             // O += P V of tile i, both of which are there
            tc_fence_after();
            if (elect_one()) {
                const uint64_t v = v_desc + static_cast<uint64_t>((i % NC) * (2 * C::kHalf >> 4));
                const uint32_t p = tb + C::cP + (i % C::kPBufs) * 32 * kParts;
#pragma unroll
                for (int part = 0; part < kParts; ++part) mma_ts_x4(tb, p + 32 * part, v, ipv);
                tc_commit(v_empty + 8 * (i % NC));
                tc_commit(pv_done + 8 * (i & 1));
            }
            __syncwarp();
        };
        auto keys = [&](int i) { return warp_wait(k_full + 8 * (i % NC), static_cast<uint32_t>(i / NC) & 1u); };
        for (int begin = us; begin < ue && ok; ++pieces) {
            const Segment sg = find_segment(A, lay, begin, kTcRows, kTcUnit);
            const int end = min(sg.u0 + sg.units, ue), last = it + end - begin;
            ok = warp_wait(q_full, static_cast<uint32_t>(pieces) & 1u) && keys(it);
            if constexpr (C::kSBufs == 1) {
                // one place for scores: the next come when the softmax has read these
                auto place = [&](int i) { return i == 0 || warp_wait(s_empty, static_cast<uint32_t>(i - 1) & 1u); };
                ok = ok && place(it);
                if (ok) scores(it);
                for (; it < last && ok; ++it) {
                    if (it + 1 < last) {
                        ok = keys(it + 1) && place(it + 1);
                        if (!ok) break;
                        scores(it + 1);
                    }
                    ok = warp_wait(v_full + 8 * (it % NC), static_cast<uint32_t>(it / NC) & 1u) &&
                         warp_wait(p_full + 8 * (it & 1), static_cast<uint32_t>(it >> 1) & 1u);
                    if (!ok) break;
                    product(it);
                }
                begin = end;
                continue;
            }
            if (ok) scores(it);
            if (ok && it + 1 < last) {
                ok = keys(it + 1);
                if (ok) scores(it + 1);
            }
            for (; it < last && ok; ++it) {
                // All that can be known before P is: the values are there, the keys of the scores after next as a rule.  What
                // follows P's arrival is the way of the next scores, so those come first: the softmax waits for them sooner
                // than for this product.  (But not if their keys are not there yet: an INT8 cache's may wait for this product.)
                ok = warp_wait(v_full + 8 * (it % NC), static_cast<uint32_t>(it / NC) & 1u);
                if (!ok) break;
                const int i = it + 2;
                const bool more = i < last;
                const bool early = more && __all_sync(0xffffffffu, mbar_test_wait(k_full + 8 * (i % NC), static_cast<uint32_t>(i / NC) & 1u));
                ok = warp_wait(p_full + 8 * (it & 1), static_cast<uint32_t>(it >> 1) & 1u);
                if (!ok) break;
                if (early) scores(i);
                product(it);
                if (more && !early) {
                    ok = keys(i);
                    if (ok) scores(i);
                }
            }
            begin = end;
        }
        if (!ok && lane == 0) fail();
        // every MMA has completed before the tensor memory is freed
        if (it > 0) warp_wait(pv_done + 8 * ((it - 1) & 1), static_cast<uint32_t>((it - 1) >> 1) & 1u);
    } else if (warp >= 4 && warp < 12) {
        // --------------------------------------------------------- softmax
        constexpr int kHalfCols = kTcUnit / 2;
        const int half = (warp - 4) >> 2, row = (warp & 3) * 32 + lane, wid = tid - 128;
        unsigned long long* top_s = reinterpret_cast<unsigned long long*>(smem + C::oTop);
        const uint32_t tl = tb + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        int it = 0;
        uint32_t wg_phase = 0, turn = 1;
        bool ok = true;
        auto wg_sync = [&]() {                  // the eight warps, with a bounded wait
            __syncwarp();
            if (lane == 0) mbar_arrive(wg_bar);
            const bool all = warp_wait(wg_bar, wg_phase & 1u);
            ++wg_phase;
            return all;
        };
        // This thread's number and that of the row's other half: each writes its number with the turn in one word and looks at
        // the other's until it has the turn, too (half of what an mbarrier takes).  The words of a turn are written again two
        // turns later, by when the other half has read them.
        auto exchanged = [&](float v, float& other) {
            unsigned long long* at = top_s + (turn & 1u) * 2 * kTcRows;
            *reinterpret_cast<volatile unsigned long long*>(at + half * kTcRows + row) =
                static_cast<unsigned long long>(turn) << 32 | __float_as_uint(v);
            const volatile unsigned long long* from = at + (half ^ 1) * kTcRows + row;
            unsigned long long got = *from;
            bool all = __all_sync(0xffffffffu, static_cast<uint32_t>(got >> 32) == turn);
            if (!all) {
                uint64_t t0 = 0;
#pragma unroll 1
                for (uint32_t i = 1; !all; ++i) {
                    got = *from;
                    all = __all_sync(0xffffffffu, static_cast<uint32_t>(got >> 32) == turn);
                    if (!all && (i & 255u) == 0u) {
                        const uint64_t now = globaltimer_ns();
                        if (i == 256u) t0 = now;
                        else if (__any_sync(0xffffffffu, now - t0 > kAtWaitNs)) break;
                    }
                }
            }
            ++turn;
            other = __uint_as_float(static_cast<uint32_t>(got));
            return all;
        };
        for (int begin = us; begin < ue && ok;) {
            const Segment sg = find_segment(A, lay, begin, kTcRows, kTcUnit);
            const int end = min(sg.u0 + sg.units, ue);
            const int rows = min(kTcRows, sg.f.n * A.G - sg.tile * kTcRows);
            const bool have = row < rows;
            const int rr = sg.tile * kTcRows + (have ? row : 0), tok = rr / A.G, tq = sg.f.q0 + tok;
            const size_t at = (static_cast<size_t>(tq) * A.Hq + sg.h * A.G + (rr - tok * A.G)) * D;
            unsigned long long see = A.mask != nullptr ? __ldg(A.mask + tq) : (2ull << tok) - 1ull;
            const int drafts = sg.f.len - sg.f.ctx;           // at most 64
            if (drafts < 64) see &= (1ull << drafts) - 1ull;
            // the row's query; the products of the last piece that read the old one are done
            {
                const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(A.q) + at);
                if constexpr (C::kQInT) {
#pragma unroll
                    for (int k = 0; k < D / 64; ++k) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint4 v = have ? __ldg(q + half * (D / 16) + 4 * k + e) : make_uint4(0u, 0u, 0u, 0u);
                            w[4 * e] = v.x; w[4 * e + 1] = v.y; w[4 * e + 2] = v.z; w[4 * e + 3] = v.w;
                        }
                        __syncwarp();
                        tmem_st16(tl + C::cQ + half * (D / 4) + 16 * k, w);
                    }
                } else {
                    uint8_t* d = smem + C::oQ + row * 128;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const int j = half * (D / 16) + k;
                        const uint4 v = have ? __ldg(q + j) : make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4*>(d + (j >> 3) * kTcRows * 128 + (((j & 7) ^ (row & 7)) << 4)) = v;
                    }
                    __syncwarp();
                }
                const uint32_t zero[16] = {};
#pragma unroll
                for (int j = 0; j < D / 32; ++j) tmem_st16(tl + half * (D / 2) + 16 * j, zero);
                tmem_wait_st();
                tc_fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            float m = neg_inf(), l = 0.0f;
            // A sum that is taken out is added in fp32 to what lies in the block's place in the workspace (column groups of
            // four, the rows of one beside each other): the error stays below 192 steps' 2^-23 each (late: 1024 a part),
            // however long the context.
            float* const part = A.part + (static_cast<size_t>(blockIdx.x) * 2 + (us < sg.u0 ? 1 : 0)) * attn_part_floats(A.part_rows, D);
            float4* const kept = reinterpret_cast<float4*>(A.kept + static_cast<size_t>(blockIdx.x) * A.part_rows * D) + (have ? row : 0);
            float m_kept = neg_inf();           // the maximum in use for the kept sum
            bool keeps = false;
            auto kept_factor = [&]() { return m_kept == neg_inf() ? 0.0f : exp2_fast(m_kept - m); };
            for (int u = begin; u < end; ++u, ++it) {
                if (kFlush > 0 && u > begin && (u - begin) % (kFlush > 0 ? kFlush : 1) == 0) {
                    ok = warp_wait(pv_done + 8 * ((it - 1) & 1), static_cast<uint32_t>((it - 1) >> 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    if constexpr (kFlush < kFlushLate) take_out<D>(tl, half, have ? kept : nullptr, A.part_rows, keeps, kept_factor());
                    else take_out_seldom<D>(tl, half, have ? kept : nullptr, A.part_rows, keeps, kept_factor());
                    tc_fence_before();          // (a tile with odd drafts: the row's other half reads these columns, behind wg_sync)
                    keeps = true;
                    m_kept = m;
                }

                ok = warp_wait(s_full + 8 * (it & 1), static_cast<uint32_t>(it >> 1) & 1u);
                if (!ok) break;
                tc_fence_after();
                float s[kHalfCols];
                {
                    uint32_t r0[16], r1[16];
                    const uint32_t a = tl + C::cS + (it % C::kSBufs) * kTcUnit + kHalfCols * half;
                    tmem_ld16x2(a, r0, a + 16, r1);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        s[k] = __uint_as_float(r0[k]);
                        s[16 + k] = __uint_as_float(r1[k]);
                    }
                }
                if constexpr (C::kSBufs == 1) { // read: the next scores may come
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_empty);
                }
                const int t0 = (u - sg.u0) * kTcUnit;
                const uint32_t there = meta_s[it % C::kMeta];
                const bool special = t0 + kTcUnit > sg.f.ctx || there != 15u;
                uint32_t vis = ~0u;                // this half's tokens
                if constexpr (kI8) {
                    const float4* ks = reinterpret_cast<const float4*>(scale_s + (it % C::kMeta) * 2 * kTcUnit + kHalfCols * half);
#pragma unroll
                    for (int j = 0; j < kHalfCols / 4; ++j) {
                        const float4 k4 = ks[j];
                        s[4 * j] *= k4.x;
                        s[4 * j + 1] *= k4.y;
                        s[4 * j + 2] *= k4.z;
                        s[4 * j + 3] *= k4.w;
                    }
                }
                if (special) {
                    // places before the drafts, the row's drafts, of pages that are there
                    const int o = sg.f.ctx - t0;
                    const unsigned long long old = o >= 64 ? ~0ull : o > 0 ? (1ull << o) - 1ull : 0ull;
                    const unsigned long long own = o >= 64 || o <= -64 ? 0ull : o >= 0 ? see << o : see >> -o;
                    vis = static_cast<uint32_t>((old | own) >> (kHalfCols * half));
                    if (!(there >> (2 * half) & 1u)) vis &= 0xffff0000u;
                    if (!(there >> (2 * half + 1) & 1u)) vis &= 0x0000ffffu;
#pragma unroll
                    for (int j = 0; j < kHalfCols; ++j)
                        if (!(vis >> j & 1u)) s[j] = neg_inf();
                }
                float top = s[0];
#pragma unroll
                for (int j = 1; j < kHalfCols; ++j) top = fmaxf(top, s[j]);
                {
                    float other;
                    ok = exchanged(top, other);
                    if (!ok) break;
                    top = fmaxf(top, other) * A.scale;
                }
                const bool raise = top > m + kRaise || (m == neg_inf() && top > m);
                if (__any_sync(0xffffffffu, raise)) {
                    const float was = m;
                    if (raise) m = top;
                    const float f = was == neg_inf() ? 0.0f : exp2_fast(was - m);
                    l *= f;
                    if (u > begin) {            // (before the first tile the output is zero)
                        ok = warp_wait(pv_done + 8 * ((it - 1) & 1), static_cast<uint32_t>((it - 1) >> 1) & 1u);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int j = 0; j < D / 32; ++j) {
                            const uint32_t a = tl + half * (D / 2) + 16 * j;
                            uint32_t r[16];
                            tmem_ld16(a, r);
#pragma unroll
                            for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * f);
                            tmem_st16(a, r);
                        }
                        tmem_wait_st();
                        tc_fence_before();      // (as above)
                    }
                }
                const float base = kLift - (m == neg_inf() ? 0.0f : m);
                float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
                for (int j = 0; j < kHalfCols; j += 2) {
                    s[j] = exp2_fast(__fmaf_rn(s[j], A.scale, base));
                    s[j + 1] = exp2_fast(__fmaf_rn(s[j + 1], A.scale, base));
                    sum0 += s[j];
                    sum1 += s[j + 1];
                }
                l += sum0 + sum1;
                if constexpr (kI8) {
                    const float4* vs = reinterpret_cast<const float4*>(scale_s + (it % C::kMeta) * 2 * kTcUnit + kTcUnit + kHalfCols * half);
#pragma unroll
                    for (int j = 0; j < kHalfCols / 4; ++j) {
                        const float4 v4 = vs[j];
                        s[4 * j] *= v4.x;
                        s[4 * j + 1] *= v4.y;
                        s[4 * j + 2] *= v4.z;
                        s[4 * j + 3] *= v4.w;
                    }
                    if (special) {
#pragma unroll
                        for (int j = 0; j < kHalfCols; ++j)
                            if (!(vis >> j & 1u)) s[j] = 0.0f;
                    }
                } else if (special) {
                    // Values that nothing may see: zeros in their stead.  A draft's infinities and NaN would reach the rows
                    // that do not see it (0 times them): such a tile's drafts are added row by row.
                    ok = warp_wait(v_full + 8 * (it % NC), static_cast<uint32_t>(it / NC) & 1u);
                    if (!ok) break;
                    uint8_t* v = smem + C::oKv + (it % NC) * 2 * C::kHalf + C::kHalf;
                    const uint32_t top16 = CT == T_F16 ? 0x7c00u : 0x7f80u;
                    auto word = [&](int t, int c) { return reinterpret_cast<uint4*>(v + (c >> 3) * kTcUnit * 128 + t * 128 + (((c & 7) ^ (t & 7)) << 4)); };
                    const int from = min(max(sg.f.ctx - t0, 0), kTcUnit);
                    bool odd = false;
                    for (int k = wid; k < kTcUnit * (D / 8); k += 256) {
                        const int t = k / (D / 8);
                        uint4* w = word(t, k % (D / 8));
                        if (t0 + t >= sg.f.len || !(there >> (t >> 4) & 1u)) {
                            *w = make_uint4(0u, 0u, 0u, 0u);
                        } else if (t >= from) {
                            const uint32_t x[4] = {w->x, w->y, w->z, w->w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) odd |= (x[i] & top16) == top16 || (x[i] >> 16 & top16) == top16;
                        }
                    }
                    if (odd) *odd_s = 1u;
                    ok = wg_sync();
                    if (!ok) break;
                    const bool plain = *odd_s != 0u;
                    if (plain) {
                        // (the last product on this output is done: as for the rescaling)
                        if (u > begin) ok = warp_wait(pv_done + 8 * ((it - 1) & 1), static_cast<uint32_t>((it - 1) >> 1) & 1u);
                        if (!ok) break;
                        // one half of each row's tokens after the other
                        if (half == 1) ok = wg_sync();
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 8; c += 2) {
                            uint32_t r[16];
                            tmem_ld16(tl + 8 * c, r);
#pragma unroll
                            for (int j = 0; j < kHalfCols; ++j) {
                                if (j + kHalfCols * half >= from && (vis >> j & 1u)) {
#pragma unroll
                                    for (int h = 0; h < 2; ++h) {
                                        const uint4 w = *word(j + kHalfCols * half, c + h);
                                        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                        for (int i = 0; i < 4; ++i) {
                                            const float2 f = unpair16<CT>(x[i]);
                                            r[8 * h + 2 * i] = __float_as_uint(__uint_as_float(r[8 * h + 2 * i]) + s[j] * f.x);
                                            r[8 * h + 2 * i + 1] = __float_as_uint(__uint_as_float(r[8 * h + 2 * i + 1]) + s[j] * f.y);
                                        }
                                    }
                                }
                            }
                            __syncwarp();
                            tmem_st16(tl + 8 * c, r);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                        if (half == 0) ok = wg_sync();
                        ok = ok && wg_sync();   // every row has read the drafts
                        if (!ok) break;
                        for (int k = wid; k < kTcUnit * (D / 8); k += 256)
                            if (k / (D / 8) >= from) *word(k / (D / 8), k % (D / 8)) = make_uint4(0u, 0u, 0u, 0u);
                        if (wid == 0) *odd_s = 0u;
                    }
                    ok = wg_sync();             // (the flag was read, or is down, before a later tile sets it)
                    if (!ok) break;
                    fence_proxy_async_smem();
                }
                // P's place has been read: of three, by the product that was ordered before these scores
                if (C::kPBufs < 3 && it >= C::kPBufs) {
                    const int b = it - C::kPBufs;
                    ok = warp_wait(pv_done + 8 * (b & 1), static_cast<uint32_t>(b >> 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                }
                const uint32_t p = tl + C::cP + (it % C::kPBufs) * 32 * kParts;
#pragma unroll
                for (int part = 0; part < kParts; ++part) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) w[k] = part16<PT, kI8>(s[2 * k], s[2 * k + 1], part + 1 == kParts);
                    tmem_st16(p + 32 * part + 16 * half, w);
                }
                tmem_wait_st();
                if constexpr (kI8 && kParts > 1) {
                    if (there > 15u) {          // a scale of this tile is vast
                        const uint32_t vasts =  // of this half's tokens
                            __ballot_sync(0xffffffffu, vast(scale_s[(it % C::kMeta) * 2 * kTcUnit + kTcUnit + kHalfCols * half + lane]));
#pragma unroll 1
                        for (int part = 1; part < kParts; ++part) {
                            uint32_t w[16];
                            tmem_ld16(p + 32 * part + 16 * half, w);
#pragma unroll
                            for (int k = 0; k < 16; ++k) w[k] = only_first(w[k], vasts >> (2 * k) & 1u, vasts >> (2 * k + 1) & 1u);
                            tmem_st16(p + 32 * part + 16 * half, w);
                        }
                        tmem_wait_st();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + 8 * (it & 1));
            }
            if (ok) ok = warp_wait(pv_done + 8 * ((it - 1) & 1), static_cast<uint32_t>((it - 1) >> 1) & 1u);
            float l2 = 0.0f;
            if (ok) ok = exchanged(l, l2);
            if (!ok) {
                if (lane == 0) fail();
                break;
            }
            l = half ? l2 + l : l + l2;
            tc_fence_after();
            // ------------------------------------------------- the row's result
            const bool whole = begin == sg.u0 && end == sg.u0 + sg.units;
            if (have && !whole && half == 0) {
                part[row] = m;
                part[A.part_rows + row] = l;
            }
            const float inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f, f_kept = kept_factor();
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
                const int j = half * (D / 32) + k;
                uint32_t r[16];
                tmem_ld16(tl + 16 * j, r);
                if (have) {
                    float v[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(r[k]);
                    if (kFlush > 0 && keeps) {
#pragma unroll
                        for (int k = 0; k < 16; k += 4) {
                            const float4 o = __ldcg(kept + (4 * j + k / 4) * A.part_rows);
                            v[k] += f_kept * o.x; v[k + 1] += f_kept * o.y; v[k + 2] += f_kept * o.z; v[k + 3] += f_kept * o.w;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] *= inv;
                    if (!whole || A.ytype == T_F32) {
                        float4* d = reinterpret_cast<float4*>(whole ? static_cast<float*>(A.y) + at + 16 * j
                                                                    : part + 2 * A.part_rows + static_cast<size_t>(row) * D + 16 * j);
#pragma unroll
                        for (int k = 0; k < 4; ++k) d[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                    } else {
                        uint32_t w[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            w[k] = A.ytype == T_F16 ? pair16<T_F16>(v[2 * k], v[2 * k + 1]) : pair16<T_BF16>(v[2 * k], v[2 * k + 1]);
                        uint4* d = reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.y) + at + 16 * j);
                        d[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        d[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    }
                }
                __syncwarp();
            }
            __syncwarp();
            begin = end;
        }
    } else if (kI8) {
        // ---------------------------------------------------- codes to 16 bits
        // Half of the warps takes the keys, half the values, each at its own pace.
        const int cw = warp < 4 ? warp - 2 : warp - 10, half = cw & 1, w = (cw >> 1) * 32 + lane;
        const uint32_t full = raw_full + 8 * half * S, empty = raw_empty + 8 * half * S;
        const uint32_t to_full = half ? v_full : k_full, to_empty = half ? v_empty : k_empty;
        const int n = ue - us;
        bool ok = true;
        for (int it = 0; it < n && ok; ++it) {
            const int st = it % S, cv = it % NC;
            ok = warp_wait(full + 8 * st, static_cast<uint32_t>(it / S) & 1u);
            if (it >= NC) ok = ok && warp_wait(to_empty + 8 * cv, static_cast<uint32_t>(it / NC - 1) & 1u);
            if (!ok) break;
            if (kParts > 1 && cw == 0) {        // (a value's scale that the softmax has to know of)
                const float* vs = scale_s + (it % C::kMeta) * 2 * kTcUnit + kTcUnit;
                if (__any_sync(0xffffffffu, vast(vs[lane]) || vast(vs[32 + lane])) && lane == 0) meta_s[it % C::kMeta] |= 16u;
                __syncwarp();
            }
            const uint8_t* src = smem + C::oRaw + (2 * st + half) * C::kRaw;
            uint8_t* dst = smem + C::oKv + (2 * cv + half) * C::kHalf;
            constexpr int kStep = 16 * kConvWarps, kTimes = kTcUnit * D / 16 / kStep;
            static_assert(kTcUnit * D / 16 % kStep == 0, "whole steps");
#pragma unroll
            for (int i = 0; i < kTimes; ++i) {
                const int k = w + kStep * i, t = k / (D / 16), c = k % (D / 16);    // sixteen codes: two 16-byte words
                const uint4 q = *reinterpret_cast<const uint4*>(src + 16 * k);
                const uint32_t x[4] = {q.x, q.y, q.z, q.w};
                uint32_t h[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (QT == T_F16 && half == 0) i8_to_f16(x[e], h[2 * e], h[2 * e + 1]);
                    else i8_to_bf16(x[e], h[2 * e], h[2 * e + 1]);
                }
                uint8_t* d = dst + (c >> 2) * kTcUnit * 128 + t * 128;
                const int a = ((2 * c) & 7) ^ (t & 7), b = a ^ 1;
                const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
                // (every other column group the other way round: eight lanes on eight different words)
                const bool flip = (c >> 2) & 1;
                *reinterpret_cast<uint4*>(d + ((flip ? b : a) << 4)) = flip ? hi : lo;
                *reinterpret_cast<uint4*>(d + ((flip ? a : b) << 4)) = flip ? lo : hi;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(to_full + 8 * cv);
                mbar_arrive(empty + 8 * st);
            }
            __syncwarp();
        }
        if (!ok && lane == 0) fail();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tb, C::kCols);
}

constexpr int kExtra = 6;                       // (4 us at 0.7 us a unit, heads of 128 and bf16; 8 us of INT8 heads of 256)

template <int D, int CT, int QT, int kParts, int kFlush>
cudaError_t launch(AttnArgs& a, int sms, cudaStream_t s)
{
    using C = Tc<D, CT, kParts>;
    auto kern = attn_tc_kernel<D, CT, QT, kParts, kFlush>;
    static SmemLimit limit;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), limit, C::smem(kAtMaxSeq));
    if constexpr (CT != T_I8) {
        const int rows = a.c.page < kTcUnit ? a.c.page : kTcUnit;
        if (e == cudaSuccess) e = encode_kv_map(&a.kmap, a, a.c.k, 128, rows);
        if (e == cudaSuccess) e = encode_kv_map(&a.vmap, a, a.c.v, 128, rows);
    }
    if (e != cudaSuccess) return e;
    a.blocks = blocks_of(sms);
    a.extra = kExtra;
    a.least = 1;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(a.blocks));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::smem(a.b.B);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int D, int CT, int QT>
cudaError_t launch_w(AttnArgs& a, int sms, cudaStream_t s)
{
    if (a.ytype == T_F32) return launch<D, CT, QT, CT == T_F16 ? 2 : 3, kFlushParts>(a, sms, s);
    const bool lasts = piece_units(a, blocks_of(sms), kTcUnit, kExtra) > kFlushLate;
    if constexpr (CT == T_F16) {
        if (a.ytype == T_BF16) return lasts ? launch<D, CT, QT, 1, kFlushLate>(a, sms, s) : launch<D, CT, QT, 1, 0>(a, sms, s);
    } else {
        if (a.ytype == T_F16) return launch<D, CT, QT, 2, kFlushParts>(a, sms, s);
    }
    return lasts ? launch<D, CT, QT, 2, kFlushLate>(a, sms, s) : launch<D, CT, QT, 2, 0>(a, sms, s);
}

template <int D>
cudaError_t launch_d(AttnArgs& a, int qtype, int sms, cudaStream_t s)
{
    if (a.c.type == T_F16) return launch_w<D, T_F16, T_F16>(a, sms, s);
    if (a.c.type == T_BF16) return launch_w<D, T_BF16, T_BF16>(a, sms, s);
    return qtype == T_F16 ? launch_w<D, T_I8, T_F16>(a, sms, s) : launch_w<D, T_I8, T_BF16>(a, sms, s);
}

}  // namespace

cudaError_t launch_attn_tc(AttnArgs& a, int qtype, int sms, cudaStream_t s)
{
    return a.c.D == 64 ? launch_d<64>(a, qtype, sms, s) : a.c.D == 128 ? launch_d<128>(a, qtype, sms, s)
                                                                            : launch_d<256>(a, qtype, sms, s);
}

}  // namespace w4k
