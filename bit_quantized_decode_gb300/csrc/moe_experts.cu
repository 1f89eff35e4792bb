// The experts of a mixture-of-experts layer for a few tokens, in one kernel:
// for every token m and chosen (or shared) expert e
//   g, u = the linear of q_x by e's gate and up rows,  h = fp32(act(g) u),
//   q_h, s_h = the INT8 codes of h,                     d = the linear of q_h by e's down rows,
//   y[m] = sum over the slots in order of weight * d (+ residual)
// with per-row INT4 or INT8 weights, exact integer sums and the library's
// epilogue fma(fp32(s_w s_x), fp32(acc), b).
//
// What bounds it is the chosen experts' weights: they are read once, by
// whichever tokens chose them.  The two halves of the layer depend on each
// other through all of h, so the kernel is one stream of work with no grid
// barrier:
//   * Tickets.  A global counter hands out 8-row tiles of the gate/up
//     matrices (one entry after another), then tasks that quantize h, then
//     tiles of the down matrices.  A warp takes its next tickets ahead and
//     fetches their weights through its own ring of bulk copies, so while the
//     last hidden values are made and quantized the down weights are already
//     on their way.  A warp waits only for tickets handed out before its own,
//     which running warps hold and finish without waiting on later ones: the
//     kernel needs no co-resident grid and two of them may share the GPU.
//   * An entry is an expert and some of its tokens; more of them are further
//     entries.  Up to two tokens: a lane holds four rows by the tokens of
//     integer sums (DP4A, as the decode GEMV: line lane / 2 of a 16-line pass,
//     rows 4 (lane & 1) .. + 3, reads permuted against bank conflicts, a shuffle
//     butterfly at the end of a tile).  One token, eight of 64 experts of 2368 x
//     3584 (102 MB of INT4): 36 us with the router.
//   * Up to eight tokens: mma.sync on two tiles at a time, the weights as the 16
//     rows of A, the tokens as the eight columns of B.  So few columns leave
//     tcgen05 nothing to gain (its smallest tile has 64 or 128 rows, and A would
//     go through tensor memory once more); here a lane loads its K of a row from
//     the ring as it lies.  INT4 needs no conversion at all: a nibble w + 8 at
//     bit 0 or 16 of a word is the fp16 number (w + 8) 2^-24, subnormal and
//     exact, so a mask makes an operand pair; the codes wait as fp16 in shared
//     memory.  (e4m3 operands would take half the products, but are converted to
//     fp16 by instructions of their own: 162 instead of 106 million.)  INT8 runs
//     on the integer product, 15 cycles for 16 x 32 x 8 (fp16: 4.2), which two
//     INT8 tiles just afford and INT4 ones would not.
//     A slice of 16 lines takes a warp some 1600 cycles and its copies and
//     bookkeeping another 1300; waits for memory are 5%.  16 tokens over 64
//     experts of 2368 x 3584 (722 MB of INT4): 178 to 181 us with the router; DP4A 202.
//   * No fence per tile (it waits for all that the warp has outstanding: it
//     took 3500 of a tile's 9500 cycles): hidden values and the slots' outputs
//     are prepared with a value that no result takes (MoeFill), and a reader
//     looks at the words themselves until every one is there.  Only the few
//     quantizing tasks publish their codes with release order, which the tiles
//     that read them through L1 acquire.
//   * Adding tasks, the last tickets, sum the slots' outputs in order: no
//     floating-point atomics, so results do not depend on timing.
#include <type_traits>

#include "exact_act.cuh"
#include "operators.h"
#include "ptx.cuh"
#include "quant_a8.cuh"
#include "typed_io.cuh"

namespace w4k {
namespace {

constexpr uint64_t kMxWaitNs = 250ull * 1000ull * 1000ull;

__host__ __device__ constexpr int mx_unit(int fmt) { return fmt == FMT_W4 ? 16 : 32; }
// Ring slots: bytes, slots per warp and warps per block.  A slot costs a wait
// and a copy however large it is, so where an entry has one or two tokens (few
// sums per weight) the slots are large.  On the tensor cores more warps, as many
// as fit beside the tokens' codes (8 tokens of 3584: 16 warps 121 us, 12 warps
// 135).
__host__ __device__ constexpr int mx_slot(int tok) { return tok <= 2 ? 8192 : 4096; }
__host__ __device__ constexpr int mx_stages(int) { return 2; }
__host__ __device__ constexpr int mx_warps(int tok) { return tok <= 2 ? 12 : 16; }
constexpr int kMxFewestWarps = 10;                 // a thread for each pair
// Entries of more than two tokens multiply on the tensor cores, two tiles at a time.
__host__ __device__ constexpr bool mx_mma(int tok) { return tok > 2; }
// Bytes of a code as a kernel reads it (INT4 on the tensor cores: fp16), and the
// stride of the tokens' staged codes: what a read takes of several tokens lies in
// banks of their own.
__host__ __device__ constexpr int mx_code(int fmt, int tok) { return mx_mma(tok) && fmt == FMT_W4 ? 2 : 1; }
__host__ __device__ constexpr int mx_stride(int fmt, int tok, int H)
{
    return !mx_mma(tok) ? H : fmt == FMT_W4 ? 2 * H + (192 - 2 * H % 128) % 128 : H + (160 - H % 128) % 128;
}

constexpr int kMxBatches = 64;

struct MxSmem {
    int bars, mask, off, ent0, pair_e, list, tok, ent_e, ent_off, ent_n, of_pos, ready, sh, hs, sx, xsum, misc, base, ring, codes, total;
};
__host__ __device__ inline MxSmem mx_smem(int tok, int warps, int staged)
{
    const int stages = mx_stages(tok);
    MxSmem L;
    int o = 0;
    L.bars = o;    o += (warps * stages + 1) * 8;      // the rings', the staged codes'
    L.mask = o;    o += kMxMaxExperts * 4;             // tokens of an expert, a bit each (or: pairs per expert)
    L.off = o;     o += kMxMaxExperts * 2;             // first place of an expert's pairs in the list
    L.ent0 = o;    o += kMxMaxExperts * 2;             // and its first entry
    L.pair_e = o;  o += kMxMaxPairs * 2;               // expert of a pair (0xffff: none)
    L.list = o;    o += kMxMaxPairs * 2;               // pairs ordered by expert
    L.tok = o;     o += kMxMaxPairs;                   // token of a place
    L.ent_e = o;   o += kMxMaxPairs * 2;
    L.ent_off = o; o += (kMxMaxPairs + 2) * 2;         // first place of an entry's pairs
    L.ent_n = o;   o += kMxMaxPairs;                   // and how many
    L.of_pos = o;  o += kMxMaxPairs * 2;               // entry of a place
    L.ready = o;   o += kMxMaxPairs;                   // the entry's hidden codes were seen complete
    o = align_up(o, 16);
    L.sh = o;      o += kMxMaxPairs * 4;               // then: scale and code sum of a place's hidden values
    L.hs = o;      o += kMxMaxPairs * 4;
    L.sx = o;      o += 16 * 4;
    L.xsum = o;    o += 16 * 4;
    L.misc = o;    o += 16;
    L.base = o;    o += kMxBatches * 8;                // first tickets of this block's batches, tagged
    o = align_up(o, 128);
    L.ring = o;    o += warps * stages * mx_slot(tok);
    L.codes = o;   o += staged;                        // the tokens' codes
    L.total = o;
    return L;
}

// n / d for 0 <= n < 2^24 * d (inv = fp32(1 / d)), and the remainder.
__device__ __forceinline__ int div_by(int n, int d, float inv, int& rem)
{
    int q = __float2int_rd(__fmul_rn(__int2float_rn(n), inv));
    rem = n - q * d;
    while (rem < 0) {
        --q;
        rem += d;
    }
    while (rem >= d) {
        ++q;
        rem -= d;
    }
    return q;
}

// Words that another block writes while this one looks (L2, no order with others).
__device__ __forceinline__ uint4 ld_relaxed_v4(const void* p)
{
    uint4 v;
    asm volatile("ld.relaxed.gpu.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_relaxed_u32(const void* p)
{
    uint32_t v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_relaxed_u32(void* p, uint32_t v)
{
    asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// A result: never the bits that mean "not written" (they are those of a NaN).
__device__ __forceinline__ void st_value(float* p, float v)
{
    const uint32_t u = __float_as_uint(v);
    st_relaxed_u32(p, u == kMxNoValue ? 0x7fffffffu : u);
}
// A quantizing task's result, ordered behind its codes, and its reader's side.
__device__ __forceinline__ void st_release_u64(unsigned long long* p, unsigned long long v)
{
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned long long ld_acquire_u64(const unsigned long long* p)
{
    unsigned long long v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ int dp4a_u(uint32_t a, uint32_t b, int c)
{
    int d;
    asm("dp4a.u32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// Four rows of one line (w0, w1: the units of rows 4h + (j ^ pp)) against one
// token's 32 codes.  INT4: low nibbles into acc, 16 times the high ones into hi.
template <int FMT>
__device__ __forceinline__ void line_dot(const uint4 (&w0)[4], const uint4 (&w1)[4], const uint4& x0, const uint4& x1,
                                         int (&acc)[4], int (&hi)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint4 w = w0[j];
        if constexpr (FMT == FMT_W4) {
            acc[j] = dp4a_u(w.x & 0x0F0F0F0Fu, x0.x, acc[j]);
            hi[j] = dp4a_u(w.x & 0xF0F0F0F0u, x0.y, hi[j]);
            acc[j] = dp4a_u(w.y & 0x0F0F0F0Fu, x0.z, acc[j]);
            hi[j] = dp4a_u(w.y & 0xF0F0F0F0u, x0.w, hi[j]);
            acc[j] = dp4a_u(w.z & 0x0F0F0F0Fu, x1.x, acc[j]);
            hi[j] = dp4a_u(w.z & 0xF0F0F0F0u, x1.y, hi[j]);
            acc[j] = dp4a_u(w.w & 0x0F0F0F0Fu, x1.z, acc[j]);
            hi[j] = dp4a_u(w.w & 0xF0F0F0F0u, x1.w, hi[j]);
        } else {
            const uint4 v = w1[j];
            acc[j] = dp4a_ss(w.x, x0.x, acc[j]);
            hi[j] = dp4a_ss(v.x, x1.x, hi[j]);
            acc[j] = dp4a_ss(w.y, x0.y, acc[j]);
            hi[j] = dp4a_ss(v.y, x1.y, hi[j]);
            acc[j] = dp4a_ss(w.z, x0.z, acc[j]);
            hi[j] = dp4a_ss(v.z, x1.z, hi[j]);
            acc[j] = dp4a_ss(w.w, x0.w, acc[j]);
            hi[j] = dp4a_ss(v.w, x1.w, hi[j]);
        }
    }
}

// Eight INT8 codes (K 0 .. 3, 4 .. 7) as the fp16 pairs K 0 2, 1 3 and, divided
// by 16, 4 6, 5 7: (1024 + (x + 128)) - 1152 and its sixteenth, all exact.
__device__ __forceinline__ uint4 codes_half(uint32_t lo, uint32_t hi)
{
    lo ^= 0x80808080u;
    hi ^= 0x80808080u;
    uint4 h;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h.x) : "r"(__byte_perm(lo, 0x64646464u, 0x4240)), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h.y) : "r"(__byte_perm(lo, 0x64646464u, 0x4341)), "r"(0x64806480u));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(h.z) : "r"(__byte_perm(hi, 0x64646464u, 0x4240)), "r"(0x2c002c00u), "r"(0xd480d480u));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(h.w) : "r"(__byte_perm(hi, 0x64646464u, 0x4341)), "r"(0x2c002c00u), "r"(0xd480d480u));
    return h;
}
// D += A B: 16 rows by 16 or 32 K of A, as many K by 8 columns of B.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int FMT, int TK>
__global__ void __launch_bounds__(32 * mx_warps(TK), 1) moe_experts_kernel(const __grid_constant__ MoeArgs A)
{
    constexpr bool kMma = mx_mma(TK);
    const int NW = kMma ? static_cast<int>(blockDim.x) >> 5 : mx_warps(TK), NT = 32 * NW;
    constexpr int kTiles = kMma ? 2 : 1;           // tiles of a ticket, each with its part of a ring slot
    constexpr int kAdd = mx_add(TK);
    constexpr int kUnit = mx_unit(FMT), kSlot = mx_slot(TK), kLines = kSlot / (kTiles * kRows * kUnit);
    static_assert(kMma || kLines % 16 == 0, "slices of whole passes: every lane steps through the codes alike");
    static_assert(!kMma || FMT != FMT_W4 || kLines * 32 * 15 * 128 <= (1 << 24), "a slice's sums are exact in fp32");
    constexpr bool kSplit = mx_code(FMT, TK) == 2;
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int S = mx_stages(TK);
    const MxSmem L = mx_smem(TK, NW, 0);
    uint32_t* mask_s = reinterpret_cast<uint32_t*>(smem + L.mask);
    uint16_t* ent0_s = reinterpret_cast<uint16_t*>(smem + L.ent0);
    uint16_t* off_s = reinterpret_cast<uint16_t*>(smem + L.off);
    uint16_t* pair_e = reinterpret_cast<uint16_t*>(smem + L.pair_e);
    uint16_t* list = reinterpret_cast<uint16_t*>(smem + L.list);
    uint8_t* tok_s = smem + L.tok;
    uint16_t* ent_e = reinterpret_cast<uint16_t*>(smem + L.ent_e);
    uint16_t* ent_off = reinterpret_cast<uint16_t*>(smem + L.ent_off);
    uint8_t* ent_n = smem + L.ent_n;
    uint16_t* of_pos = reinterpret_cast<uint16_t*>(smem + L.of_pos);
    volatile uint8_t* ready_s = smem + L.ready;
    float* sh_s = reinterpret_cast<float*>(smem + L.sh);
    int* hs_s = reinterpret_cast<int*>(smem + L.hs);
    float* sx_s = reinterpret_cast<float*>(smem + L.sx);
    int* xsum_s = reinterpret_cast<int*>(smem + L.xsum);
    volatile int* misc = reinterpret_cast<volatile int*>(smem + L.misc);       // [0] entries, [1] pairs, [2] tickets taken here
    volatile unsigned long long* base_s = reinterpret_cast<volatile unsigned long long*>(smem + L.base);

    const int slots = A.top_k + A.S;
    const int P = A.M * slots;
    const int C1 = A.H >> 5, C2 = A.I >> 5;
    const int T1 = (A.I + 3) >> 2, T2 = (A.H + 7) >> 3;
    const int U1 = (T1 + kTiles - 1) / kTiles, U2 = (T2 + kTiles - 1) / kTiles;      // tickets of a matrix
    const int HS = mx_stride(FMT, TK, A.H);
    unsigned* ticket = A.ticket;

    uint8_t* ring = smem + L.ring + static_cast<size_t>(warp) * S * kSlot;
    const uint32_t bars = smem_u32(smem + L.bars) + static_cast<uint32_t>(warp * S) * 8u;
    if (lane == 0) {
        for (int s = 0; s < S; ++s) mbar_init(bars + 8 * s, 1);
        if (warp == 1) mbar_init(smem_u32(smem + L.bars) + static_cast<uint32_t>(NW * S) * 8u, 1);
        fence_mbar_init();
    }
    if (tid > 1 && tid < kMxBatches) base_s[tid] = ~0ull;
    if (tid == NT - 1) misc[2] = 0;
    if (tid >= 64 && tid < 80) xsum_s[tid - 64] = 0;
    const int EE = A.E + A.S;
    if (TK > 1)
        for (int e = tid; e < EE; e += NT) mask_s[e] = 0u;
    for (int i = tid; i < P; i += NT) ready_s[i] = 0;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();

    // ---- the entries, the same in every block: pairs counted by expert in
    // the order of the pairs (warp 0); scales and code sums of the tokens (the others)
    if (tid == NT - 1) {
        base_s[0] = atomicAdd(ticket, static_cast<unsigned>(A.batch0));
        base_s[1] = (1ull << 32) | atomicAdd(ticket, static_cast<unsigned>(A.batch));
    }
    // (the codes before any weights: behind those a load waits for microseconds)
    const uint32_t xbar = smem_u32(smem + L.bars) + static_cast<uint32_t>(NW * S) * 8u;
    if (A.stage_x && !kSplit && tid == 32) {
        mbar_arrive_expect_tx(xbar, static_cast<uint32_t>(A.M * A.H));
        const int n = kMma ? A.M : 1, bytes = kMma ? A.H : A.M * A.H;
        for (int m = 0; m < n; ++m)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             smem_u32(smem + L.codes) + static_cast<uint32_t>(m * HS)),
                         "l"(A.qx + static_cast<size_t>(m) * A.H), "r"(static_cast<uint32_t>(bytes)), "r"(xbar)
                         : "memory");
    }
    auto expert_of = [&](int p) -> int {
        const int m = p / slots, s = p - m * slots;
        if (s >= A.top_k) return A.E + s - A.top_k;
        const int e = __ldg(A.ids + m * A.top_k + s);
        return e < 0 || e >= A.E ? 0xffff : e;
    };
    // (every warp but the first)
    auto stage_split = [&]() {
        const int WT = NT - 32;
        const int wt = tid - 32;
        // the split codes of every token, eight reads of 16 codes to a thread at a time
        if (wt < A.M) sx_s[wt] = __ldg(A.sx + wt);
        const int per = A.H >> 4, n = A.M * per;
        const uint4* q = reinterpret_cast<const uint4*>(A.qx);
        for (int i0 = 0; i0 < n; i0 += 8 * WT) {
            uint4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int i = i0 + k * WT + wt;
                v[k] = i < n ? __ldg(q + i) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int i = i0 + k * WT + wt;
                if (i0 + k * WT >= n) break;
                int at = 0, s = 0;
                const int m = i < n ? div_by(i, per, A.inv_x16, at) : A.M - 1;
                if (i < n) {
                    uint4* to = reinterpret_cast<uint4*>(smem + L.codes + m * HS) + 2 * at;
                    to[0] = codes_half(v[k].x, v[k].y);
                    to[1] = codes_half(v[k].z, v[k].w);
                    s = __dp4a(static_cast<int>(v[k].x), 0x01010101, s);
                    s = __dp4a(static_cast<int>(v[k].y), 0x01010101, s);
                    s = __dp4a(static_cast<int>(v[k].z), 0x01010101, s);
                    s = __dp4a(static_cast<int>(v[k].w), 0x01010101, s);
                }
                // for the nibble bias
                if (__all_sync(0xffffffffu, m == __shfl_sync(0xffffffffu, m, 0))) {
                    s = __reduce_add_sync(0xffffffffu, s);
                    if (lane == 0) atomicAdd(xsum_s + m, 8 * s);
                } else {
                    atomicAdd(xsum_s + m, 8 * s);
                }
            }
        }
    };
    if (TK == 1) {
        // one token: every pair is an entry (at most kMxMaxSlots <= 32 of them)
        if (warp == 0) {
            const int e = lane < P ? expert_of(lane) : 0xffff;
            const unsigned have = __ballot_sync(0xffffffffu, e != 0xffff);
            const int at = __popc(have & ((1u << lane) - 1u));
            if (lane < P) pair_e[lane] = static_cast<uint16_t>(e);
            if (e != 0xffff) {
                list[at] = static_cast<uint16_t>(lane);
                tok_s[at] = 0;
                ent_e[at] = static_cast<uint16_t>(e);
                ent_n[at] = 1;
                ent_off[at] = of_pos[at] = static_cast<uint16_t>(at);
            }
            if (lane == 0) misc[0] = misc[1] = __popc(have);
        }
    } else {
        static_assert(kMxMaxPairs <= 32 * kMxFewestWarps && mx_warps(TK) >= kMxFewestWarps, "a thread for each pair");
        const int e = tid < P ? expert_of(tid) : 0xffff;
        const int m = tid / slots;
        if (tid < P) pair_e[tid] = static_cast<uint16_t>(e);
        if (e != 0xffff) atomicOr(mask_s + e, 1u << m);
        const int valid = __syncthreads_count(e != 0xffff);
        if (warp == 0) {
            // places and entries of the experts: prefix sums of two counts in one word
            auto scan = [&](auto&& count) -> int {
                int at = 0, ne = 0;
                for (int e0 = 0; e0 < EE; e0 += 32) {
                    const int c = e0 + lane < EE ? count(e0 + lane) : 0;
                    const int k = (c + TK - 1) / TK;
                    int both = c | (k << 16);
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int v = __shfl_up_sync(0xffffffffu, both, o);
                        if (lane >= o) both += v;
                    }
                    if (c > 0) {
                        const int a0 = at + (both & 0xffff) - c, n0 = ne + (both >> 16) - k;
                        off_s[e0 + lane] = static_cast<uint16_t>(a0);
                        ent0_s[e0 + lane] = static_cast<uint16_t>(n0);
                        for (int i = 0; i < k; ++i) {
                            ent_e[n0 + i] = static_cast<uint16_t>(e0 + lane);
                            ent_off[n0 + i] = static_cast<uint16_t>(a0 + i * TK);
                            ent_n[n0 + i] = static_cast<uint8_t>(min(TK, c - i * TK));
                        }
                    }
                    both = __shfl_sync(0xffffffffu, both, 31);
                    at += both & 0xffff;
                    ne += both >> 16;
                }
                if (lane == 0) {
                    misc[0] = ne;
                    misc[1] = at;
                }
                return at;
            };
            const int at = scan([&](int x) { return __popc(mask_s[x]); });
            if (at != valid) {
                // some token names an expert twice: count pair by pair
                for (int x = lane; x < EE; x += 32) mask_s[x] = 0u;
                __syncwarp();
                for (int p0 = 0; p0 < P; p0 += 32) {
                    const int x = p0 + lane < P ? pair_e[p0 + lane] : 0xffff;
                    const unsigned same = __match_any_sync(0xffffffffu, x);
                    const int rank = __popc(same & ((1u << lane) - 1u));
                    const unsigned base = x != 0xffff ? mask_s[x] : 0u;
                    __syncwarp();
                    if (x != 0xffff) {
                        of_pos[p0 + lane] = static_cast<uint16_t>(base + rank);          // the pair's rank, for now
                        if (rank == 0) mask_s[x] = base + __popc(same);
                    }
                    __syncwarp();
                }
                scan([&](int x) { return static_cast<int>(mask_s[x]); });
            }
            if (lane == 0) misc[3] = at != valid;
        } else if (kSplit) {
            stage_split();
        }
        __syncthreads();
        const int rank = e == 0xffff ? 0 : misc[3] ? of_pos[tid] : __popc(mask_s[e] & ((1u << m) - 1u));
        if (misc[3]) __syncthreads();
        if (e != 0xffff) {
            const int pos = off_s[e] + rank;
            list[pos] = static_cast<uint16_t>(tid);
            tok_s[pos] = static_cast<uint8_t>(m);
            of_pos[pos] = static_cast<uint16_t>(ent0_s[e] + rank / TK);
        }
    }
    if (!kSplit && warp > 0) {
        bool ok = true;
        if (A.stage_x) ok = mbar_wait_bounded(xbar, 0u, kMxWaitNs);
        if (!ok && A.err != nullptr) atomicExch(A.err, kErrWaitTimeout);
        const int8_t* src = A.stage_x ? reinterpret_cast<const int8_t*>(smem + L.codes) : A.qx;
        for (int m = warp - 1; m < A.M; m += NW - 1) {
            int s = 0;
            if (FMT == FMT_W4) {                                            // for the nibble bias
                const uint4* q = reinterpret_cast<const uint4*>(src + static_cast<size_t>(m) * (A.stage_x ? HS : A.H));
#pragma unroll 4
                for (int i = lane; i < A.H / 16; i += 32) {
                    const uint4 v = q[i];
                    s = __dp4a(static_cast<int>(v.x), 0x01010101, s);
                    s = __dp4a(static_cast<int>(v.y), 0x01010101, s);
                    s = __dp4a(static_cast<int>(v.z), 0x01010101, s);
                    s = __dp4a(static_cast<int>(v.w), 0x01010101, s);
                }
                s = __reduce_add_sync(0xffffffffu, s);
            }
            if (lane == 0) {
                xsum_s[m] = 8 * s;
                sx_s[m] = __ldg(A.sx + m);
            }
        }
    }
    __syncthreads();
    const int NE = misc[0], PV = misc[1];
    const int nseg = (A.I + kMxSeg - 1) / kMxSeg;
    const int nadd = (A.H + kAdd - 1) / kAdd;
    const int n1 = NE * U1, nq = n1 + PV * nseg, n2 = nq + NE * U2, total = n2 + A.M * nadd;

    // ---- tickets.  A block takes them from the global counter a batch at a
    // time (thousands of warps on one counter would wait for it: some 2 ns
    // each), its warps from a counter of their own; the warp that opens a batch
    // fetches the one after the next.  Claimed tickets wait in the lanes of `fifo` until
    // their weights are consumed, as kind (0 gate/up, 1 quantize, 2 down,
    // 3 add), entry, place or token, and tile or segment.
    const uint64_t pol = l2_policy_evict_first();
    uint32_t fifo = 0;
    unsigned head = 0, tail = 0;
    int issued = 0, islot = 0, cslot = 0, consumed = 0;
    uint32_t cph = 0u;
    bool dead = false;
    // the ticket whose slices are being issued
    const uint8_t* isrc = nullptr;
    int ileft = 0;                        // lines left of it
    uint32_t isecond = 0;                 // bytes from its tile to the next one, 0 where there is none
    bool more = true;
    bool task = false;                    // a quantizing or adding task is claimed and not done
    const float inv_batch = 1.0f / static_cast<float>(A.batch);
    // First ticket of the block's batch b, from the warp that opened the batch before the last.
    auto base_of = [&](int b) -> int {
        unsigned long long v = base_s[b % kMxBatches];
        if (static_cast<int>(v >> 32) != b) {
            const uint64_t t0 = globaltimer_ns();
            while (static_cast<int>((v = base_s[b % kMxBatches]) >> 32) != b) {
                if (globaltimer_ns() - t0 > kMxWaitNs) {
                    if (A.err != nullptr) atomicExch(A.err, kErrWaitTimeout);
                    return 0x7fffffff;
                }
            }
        }
        return static_cast<int>(static_cast<uint32_t>(v));
    };
    // Whether the block's next ticket is known by now (another warp may be faster).
    auto known = [&]() -> bool {
        const int l = misc[2];
        int i;
        const int b = l < A.batch0 ? 0 : 1 + div_by(l - A.batch0, A.batch, inv_batch, i);
        return static_cast<int>(base_s[b % kMxBatches] >> 32) == b;
    };
    // The next ticket, or one past the last.
    auto claim = [&]() -> int {
        int next = 0;
        if (lane == 0) {
            int i;
            const int l = atomicAdd(const_cast<int*>(misc + 2), 1);
            const int b = l < A.batch0 ? 0 : 1 + div_by(l - A.batch0, A.batch, inv_batch, i);
            if (b == 0) i = l;
            if (i == 0) {
                // only once the batch in between is known: batches of a block come in the order of their tickets
                const int last = base_of(b + 1);
                const unsigned got = last >= total ? static_cast<unsigned>(last) : atomicAdd(ticket, static_cast<unsigned>(A.batch));
                base_s[(b + 2) % kMxBatches] = (static_cast<unsigned long long>(b + 2) << 32) | got;
            }
            const int base = base_of(b);
            next = base >= total ? 0x7fffffff : base + i;
        }
        return __shfl_sync(0xffffffffu, next, 0);
    };
    const uint32_t ring_u = smem_u32(ring);
    auto issue_one = [&]() {
        // claim tickets until one has slices (or none is left)
        while (ileft == 0) {
            // (a warp takes one task at a time and leaves further tickets to others; with work at hand it waits for none)
            if (!more || task || tail - head >= 32u) return;
            if (head != tail && !__shfl_sync(0xffffffffu, static_cast<int>(lane != 0 || known()), 0)) return;
            const int next = claim();
            if (next >= total) {
                more = false;
                return;
            }
            const int kind = next < n1 ? 0 : next < nq ? 1 : next < n2 ? 2 : 3;
            const int TT = kind == 0 ? U1 : kind == 1 ? nseg : kind == 2 ? U2 : nadd;
            int sub;
            const int en = div_by(next - (kind == 0 ? 0 : kind == 1 ? n1 : kind == 2 ? nq : n2), TT,
                                  kind == 0 ? A.inv_t1 : kind == 1 ? A.inv_seg : kind == 2 ? A.inv_t2 : A.inv_add, sub);
            if (lane == static_cast<int>(tail & 31u))
                fifo = (static_cast<uint32_t>(kind) << 30) | (static_cast<uint32_t>(en) << 16) | static_cast<uint32_t>(sub);
            ++tail;
            if (kind & 1) {
                task = true;
            } else {
                const int C = kind == 0 ? C1 : C2, T = kind == 0 ? T1 : T2;
                isrc = (kind == 0 ? A.w_gu : A.w_dn) +
                       static_cast<size_t>(static_cast<uint32_t>(ent_e[en]) * static_cast<uint32_t>(T) + static_cast<uint32_t>(kTiles * sub)) *
                           static_cast<uint32_t>(C * kRows * kUnit);
                ileft = C;
                if (kMma) isecond = 2 * sub + 1 < T ? static_cast<uint32_t>(C * kRows * kUnit) : 0u;
            }
        }
        const uint32_t n = static_cast<uint32_t>(min(ileft, kLines));
        // (the slot's reads are complete: their values have been used)
        if (elect_one()) {
            const uint32_t bar = bars + 8 * islot;
            const uint32_t dst = ring_u + static_cast<uint32_t>(islot * kSlot);
            mbar_arrive_expect_tx(bar, (kMma && isecond != 0u ? 2u : 1u) * n * (kRows * kUnit));
            bulk_g2s(dst, isrc, n * (kRows * kUnit), bar, pol);
            if (kMma && isecond != 0u) bulk_g2s(dst + kSlot / 2, isrc + isecond, n * (kRows * kUnit), bar, pol);
        }
        __syncwarp();
        isrc += n * (kRows * kUnit);
        ileft -= static_cast<int>(n);
        ++issued;
        if (++islot == S) islot = 0;
    };
    // As many slices in flight as the ring holds, or as there is work known for.
    auto issue = [&]() {
#pragma unroll 1
        while (issued - consumed < S) {
            const int before = issued;
            issue_one();
            if (issued == before) break;
        }
    };
    issue();

    // Looks at words until `there` holds for the whole warp, for a bounded time.
    auto wait_words = [&](auto&& there) {
        if (__all_sync(0xffffffffu, there())) return true;
        const uint64_t t0 = globaltimer_ns();
        while (true) {
            __nanosleep(20);
            if (__all_sync(0xffffffffu, there())) return true;
            if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > kMxWaitNs)) break;
        }
        dead = true;
        if (lane == 0 && A.err != nullptr) atomicExch(A.err, kErrWaitTimeout);
        return false;
    };

    const int hb = lane & 1, pl = lane >> 1, pp = pl & 3;
    const int my_row = 4 * hb + pp;                     // this lane's row of a tile after the butterfly
    const int qd = lane >> 3;                           // and its share of the tokens: m % 4
    int perm[4];                                        // reading order of its four rows (INT8: and of a unit's halves)
#pragma unroll
    for (int j = 0; j < 4; ++j) perm[j] = (j ^ pp) * kUnit + (FMT == FMT_W4 ? 0 : hb << 4);

    while (!dead) {
        if (head == tail) issue();
        if (head == tail) break;
        const uint32_t t = __shfl_sync(0xffffffffu, fifo, static_cast<int>(head & 31u));
        ++head;
        const int kind = static_cast<int>(t >> 30), tile = static_cast<int>(t & 0xffffu);
        if (kind == 1) {
            // -------------------------------------- quantize a piece of h
            const int p = list[(t >> 16) & 0x3fffu];
            const float* hp = A.h + static_cast<size_t>(p) * A.I;
            const int n4 = A.I >> 2;
            constexpr int kPiece = kMxSeg / 4, kEach = kPiece / 32;      // float4 of a piece, and of a lane
            float mx = 0.0f;
            bool ok = true;
            // the largest value of all pieces, the own one last: it stays in registers
            uint4 v[kEach];
            for (int g = 0; g < nseg && ok; ++g) {
                const int i0 = (g + 1 == nseg ? tile : g < tile ? g : g + 1) * kPiece;
                ok = wait_words([&]() {
                    bool all = true;
#pragma unroll
                    for (int k = 0; k < kEach; ++k) {
                        const int i = i0 + 32 * k + lane;
                        v[k] = i < n4 ? ld_relaxed_v4(hp + 4 * i) : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int k = 0; k < kEach; ++k)
                        all = all && v[k].x != kMxNoValue && v[k].y != kMxNoValue && v[k].z != kMxNoValue && v[k].w != kMxNoValue;
                    return all;
                });
#pragma unroll
                for (int k = 0; k < kEach; ++k)
                    mx = fmaxf(fmaxf(mx, fmaxf(fabsf(__uint_as_float(v[k].x)), fabsf(__uint_as_float(v[k].y)))),
                               fmaxf(fabsf(__uint_as_float(v[k].z)), fabsf(__uint_as_float(v[k].w))));
            }
            if (!ok) break;
            mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
            const A8Scale ks = a8_scale(mx);
            const uint64_t rr = f2_pack(ks.r, ks.r);
            // a row of codes for each pair, or (tensor cores) the entry's tokens line by line, 32 codes of each
            uint32_t* qp = reinterpret_cast<uint32_t*>(A.qh + static_cast<size_t>(p) * A.I);
            int qstep = 8;
            if constexpr (kMma) {
                const int at = static_cast<int>((t >> 16) & 0x3fffu), en = of_pos[at];
                qstep = 8 * mx_code(FMT, TK) * ent_n[en];
                qp = reinterpret_cast<uint32_t*>(A.qh + static_cast<size_t>(ent_off[en]) * A.I * mx_code(FMT, TK)) +
                     8 * mx_code(FMT, TK) * (at - ent_off[en]);
            }
            int sum = 0;
            auto quantize = [&](const uint4& u, int i) {
                const float4 f = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
                uint32_t good = 0xffffffffu;
                uint32_t q = a8_pack4_fast2(f, rr, good);
                if (a8_needs_exact(ks) || (good >> 31) == 0u) q = a8_pack4_exact(f, ks);
                if constexpr (kSplit) {
                    // (words of K 0 .. 3 and 4 .. 7 in turn)
                    const uint4 h2 = codes_half(q, q);
                    *reinterpret_cast<uint2*>(qp + (i >> 3) * qstep + ((i & 7) << 1)) = i & 1 ? make_uint2(h2.z, h2.w) : make_uint2(h2.x, h2.y);
                } else if constexpr (kMma) {
                    qp[(i >> 3) * qstep + (i & 7)] = q;
                } else {
                    qp[i] = q;
                }
                sum = __dp4a(static_cast<int>(q), 0x01010101, sum);
            };
            if constexpr (kMma) {
                // (read again: the code for eight at once is long, and other warps run other code meanwhile)
                const int i1 = min(n4, (tile + 1) * kPiece);
#pragma unroll 4
                for (int i = tile * kPiece + lane; i < i1; i += 32) quantize(ld_relaxed_v4(hp + 4 * i), i);
            } else {
#pragma unroll
                for (int k = 0; k < kEach; ++k) {
                    const int i = tile * kPiece + 32 * k + lane;
                    if (i < n4) quantize(v[k], i);
                }
            }
            sum = __reduce_add_sync(0xffffffffu, sum);
            __syncwarp();
            // (the sum as a float: exact, and never the bits of "not written")
            if (lane == 0)
                st_release_u64(A.qdone + static_cast<size_t>(p) * nseg + tile,
                               (static_cast<unsigned long long>(__float_as_uint(__int2float_rn(sum))) << 32) | __float_as_uint(ks.s));
            task = false;
            continue;
        }
        if (kind == 3) {
            // ------------------------------ add the slots of kAdd outputs
            constexpr int kAddSlots = TK <= 2 ? 8 : 1;       // looked at together (as registers allow)
            const int m = static_cast<int>((t >> 16) & 0x3fffu);
            float acc[kAdd / 32];
#pragma unroll
            for (int k = 0; k < kAdd / 32; ++k) acc[k] = 0.0f;
            bool ok = true;
            for (int s0 = 0; s0 < slots && ok; s0 += kAddSlots) {
                // (a slot's values take a trip to L2: several slots at once)
                uint32_t v[kAddSlots][kAdd / 32];
                ok = wait_words([&]() {
                    bool all = true;
#pragma unroll
                    for (int j = 0; j < kAddSlots; ++j) {
                        const int p = m * slots + min(s0 + j, slots - 1);
                        const bool have = s0 + j < slots && pair_e[p] != 0xffff;
#pragma unroll
                        for (int k = 0; k < kAdd / 32; ++k) {
                            const int row = kAdd * tile + 32 * k + lane;
                            v[j][k] = have && row < A.H ? ld_relaxed_u32(A.part + static_cast<size_t>(p) * A.H + row) : 0u;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < kAddSlots; ++j)
#pragma unroll
                        for (int k = 0; k < kAdd / 32; ++k) all = all && v[j][k] != kMxNoValue;
                    return all;
                });
#pragma unroll
                for (int j = 0; j < kAddSlots; ++j) {
                    const int s = s0 + j;
                    if (s >= slots || pair_e[m * slots + s] == 0xffff) continue;
                    const float w = s < A.top_k ? __ldg(A.weights + m * A.top_k + s) : 1.0f;
#pragma unroll
                    for (int k = 0; k < kAdd / 32; ++k) acc[k] = __fmaf_rn(w, __uint_as_float(v[j][k]), acc[k]);
                }
            }
            if (!ok) break;
#pragma unroll
            for (int k = 0; k < kAdd / 32; ++k) {
                const int row = kAdd * tile + 32 * k + lane;
                if (row < A.H) {
                    const size_t o = static_cast<size_t>(m) * A.H + row;
                    float v = acc[k];
                    if (A.residual != nullptr) v = __fadd_rn(A.residual[o], v);
                    store_typed(A.y, A.ytype, o, v);
                }
            }
            task = false;
            continue;
        }
        // ------------------------------------------------ a tile of weights
        const bool down = kind == 2;
        const int en = static_cast<int>((t >> 16) & 0x3fffu);
        const int e = ent_e[en], pos0 = ent_off[en];
        const int cnt = TK == 1 ? 1 : ent_n[en];
        const int C = down ? C2 : C1;
        // this lane's row parameters, wanted at the tile's end
        auto row_params = [&](int row8, float& sw, float& bv) {      // row8: row counted in tiles of eight
            const int row = down ? (row8 < A.H ? row8 : -1) : glu_param_row(row8, A.I);
            const uint32_t at = static_cast<uint32_t>(e) * static_cast<uint32_t>(down ? A.H : 2 * A.I) + static_cast<uint32_t>(row);
            const float* bias = down ? A.b_dn : A.b_gu;
            sw = bv = 0.0f;
            if (row >= 0) {
                sw = __ldg((down ? A.s_dn : A.s_gu) + at);
                if (bias != nullptr) bv = __ldg(bias + at);
            }
        };
        float sw[kTiles], bv[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) row_params(8 * (kTiles * tile + i) + (kMma ? lane >> 2 : my_row), sw[i], bv[i]);
        if (down) {
            // One answer for the warp: another warp may set the byte between two lanes' loads of it, and the code behind the
            // branch votes with all of them.  (Looking twice at finished pieces changes nothing.)
            if (!__all_sync(0xffffffffu, ready_s[en] != 0)) {
                // the pieces of the entry's pairs: there, and their sums (four pieces of eight pairs at a time)
                bool ok = true;
                int sums = 0;
                float scale = 0.0f;
                const unsigned long long* done = A.qdone + static_cast<size_t>(list[pos0 + min(lane & 7, cnt - 1)]) * nseg;
                for (int g0 = 0; g0 < nseg && ok; g0 += 4) {
                    unsigned long long v = 0;
                    const int g = g0 + (lane >> 3);
                    ok = wait_words([&]() {
                        v = ld_acquire_u64(done + min(g, nseg - 1));
                        return static_cast<uint32_t>(v >> 32) != kMxNoValue;
                    });
                    if (g < nseg) sums += __float2int_rn(__uint_as_float(static_cast<uint32_t>(v >> 32)));
                    scale = __uint_as_float(static_cast<uint32_t>(v));
                }
                if (!ok) break;
                sums += __shfl_xor_sync(0xffffffffu, sums, 8);
                sums += __shfl_xor_sync(0xffffffffu, sums, 16);
                if (lane < cnt) {
                    sh_s[pos0 + lane] = scale;
                    hs_s[pos0 + lane] = 8 * sums;
                }
                __syncwarp();
                __threadfence_block();
                if (lane == 0) ready_s[en] = 1;
            }
            __threadfence_block();
        }
        const uint32_t KK = static_cast<uint32_t>(down ? A.I : A.H);
        // Waits for the tile's next slice; false after a wait that ran out.
        auto slice_landed = [&]() {
            const uint32_t bar = bars + 8 * cslot;
            bool ok = __all_sync(0xffffffffu, mbar_test_wait(bar, cph));
            if (!ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, cph, kMxWaitNs));
            if (!ok) {
                dead = true;
                if (lane == 0 && A.err != nullptr) atomicExch(A.err, kErrWaitTimeout);
            }
            __syncwarp();
            return ok;
        };
        auto slice_read = [&]() {
            if (++cslot == S) {
                cslot = 0;
                cph ^= 1u;
            }
            ++consumed;
            __syncwarp();
            issue();
        };
        if constexpr (kMma) {
            constexpr int kCode = mx_code(FMT, TK);
            const int g = lane >> 2, tq = lane & 3, gm = min(g, cnt - 1);
            const uint8_t* xp = down ? reinterpret_cast<const uint8_t*>(A.qh) + static_cast<size_t>(pos0) * A.I * kCode + gm * 32 * kCode
                                     : smem + L.codes + tok_s[pos0 + gm] * HS;
            const int xstep = down ? 32 * kCode * cnt : 32 * kCode;
            xp += 8 * kCode * tq;
            int acc[4] = {0, 0, 0, 0};       // rows g of both tiles by tokens 2 tq, 2 tq + 1
            for (int c = 0; c < C; c += kLines) {
                if (!slice_landed()) break;
                const uint8_t* ub = ring + cslot * kSlot + g * kUnit + tq * (kUnit / 4);
                const int n = min(kLines, C - c);
                if constexpr (FMT == FMT_W4) {
                    // nibble w + 8 at bit 0 or 16 of a pair's half is, as it stands, the fp16 number (w + 8) 2^-24, at
                    // bit 4 16 times that: the sums are multiples of 2^-24 below 1, exact in fp32
                    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f}, d2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    auto lines = [&](auto count) {
                        constexpr int kN = decltype(count)::value;
                        uint32_t w0[kN], w1[kN];
                        uint4 x[kN];
#pragma unroll
                        for (int l = 0; l < kN; ++l) {
                            w0[l] = *reinterpret_cast<const uint32_t*>(ub + l * (kRows * kUnit));
                            w1[l] = *reinterpret_cast<const uint32_t*>(ub + l * (kRows * kUnit) + kSlot / 2);
                            x[l] = *reinterpret_cast<const uint4*>(xp + l * xstep);
                        }
#pragma unroll
                        for (int l = 0; l < kN; ++l) {
                            mma_f16(d, w0[l] & 0x000f000fu, w1[l] & 0x000f000fu, w0[l] & 0x00f000f0u, w1[l] & 0x00f000f0u, x[l].x, x[l].z);
                            const uint32_t v0 = w0[l] >> 8, v1 = w1[l] >> 8;
                            mma_f16(d2, v0 & 0x000f000fu, v1 & 0x000f000fu, v0 & 0x00f000f0u, v1 & 0x00f000f0u, x[l].y, x[l].w);
                        }
                        ub += kN * (kRows * kUnit);
                        xp += kN * xstep;
                    };
                    int l = 0;
#pragma unroll 1
                    for (; l + 8 <= n; l += 8) lines(std::integral_constant<int, 8>());
#pragma unroll 1
                    for (; l < n; ++l) lines(std::integral_constant<int, 1>());
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[i] += __float2int_rn(__fmul_rn(__fadd_rn(d[i], d2[i]), 16777216.0f));
                } else {
                    auto lines = [&](auto count) {
                        constexpr int kN = decltype(count)::value;
                        uint2 w0[kN], w1[kN], x[kN];
#pragma unroll
                        for (int l = 0; l < kN; ++l) {
                            w0[l] = *reinterpret_cast<const uint2*>(ub + l * (kRows * kUnit));
                            w1[l] = *reinterpret_cast<const uint2*>(ub + l * (kRows * kUnit) + kSlot / 2);
                            x[l] = *reinterpret_cast<const uint2*>(xp + l * xstep);
                        }
#pragma unroll
                        for (int l = 0; l < kN; ++l) mma_s8(acc, w0[l].x, w1[l].x, w0[l].y, w1[l].y, x[l].x, x[l].y);
                        ub += kN * (kRows * kUnit);
                        xp += kN * xstep;
                    };
                    if (n == kLines) lines(std::integral_constant<int, kLines>());
                    else
#pragma unroll 1
                        for (int l = 0; l < n; ++l) lines(std::integral_constant<int, 1>());
                }
                slice_read();
            }
            if (dead) break;
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = pos0 + min(2 * tq + (i & 1), cnt - 1), tok = tok_s[at];
                const int a = FMT == FMT_W4 ? acc[i] - (down ? hs_s[at] : xsum_s[tok]) : acc[i];
                v[i] = __fmaf_rn(__fmul_rn(sw[i >> 1], down ? sh_s[at] : sx_s[tok]), __int2float_rn(a), bv[i >> 1]);
            }
            if (down) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = 2 * tq + (i & 1), row = 8 * (2 * tile + (i >> 1)) + g;
                    if (m < cnt && row < A.H) st_value(A.part + static_cast<size_t>(list[pos0 + min(m, cnt - 1)]) * A.H + row, v[i]);
                }
                continue;
            }
            // Rows 0 .. 3 are gates, 4 .. 7 their ups: the lanes of gates take the first tile's values, the others the
            // second's.  Lanes have tokens 2 tq and 2 tq + 1, or (up to four) token tq: one activation instead of two.
            float gt[2], up[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float got = __shfl_xor_sync(0xffffffffu, g < 4 ? v[2 + i] : v[i], 16);
                gt[i] = g < 4 ? v[i] : got;
                up[i] = g < 4 ? got : v[2 + i];
            }
            const int j = 4 * (2 * tile + (g >> 2)) + (g & 3);
            const bool spread = cnt <= 4;
            if (spread) {
                const int from = (lane & 28) | (tq >> 1);
                const float g0 = __shfl_sync(0xffffffffu, gt[0], from), g1 = __shfl_sync(0xffffffffu, gt[1], from);
                const float u0 = __shfl_sync(0xffffffffu, up[0], from), u1 = __shfl_sync(0xffffffffu, up[1], from);
                gt[0] = tq & 1 ? g1 : g0;
                up[0] = tq & 1 ? u1 : u0;
            }
#pragma unroll 1
            for (int i = 0; i < (spread ? 1 : 2); ++i) {
                const int m = spread ? tq : 2 * tq + i;
                if (m < cnt && j < A.I)
                    st_value(A.h + static_cast<size_t>(list[pos0 + m]) * A.I + j, xa_glu(A.glu, i == 0 ? gt[0] : gt[1], i == 0 ? up[0] : up[1]));
            }
            continue;
        } else {
        const int8_t* codes = (down ? A.qh : A.stage_x ? reinterpret_cast<const int8_t*>(smem + L.codes) : A.qx) + pl * 32;
        uint32_t off[TK];
#pragma unroll
        for (int m = 0; m < TK; ++m) {
            const int at = pos0 + min(m, cnt - 1);
            off[m] = static_cast<uint32_t>(down ? list[at] : tok_s[at]) * KK;
        }
        int acc[TK][4], acch[TK][4];             // low and high halves in accumulators of their own
#pragma unroll
        for (int m = 0; m < TK; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[m][j] = 0;
                acch[m][j] = 0;
            }
        for (int c = 0; c < C; c += kLines) {
            if (!slice_landed()) break;
            const uint8_t* ub = ring + cslot * kSlot + (pl * kRows + 4 * hb) * kUnit;
            const int n = min(kLines, C - c) - pl;          // this lane's lines: 0, 16, .. < n
#pragma unroll 2
            for (int l = 0; l < n; l += 16) {
                uint4 w0[4], w1[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (FMT == FMT_W4) {
                        w0[j] = *reinterpret_cast<const uint4*>(ub + perm[j]);
                    } else {
                        // the halves are read in a lane-dependent order to spread the banks
                        const uint4 first = *reinterpret_cast<const uint4*>(ub + perm[j]);
                        const uint4 second = *reinterpret_cast<const uint4*>(ub + (perm[j] ^ 16));
                        w0[j] = hb ? second : first;
                        w1[j] = hb ? first : second;
                    }
                }
#pragma unroll
                for (int m = 0; m < TK; ++m) {
                    if (m == 0 || m < cnt) {
                        const uint4* xp = reinterpret_cast<const uint4*>(codes + off[m]);
                        const uint4 x0 = xp[0], x1 = xp[1];
                        line_dot<FMT>(w0, w1, x0, x1, acc[m], acch[m]);
                    }
                }
                ub += 16 * kRows * kUnit;
                codes += 16 * 32;
            }
            slice_read();
        }
        if (dead) break;
        // lanes of equal (hb, pp) add up, then the read permutation is undone:
        // lane l keeps row my_row of every token (four copies, by lane / 8)
#pragma unroll
        for (int m = 0; m < TK; ++m) {
            if (m < cnt) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[m][j] += FMT == FMT_W4 ? acch[m][j] >> 4 : acch[m][j];
                    acc[m][j] += __shfl_xor_sync(0xffffffffu, acc[m][j], 8);
                    acc[m][j] += __shfl_xor_sync(0xffffffffu, acc[m][j], 16);
                }
                acc[m][0] += __shfl_xor_sync(0xffffffffu, acc[m][2], 4);
                acc[m][1] += __shfl_xor_sync(0xffffffffu, acc[m][3], 4);
                acc[m][0] += __shfl_xor_sync(0xffffffffu, acc[m][1], 2);
            }
        }
#pragma unroll
        for (int i = 0; i < (TK + 3) / 4; ++i) {
            const int m = 4 * i + qd;                   // this lane's token
            if (4 * i >= cnt) break;
            int a = acc[4 * i][0];
#pragma unroll
            for (int q = 1; q < 4; ++q)
                if (4 * i + q < TK && qd == q) a = acc[4 * i + q < TK ? 4 * i + q : 0][0];
            const bool have = m < cnt;
            const int at = pos0 + min(m, cnt - 1);
            const int p = list[at];
            if (down) {
                if (FMT == FMT_W4) a -= hs_s[at];
                const int row = 8 * tile + my_row;
                if (have && row < A.H)
                    st_value(A.part + static_cast<size_t>(p) * A.H + row, __fmaf_rn(__fmul_rn(sw[0], sh_s[at]), __int2float_rn(a), bv[0]));
            } else {
                const int tok = tok_s[at];
                if (FMT == FMT_W4) a -= xsum_s[tok];
                const float v = __fmaf_rn(__fmul_rn(sw[0], sx_s[tok]), __int2float_rn(a), bv[0]);
                const float u = __shfl_xor_sync(0xffffffffu, v, 1);      // gate lanes are even, up lanes odd
                const int j = 4 * tile + pp;
                if (have && hb == 0 && j < A.I) st_value(A.h + static_cast<size_t>(p) * A.I + j, xa_glu(A.glu, v, u));
            }
        }
        }
    }
    // after a wait that ran out: the copies in flight land before the block ends
    if (dead)
        for (int k = consumed; k < issued; ++k)
            if (!mbar_wait_bounded(bars + 8 * (k % S), static_cast<uint32_t>(k / S) & 1u, kMxWaitNs)) break;
}

__global__ void __launch_bounds__(256) moe_fill_kernel(const MoeFill f)
{
    pdl_launch_dependents();
    pdl_wait();
    moe_fill(f);
}

template <int FMT, int TK>
cudaError_t launch_experts_t(const MoeArgs& a, int grid, int warps, size_t smem, bool pdl, cudaStream_t s)
{
    auto kern = moe_experts_kernel<FMT, TK>;
    static SmemLimit limit;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), limit, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int FMT>
cudaError_t launch_experts_f(int tok, const MoeArgs& a, int grid, int warps, size_t smem, bool pdl, cudaStream_t s)
{
    if (tok <= 1) return launch_experts_t<FMT, 1>(a, grid, warps, smem, pdl, s);
    if (tok <= 2) return launch_experts_t<FMT, 2>(a, grid, warps, smem, pdl, s);
    return launch_experts_t<FMT, 8>(a, grid, warps, smem, pdl, s);
}

}  // namespace

MoePlan moe_plan(int fmt, int tok, int M, int H, size_t most)
{
    MoePlan p;
    p.tiles = mx_mma(tok) ? 2 : 1;
    p.warps = mx_warps(tok);
    const size_t staged = static_cast<size_t>(M) * static_cast<size_t>(mx_stride(fmt, tok, H));
    auto total = [&](size_t codes) { return static_cast<size_t>(mx_smem(tok, p.warps, 0).total) + codes; };
    while (mx_mma(tok) && p.warps > kMxFewestWarps && total(staged) > most) --p.warps;
    p.staged = total(staged) <= most;
    p.smem = total(p.staged ? staged : 0);
    p.fits = p.smem <= most && (p.staged || !mx_mma(tok));
    return p;
}

cudaError_t launch_moe_experts(int fmt, int tok, const MoeArgs& a, int grid, int warps, size_t smem, bool pdl, cudaStream_t s)
{
    return fmt == FMT_W4 ? launch_experts_f<FMT_W4>(tok, a, grid, warps, smem, pdl, s)
                         : launch_experts_f<FMT_W8F>(tok, a, grid, warps, smem, pdl, s);
}

cudaError_t launch_moe_fill(const MoeFill& f, bool pdl, cudaStream_t s)
{
    const unsigned words = kMxHead / 4 + f.values;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(words < 256u * 256u ? (words + 255u) / 256u : 256u);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, moe_fill_kernel, f);
}

}  // namespace w4k
