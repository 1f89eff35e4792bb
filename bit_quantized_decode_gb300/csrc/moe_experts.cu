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
//   * An entry is an expert and up to eight of its tokens; a lane holds four
//     rows by eight tokens of integer sums (DP4A, as the decode GEMV: line
//     lane / 2 of a 16-line pass, rows 4 (lane & 1) .. + 3, reads permuted
//     against bank conflicts, a shuffle butterfly at the end of a tile).
//     More tokens of one expert are further entries.
//   * No fence per tile (it waits for all that the warp has outstanding: it
//     took 3500 of a tile's 9500 cycles): hidden values and the slots' outputs
//     are prepared with a value that no result takes (MoeFill), and a reader
//     looks at the words themselves until every one is there.  Only the few
//     quantizing tasks publish their codes with release order, which the tiles
//     that read them through L1 acquire.
//   * Adding tasks, the last tickets, sum the slots' outputs in order: no
//     floating-point atomics, so results do not depend on timing.
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
// sums per weight) the slots are large; with more, more warps.
__host__ __device__ constexpr int mx_slot(int tok) { return tok <= 2 ? 8192 : 4096; }
__host__ __device__ constexpr int mx_stages(int) { return 2; }
__host__ __device__ constexpr int mx_warps(int tok) { return tok <= 2 ? 12 : tok <= 4 ? 20 : 16; }

constexpr int kMxBatches = 64;

struct MxSmem {
    int bars, mask, off, ent0, pair_e, list, tok, ent_e, ent_off, ent_n, of_pos, ready, sh, hs, sx, xsum, misc, base, ring, codes, total;
};
__host__ __device__ inline MxSmem mx_smem(int tok, int staged)
{
    const int warps = mx_warps(tok), stages = mx_stages(tok);
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

template <int FMT, int TK>
__global__ void __launch_bounds__(32 * mx_warps(TK), 1) moe_experts_kernel(const __grid_constant__ MoeArgs A)
{
    constexpr int NW = mx_warps(TK), NT = 32 * NW;
    constexpr int kUnit = mx_unit(FMT), kSlot = mx_slot(TK), kLines = kSlot / (kRows * kUnit);
    static_assert(kLines % 16 == 0, "slices of whole passes: every lane steps through the codes alike");
    constexpr bool kPairSums = TK <= 4;            // low and high halves in accumulators of their own
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int S = mx_stages(TK);
    const MxSmem L = mx_smem(TK, 0);
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
    unsigned* ticket = A.ticket;

    uint8_t* ring = smem + L.ring + static_cast<size_t>(warp) * S * kSlot;
    const uint32_t bars = smem_u32(smem + L.bars) + static_cast<uint32_t>(warp * S) * 8u;
    if (lane == 0) {
        for (int s = 0; s < S; ++s) mbar_init(bars + 8 * s, 1);
        if (warp == 1) mbar_init(smem_u32(smem + L.bars) + static_cast<uint32_t>(NW * S) * 8u, 1);
        fence_mbar_init();
    }
    if (tid > 0 && tid < kMxBatches) base_s[tid] = ~0ull;
    if (tid == NT - 1) misc[2] = 0;
    const int EE = A.E + A.S;
    if (TK > 1)
        for (int e = tid; e < EE; e += NT) mask_s[e] = 0u;
    for (int i = tid; i < P; i += NT) ready_s[i] = 0;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();

    // ---- the entries, the same in every block: pairs counted by expert in
    // the order of the pairs (warp 0); scales and code sums of the tokens (the others)
    if (tid == NT - 1) base_s[0] = atomicAdd(ticket, static_cast<unsigned>(A.batch));
    // (the codes before any weights: behind those a load waits for microseconds)
    const uint32_t xbar = smem_u32(smem + L.bars) + static_cast<uint32_t>(NW * S) * 8u;
    if (A.stage_x && tid == 32) {
        mbar_arrive_expect_tx(xbar, static_cast<uint32_t>(A.M * A.H));
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         smem_u32(smem + L.codes)),
                     "l"(A.qx), "r"(static_cast<uint32_t>(A.M * A.H)), "r"(xbar)
                     : "memory");
    }
    auto expert_of = [&](int p) -> int {
        const int m = p / slots, s = p - m * slots;
        if (s >= A.top_k) return A.E + s - A.top_k;
        const int e = __ldg(A.ids + m * A.top_k + s);
        return e < 0 || e >= A.E ? 0xffff : e;
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
        static_assert(kMxMaxPairs <= 320 && NT >= 320, "a thread for each pair");
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
    if (warp > 0) {
        bool ok = true;
        if (A.stage_x) ok = mbar_wait_bounded(xbar, 0u, kMxWaitNs);
        if (!ok && A.err != nullptr) atomicExch(A.err, kErrWaitTimeout);
        const int8_t* src = A.stage_x ? reinterpret_cast<const int8_t*>(smem + L.codes) : A.qx;
        for (int m = warp - 1; m < A.M; m += NW - 1) {
            int s = 0;
            if (FMT == FMT_W4) {                                            // for the nibble bias
                const uint4* q = reinterpret_cast<const uint4*>(src + static_cast<size_t>(m) * A.H);
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
    const int nadd = (A.H + kMxAdd - 1) / kMxAdd;
    const int n1 = NE * T1, nq = n1 + PV * nseg, n2 = nq + NE * T2, total = n2 + A.M * nadd;

    // ---- tickets.  A block takes them from the global counter a batch at a
    // time (thousands of warps on one counter would wait for it: some 2 ns
    // each), its warps from a counter of their own; the warp that opens a batch
    // fetches the next.  Claimed tickets wait in the lanes of `fifo` until
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
    bool more = true;
    const float inv_batch = 1.0f / static_cast<float>(A.batch);
    // The next ticket, or one past the last.
    auto claim = [&]() -> int {
        int next = 0;
        if (lane == 0) {
            int i;
            const int l = atomicAdd(const_cast<int*>(misc + 2), 1);
            const int b = div_by(l, A.batch, inv_batch, i);
            if (i == 0) {
                const unsigned long long got = atomicAdd(ticket, static_cast<unsigned>(A.batch));
                base_s[(b + 1) % kMxBatches] = (static_cast<unsigned long long>(b + 1) << 32) | got;
            }
            unsigned long long v = base_s[b % kMxBatches];
            if (static_cast<int>(v >> 32) != b) {
                const uint64_t t0 = globaltimer_ns();
                while (static_cast<int>((v = base_s[b % kMxBatches]) >> 32) != b) {
                    if (globaltimer_ns() - t0 > kMxWaitNs) {
                        if (A.err != nullptr) atomicExch(A.err, kErrWaitTimeout);
                        break;
                    }
                }
            }
            next = static_cast<int>(v >> 32) == b ? static_cast<int>(static_cast<uint32_t>(v)) + i : 0x7fffffff;
        }
        return __shfl_sync(0xffffffffu, next, 0);
    };
    const uint32_t ring_u = smem_u32(ring);
    auto issue_one = [&]() {
        // claim tickets until one has slices (or none is left)
        while (ileft == 0) {
            if (!more || tail - head >= 32u) return;
            const int next = claim();
            if (next >= total) {
                more = false;
                return;
            }
            const int kind = next < n1 ? 0 : next < nq ? 1 : next < n2 ? 2 : 3;
            const int TT = kind == 0 ? T1 : kind == 1 ? nseg : kind == 2 ? T2 : nadd;
            int sub;
            const int en = div_by(next - (kind == 0 ? 0 : kind == 1 ? n1 : kind == 2 ? nq : n2), TT,
                                  kind == 0 ? A.inv_t1 : kind == 1 ? A.inv_seg : kind == 2 ? A.inv_t2 : A.inv_add, sub);
            if (lane == static_cast<int>(tail & 31u))
                fifo = (static_cast<uint32_t>(kind) << 30) | (static_cast<uint32_t>(en) << 16) | static_cast<uint32_t>(sub);
            ++tail;
            if (!(kind & 1)) {
                const int C = kind == 0 ? C1 : C2;
                isrc = (kind == 0 ? A.w_gu : A.w_dn) +
                       static_cast<size_t>(static_cast<uint32_t>(ent_e[en]) * static_cast<uint32_t>(TT) + static_cast<uint32_t>(sub)) *
                           static_cast<uint32_t>(C * kRows * kUnit);
                ileft = C;
            }
        }
        const uint32_t n = static_cast<uint32_t>(min(ileft, kLines));
        // (the slot's reads are complete: their values have been used)
        if (elect_one()) {
            const uint32_t bar = bars + 8 * islot;
            mbar_arrive_expect_tx(bar, n * (kRows * kUnit));
            bulk_g2s(ring_u + static_cast<uint32_t>(islot * kSlot), isrc, n * (kRows * kUnit), bar, pol);
        }
        __syncwarp();
        isrc += n * (kRows * kUnit);
        ileft -= static_cast<int>(n);
        ++issued;
        if (++islot == S) islot = 0;
    };
    for (int s = 0; s < S; ++s) issue_one();

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
        if (head == tail) issue_one();
        if (head == tail) break;
        const uint32_t t = __shfl_sync(0xffffffffu, fifo, static_cast<int>(head & 31u));
        ++head;
        const int kind = static_cast<int>(t >> 30), tile = static_cast<int>(t & 0xffffu);
        if (kind == 1) {
            // -------------------------------------- quantize a piece of h
            const int p = list[(t >> 16) & 0x3fffu];
            const float* hp = A.h + static_cast<size_t>(p) * A.I;
            const int n4 = A.I >> 2;
            float mx = 0.0f;
            bool ok = true;
            for (int i0 = 0; i0 < n4 && ok; i0 += 8 * 32) {
                uint4 v[8];
                ok = wait_words([&]() {
                    bool all = true;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int i = i0 + 32 * k + lane;
                        v[k] = i < n4 ? ld_relaxed_v4(hp + 4 * i) : make_uint4(0u, 0u, 0u, 0u);
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        all = all && v[k].x != kMxNoValue && v[k].y != kMxNoValue && v[k].z != kMxNoValue && v[k].w != kMxNoValue;
                    return all;
                });
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mx = fmaxf(fmaxf(mx, fmaxf(fabsf(__uint_as_float(v[k].x)), fabsf(__uint_as_float(v[k].y)))),
                               fmaxf(fabsf(__uint_as_float(v[k].z)), fabsf(__uint_as_float(v[k].w))));
            }
            if (!ok) break;
            mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
            const A8Scale ks = a8_scale(mx);
            const uint64_t rr = f2_pack(ks.r, ks.r);
            uint32_t* qp = reinterpret_cast<uint32_t*>(A.qh + static_cast<size_t>(p) * A.I);
            const int i1 = min(n4, (tile + 1) * (kMxSeg / 4));
            int sum = 0;
#pragma unroll 4
            for (int i = tile * (kMxSeg / 4) + lane; i < i1; i += 32) {
                const uint4 u = ld_relaxed_v4(hp + 4 * i);
                const float4 v = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
                uint32_t good = 0xffffffffu;
                uint32_t q = a8_pack4_fast2(v, rr, good);
                if (a8_needs_exact(ks) || (good >> 31) == 0u) q = a8_pack4_exact(v, ks);
                qp[i] = q;
                sum = __dp4a(static_cast<int>(q), 0x01010101, sum);
            }
            sum = __reduce_add_sync(0xffffffffu, sum);
            __syncwarp();
            // (the sum as a float: exact, and never the bits of "not written")
            if (lane == 0)
                st_release_u64(A.qdone + static_cast<size_t>(p) * nseg + tile,
                               (static_cast<unsigned long long>(__float_as_uint(__int2float_rn(sum))) << 32) | __float_as_uint(ks.s));
            continue;
        }
        if (kind == 3) {
            // ------------------------------ add the slots of 256 outputs
            const int m = static_cast<int>((t >> 16) & 0x3fffu);
            float acc[kMxAdd / 32];
#pragma unroll
            for (int k = 0; k < kMxAdd / 32; ++k) acc[k] = 0.0f;
            bool ok = true;
            for (int s = 0; s < slots && ok; ++s) {
                const int p = m * slots + s;
                if (pair_e[p] == 0xffff) continue;
                const float w = s < A.top_k ? __ldg(A.weights + m * A.top_k + s) : 1.0f;
                const float* pp_ = A.part + static_cast<size_t>(p) * A.H;
                uint32_t v[kMxAdd / 32];
                ok = wait_words([&]() {
                    bool all = true;
#pragma unroll
                    for (int k = 0; k < kMxAdd / 32; ++k) {
                        const int row = kMxAdd * tile + 32 * k + lane;
                        v[k] = row < A.H ? ld_relaxed_u32(pp_ + row) : 0u;
                    }
#pragma unroll
                    for (int k = 0; k < kMxAdd / 32; ++k) all = all && v[k] != kMxNoValue;
                    return all;
                });
#pragma unroll
                for (int k = 0; k < kMxAdd / 32; ++k) acc[k] = __fmaf_rn(w, __uint_as_float(v[k]), acc[k]);
            }
            if (!ok) break;
#pragma unroll
            for (int k = 0; k < kMxAdd / 32; ++k) {
                const int row = kMxAdd * tile + 32 * k + lane;
                if (row < A.H) {
                    const size_t o = static_cast<size_t>(m) * A.H + row;
                    float v = acc[k];
                    if (A.residual != nullptr) v = __fadd_rn(A.residual[o], v);
                    store_typed(A.y, A.ytype, o, v);
                }
            }
            continue;
        }
        // ------------------------------------------------ a tile of weights
        const bool down = kind == 2;
        const int en = static_cast<int>((t >> 16) & 0x3fffu);
        const int e = ent_e[en], pos0 = ent_off[en];
        const int cnt = TK == 1 ? 1 : ent_n[en];
        const int C = down ? C2 : C1;
        const int8_t* codes = (down ? A.qh : A.stage_x ? reinterpret_cast<const int8_t*>(smem + L.codes) : A.qx) + pl * 32;
        // this lane's row parameters, wanted at the tile's end
        float sw = 0.0f, bv = 0.0f;
        {
            const int row = down ? (8 * tile + my_row < A.H ? 8 * tile + my_row : -1) : glu_param_row(8 * tile + my_row, A.I);
            const uint32_t at = static_cast<uint32_t>(e) * static_cast<uint32_t>(down ? A.H : 2 * A.I) + static_cast<uint32_t>(row);
            const float* bias = down ? A.b_dn : A.b_gu;
            if (row >= 0) {
                sw = __ldg((down ? A.s_dn : A.s_gu) + at);
                if (bias != nullptr) bv = __ldg(bias + at);
            }
        }
        if (down) {
            if (ready_s[en] == 0) {
                // the pieces of the entry's pairs: there, and their sums
                bool ok = true;
                int sums = 0;
                float scale = 0.0f;
                for (int g = 0; g < nseg && ok; ++g) {
                    unsigned long long v = 0;
                    const int p = list[pos0 + min(lane, cnt - 1)];
                    ok = wait_words([&]() {
                        v = ld_acquire_u64(A.qdone + static_cast<size_t>(p) * nseg + g);
                        return static_cast<uint32_t>(v >> 32) != kMxNoValue;
                    });
                    sums += __float2int_rn(__uint_as_float(static_cast<uint32_t>(v >> 32)));
                    scale = __uint_as_float(static_cast<uint32_t>(v));
                }
                if (!ok) break;
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
        uint32_t off[TK];
        const uint32_t KK = static_cast<uint32_t>(down ? A.I : A.H);
#pragma unroll
        for (int m = 0; m < TK; ++m) {
            const int at = pos0 + min(m, cnt - 1);
            off[m] = static_cast<uint32_t>(down ? list[at] : tok_s[at]) * KK;
        }
        int acc[TK][4], acch[kPairSums ? TK : 1][4];
#pragma unroll
        for (int m = 0; m < TK; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[m][j] = 0;
                if (kPairSums) acch[m][j] = 0;
            }
        for (int c = 0; c < C; c += kLines) {
            const uint32_t bar = bars + 8 * cslot;
            bool ok = __all_sync(0xffffffffu, mbar_test_wait(bar, cph));
            if (!ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, cph, kMxWaitNs));
            if (!ok) {
                dead = true;
                if (lane == 0 && A.err != nullptr) atomicExch(A.err, kErrWaitTimeout);
                break;
            }
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
                        if constexpr (kPairSums) {
                            line_dot<FMT>(w0, w1, x0, x1, acc[m], acch[m]);
                        } else {
                            int hi[4] = {0, 0, 0, 0};
                            line_dot<FMT>(w0, w1, x0, x1, acc[m], hi);
#pragma unroll
                            for (int j = 0; j < 4; ++j) acc[m][j] += FMT == FMT_W4 ? hi[j] >> 4 : hi[j];
                        }
                    }
                }
                ub += 16 * kRows * kUnit;
                codes += 16 * 32;
            }
            if (++cslot == S) {
                cslot = 0;
                cph ^= 1u;
            }
            ++consumed;
            __syncwarp();
            issue_one();
        }
        if (dead) break;
        // lanes of equal (hb, pp) add up, then the read permutation is undone:
        // lane l keeps row my_row of every token (four copies, by lane / 8)
#pragma unroll
        for (int m = 0; m < TK; ++m) {
            if (m < cnt) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (kPairSums) acc[m][j] += FMT == FMT_W4 ? acch[m][j] >> 4 : acch[m][j];
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
                    st_value(A.part + static_cast<size_t>(p) * A.H + row, __fmaf_rn(__fmul_rn(sw, sh_s[at]), __int2float_rn(a), bv));
            } else {
                const int tok = tok_s[at];
                if (FMT == FMT_W4) a -= xsum_s[tok];
                const float v = __fmaf_rn(__fmul_rn(sw, sx_s[tok]), __int2float_rn(a), bv);
                const float u = __shfl_xor_sync(0xffffffffu, v, 1);      // gate lanes are even, up lanes odd
                const int j = 4 * tile + pp;
                if (have && hb == 0 && j < A.I) st_value(A.h + static_cast<size_t>(p) * A.I + j, xa_glu(A.glu, v, u));
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
cudaError_t launch_experts_t(const MoeArgs& a, int grid, size_t smem, bool pdl, cudaStream_t s)
{
    auto kern = moe_experts_kernel<FMT, TK>;
    static SmemLimit limit;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), limit, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(32 * mx_warps(TK));
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
cudaError_t launch_experts_f(int tok, const MoeArgs& a, int grid, size_t smem, bool pdl, cudaStream_t s)
{
    if (tok <= 1) return launch_experts_t<FMT, 1>(a, grid, smem, pdl, s);
    if (tok <= 2) return launch_experts_t<FMT, 2>(a, grid, smem, pdl, s);
    if (tok <= 4) return launch_experts_t<FMT, 4>(a, grid, smem, pdl, s);
    return launch_experts_t<FMT, 8>(a, grid, smem, pdl, s);
}

}  // namespace

int moe_warps(int tok) { return mx_warps(tok); }
size_t moe_experts_smem(int tok, int staged_bytes)
{
    return static_cast<size_t>(mx_smem(tok, staged_bytes).total);
}

cudaError_t launch_moe_experts(int fmt, int tok, const MoeArgs& a, int grid, size_t smem, bool pdl, cudaStream_t s)
{
    return fmt == FMT_W4 ? launch_experts_f<FMT_W4>(tok, a, grid, smem, pdl, s)
                         : launch_experts_f<FMT_W8F>(tok, a, grid, smem, pdl, s);
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
