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
//   * Counters with release / acquire order carry the dependencies: tiles
//     done per entry, tasks done per entry, entries done per output tile.  The
//     warp that finishes an output tile's last entry adds the slots up, in
//     order: no floating-point atomics, so results do not depend on timing.
//   * The hidden maximum is an integer atomic maximum over the bits of |h|.
#include "exact_act.cuh"
#include "operators.h"
#include "ptx.cuh"
#include "quant_a8.cuh"
#include "typed_io.cuh"

namespace w4k {
namespace {

constexpr uint64_t kMxWaitNs = 250ull * 1000ull * 1000ull;

__host__ __device__ constexpr int mx_unit(int fmt) { return fmt == FMT_W4 ? 16 : 32; }
__host__ __device__ constexpr int mx_slot(int fmt) { return kMxLines * kRows * mx_unit(fmt); }

struct MxSmem {
    int bars, cnt, off, pair_e, list, ent_e, ent_off, of_pos, ready, xsum, misc, ring, total;
};
__host__ __device__ inline MxSmem mx_smem(int fmt, int stages)
{
    MxSmem L;
    int o = 0;
    L.bars = o;    o += kMxWarps * 8 * 8;
    L.cnt = o;     o += kMxMaxExperts * 2;             // pairs per expert
    L.off = o;     o += kMxMaxExperts * 2;             // first place of an expert's pairs in the list
    L.pair_e = o;  o += kMxMaxPairs * 2;               // expert of a pair (0xffff: none)
    L.list = o;    o += kMxMaxPairs * 2;               // pairs ordered by expert
    L.ent_e = o;   o += kMxMaxPairs * 2;
    L.ent_off = o; o += (kMxMaxPairs + 2) * 2;         // first place of an entry's pairs
    L.of_pos = o;  o += kMxMaxPairs * 2;               // entry of a place
    L.ready = o;   o += kMxMaxPairs;                   // the entry's hidden codes were seen complete
    L.xsum = o;    o += 16 * 4;
    L.misc = o;    o += 16;
    o = align_up(o, 128);
    L.ring = o;    o += kMxWarps * stages * mx_slot(fmt);
    L.total = o;
    return L;
}

__device__ __forceinline__ unsigned ld_volatile_s8(const volatile uint8_t* p) { return *p; }

// One lane's share of a slice: four rows of its line against MT tokens.
template <int FMT, int MT>
__device__ __forceinline__ void slice_dot(const uint8_t* slot, int pl, int h, int pp, const int8_t* codes,
                                          const uint32_t (&off)[kMxTok], int cnt, int (&acc)[kMxTok][4], int (&accA)[4][4])
{
    const uint8_t* ub = slot + (pl * kRows + 4 * h) * mx_unit(FMT);
    uint4 w0[4], w1[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (FMT == FMT_W4) {
            w0[j] = *reinterpret_cast<const uint4*>(ub + ((j ^ pp) << 4));
        } else {
            const uint8_t* u = ub + ((j ^ pp) << 5);
            const uint4 first = *reinterpret_cast<const uint4*>(u + (h << 4));
            const uint4 second = *reinterpret_cast<const uint4*>(u + ((h ^ 1) << 4));
            w0[j] = h ? second : first;
            w1[j] = h ? first : second;
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        if (MT == 1 || m < cnt) {
            const uint4* xp = reinterpret_cast<const uint4*>(codes + off[m]);
            const uint4 x0 = xp[0], x1 = xp[1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (FMT == FMT_W4) {
                    // low nibbles into acc, high nibbles (16 n) into accA or shifted back
                    auto us = [](uint32_t a, uint32_t b, int c) {
                        int d;
                        asm("dp4a.u32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
                        return d;
                    };
                    const uint4 w = w0[j];
                    acc[m][j] = us(w.x & 0x0F0F0F0Fu, x0.x, acc[m][j]);
                    acc[m][j] = us(w.y & 0x0F0F0F0Fu, x0.z, acc[m][j]);
                    acc[m][j] = us(w.z & 0x0F0F0F0Fu, x1.x, acc[m][j]);
                    acc[m][j] = us(w.w & 0x0F0F0F0Fu, x1.z, acc[m][j]);
                    int A = MT <= 4 ? accA[m & 3][j] : 0;
                    A = us(w.x & 0xF0F0F0F0u, x0.y, A);
                    A = us(w.y & 0xF0F0F0F0u, x0.w, A);
                    A = us(w.z & 0xF0F0F0F0u, x1.y, A);
                    A = us(w.w & 0xF0F0F0F0u, x1.w, A);
                    if (MT <= 4) accA[m & 3][j] = A;
                    else acc[m][j] += A >> 4;
                } else {
                    int g = dp4a_ss(w0[j].x, x0.x, acc[m][j]);
                    g = dp4a_ss(w0[j].y, x0.y, g);
                    g = dp4a_ss(w0[j].z, x0.z, g);
                    g = dp4a_ss(w0[j].w, x0.w, g);
                    g = dp4a_ss(w1[j].x, x1.x, g);
                    g = dp4a_ss(w1[j].y, x1.y, g);
                    g = dp4a_ss(w1[j].z, x1.z, g);
                    acc[m][j] = dp4a_ss(w1[j].w, x1.w, g);
                }
            }
        }
    }
}

template <int FMT>
__global__ void __launch_bounds__(kMxThreads, 1) moe_experts_kernel(const __grid_constant__ MoeArgs A)
{
    extern __shared__ __align__(128) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = A.stages;
    const MxSmem L = mx_smem(FMT, S);
    uint16_t* cnt_s = reinterpret_cast<uint16_t*>(smem + L.cnt);
    uint16_t* off_s = reinterpret_cast<uint16_t*>(smem + L.off);
    uint16_t* pair_e = reinterpret_cast<uint16_t*>(smem + L.pair_e);
    uint16_t* list = reinterpret_cast<uint16_t*>(smem + L.list);
    uint16_t* ent_e = reinterpret_cast<uint16_t*>(smem + L.ent_e);
    uint16_t* ent_off = reinterpret_cast<uint16_t*>(smem + L.ent_off);
    uint16_t* of_pos = reinterpret_cast<uint16_t*>(smem + L.of_pos);
    volatile uint8_t* ready_s = smem + L.ready;
    int* xsum_s = reinterpret_cast<int*>(smem + L.xsum);
    volatile int* misc = reinterpret_cast<volatile int*>(smem + L.misc);       // [0] entries, [1] pairs, [2] first ticket

    const int slots = A.top_k + A.S;
    const int P = A.M * slots;
    const int C1 = A.H >> 5, C2 = A.I >> 5;
    const int T1 = (A.I + 3) >> 2, T2 = (A.H + 7) >> 3;
    unsigned* ticket = A.ctrl;
    unsigned* hmax = A.ctrl + 4;
    int* hsum = reinterpret_cast<int*>(hmax + P);
    unsigned* done1 = reinterpret_cast<unsigned*>(hsum + P);
    unsigned* doneq = done1 + P;
    unsigned* done2 = doneq + P;

    uint8_t* ring = smem + L.ring + static_cast<size_t>(warp) * S * mx_slot(FMT);
    const uint32_t bars = smem_u32(smem + L.bars) + static_cast<uint32_t>(warp) * 64u;
    if (lane == 0) {
        for (int s = 0; s < S; ++s) mbar_init(bars + 8 * s, 1);
        fence_mbar_init();
    }
    const int EE = A.E + A.S;
    for (int e = tid; e < EE; e += kMxThreads) cnt_s[e] = 0;
    for (int i = tid; i < kMxMaxPairs; i += kMxThreads) ready_s[i] = 0;
    pdl_launch_dependents();
    pdl_wait();

    // ---- the entries, the same in every block: pairs counted by expert in
    // the order of the pairs (warp 0), code sums of the tokens (the others)
    for (int p = tid; p < P; p += kMxThreads) {
        const int m = p / slots, s = p - m * slots;
        int e;
        if (s < A.top_k) {
            e = __ldg(A.ids + m * A.top_k + s);
            if (e < 0 || e >= A.E) e = 0xffff;
        } else {
            e = A.E + s - A.top_k;
        }
        pair_e[p] = static_cast<uint16_t>(e);
    }
    if (tid == 0) misc[2] = static_cast<int>(atomicAdd(ticket, static_cast<unsigned>(kMxWarps)));
    __syncthreads();
    if (warp == 0) {
        for (int p0 = 0; p0 < P; p0 += 32) {
            const int p = p0 + lane;
            const int e = p < P ? pair_e[p] : 0xffff;
            const unsigned same = __match_any_sync(0xffffffffu, e);
            const int rank = __popc(same & ((1u << lane) - 1u));
            int base = 0;
            if (e != 0xffff) base = cnt_s[e];
            __syncwarp();
            if (e != 0xffff) {
                list[p] = static_cast<uint16_t>(base + rank);           // rank for now
                if (rank == 0) cnt_s[e] = static_cast<uint16_t>(base + __popc(same));
            }
            __syncwarp();
        }
        int at = 0, ne = 0;
        for (int e0 = 0; e0 < EE; e0 += 32) {
            const int c = e0 + lane < EE ? cnt_s[e0 + lane] : 0;
            const int k = (c + kMxTok - 1) / kMxTok;
            int sc = c, sk = k;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int vc = __shfl_up_sync(0xffffffffu, sc, o), vk = __shfl_up_sync(0xffffffffu, sk, o);
                if (lane >= o) {
                    sc += vc;
                    sk += vk;
                }
            }
            if (c > 0) {
                const int a0 = at + sc - c, n0 = ne + sk - k;
                off_s[e0 + lane] = static_cast<uint16_t>(a0);
                for (int i = 0; i < k; ++i) {
                    ent_e[n0 + i] = static_cast<uint16_t>(e0 + lane);
                    ent_off[n0 + i] = static_cast<uint16_t>(a0 + i * kMxTok);
                    for (int q = i * kMxTok; q < min(c, (i + 1) * kMxTok); ++q) of_pos[a0 + q] = static_cast<uint16_t>(n0 + i);
                }
            }
            at += __shfl_sync(0xffffffffu, sc, 31);
            ne += __shfl_sync(0xffffffffu, sk, 31);
        }
        __syncwarp();
        if (lane == 0) {
            misc[0] = ne;
            misc[1] = at;
            ent_off[ne] = static_cast<uint16_t>(at);
        }
        // ranks to places (each pair's rank is read before any place is written)
        __syncwarp();
        int place[kMxMaxPairs / 32];
#pragma unroll
        for (int i = 0; i < kMxMaxPairs / 32; ++i) {
            const int p = 32 * i + lane;
            place[i] = p < P && pair_e[p] != 0xffff ? off_s[pair_e[p]] + list[p] : -1;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kMxMaxPairs / 32; ++i)
            if (place[i] >= 0) list[place[i]] = static_cast<uint16_t>(32 * i + lane);
    } else if (FMT == FMT_W4) {
        // the nibble bias: code sums of the tokens
        for (int m = warp - 1; m < A.M; m += kMxWarps - 1) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>(A.qx + static_cast<size_t>(m) * A.H);
            int s = 0;
            for (int i = lane; i < A.H / 4; i += 32) s = __dp4a(static_cast<int>(__ldg(q + i)), 0x01010101, s);
            s = __reduce_add_sync(0xffffffffu, s);
            if (lane == 0) xsum_s[m] = s;
        }
    }
    __syncthreads();
    const int NE = misc[0], PV = misc[1];
    const int nseg = (A.I + kMxSeg - 1) / kMxSeg;
    const int n1 = NE * T1, nq = PV * nseg, total = n1 + nq + NE * T2;

    // the output of a token without any expert: the residual
    auto add_up = [&](int t) {
        for (int i = lane; i < A.M * 8; i += 32) {
            const int m = i >> 3, row = 8 * t + (i & 7);
            if (row >= A.H) continue;
            float v = 0.0f;
            for (int s = 0; s < slots; ++s) {
                const int p = m * slots + s;
                if (pair_e[p] == 0xffff) continue;
                const float w = s < A.top_k ? __ldg(A.weights + m * A.top_k + s) : 1.0f;
                v = __fmaf_rn(w, __ldcg(A.part + static_cast<size_t>(p) * A.H + row), v);
            }
            const size_t o = static_cast<size_t>(m) * A.H + row;
            if (A.residual != nullptr) v = __fadd_rn(A.residual[o], v);
            store_typed(A.y, A.ytype, o, v);
        }
    };
    if (NE == 0) {
        for (int t = blockIdx.x * kMxWarps + warp; t < T2; t += static_cast<int>(gridDim.x) * kMxWarps) add_up(t);
        return;
    }

    // ---- this warp's tickets: `next` is the one to issue, the claimed ones
    // wait in the lanes of `fifo` until their weights are consumed
    const uint64_t pol = l2_policy_evict_first();
    int next = misc[2] + warp;
    int fifo = 0;
    unsigned head = 0, tail = 0;
    int issued = 0, islot = 0, cslot = 0, consumed = 0;
    uint32_t cph = 0u;
    bool dead = false;
    // the ticket whose slices are being issued
    const uint8_t* isrc = nullptr;
    int ileft = 0;                        // lines left of it
    unsigned fetched = 0u;                // lane 0: the ticket after `next`
    if (lane == 0) fetched = atomicAdd(ticket, 1u);
    auto issue_one = [&]() {
        // claim tickets until one has slices (or none is left)
        while (ileft == 0) {
            if (next >= total || tail - head >= 32u) return;
            if (lane == static_cast<int>(tail & 31u)) fifo = next;
            ++tail;
            if (next < n1) {
                const int en = next / T1;
                isrc = A.w_gu + (static_cast<size_t>(ent_e[en]) * T1 + (next - en * T1)) * (static_cast<size_t>(C1) * kRows * mx_unit(FMT));
                ileft = C1;
            } else if (next >= n1 + nq) {
                const int k = next - n1 - nq;
                const int en = k / T2;
                isrc = A.w_dn + (static_cast<size_t>(ent_e[en]) * T2 + (k - en * T2)) * (static_cast<size_t>(C2) * kRows * mx_unit(FMT));
                ileft = C2;
            }
            next = static_cast<int>(__shfl_sync(0xffffffffu, fetched, 0));
            if (lane == 0 && next < total) fetched = atomicAdd(ticket, 1u);
        }
        const int n = min(ileft, kMxLines);
        if (lane == 0) {
            const uint32_t bar = bars + 8 * islot;
            const uint32_t bytes = static_cast<uint32_t>(n * kRows * mx_unit(FMT));
            if (issued >= S) fence_proxy_async_smem();
            mbar_arrive_expect_tx(bar, bytes);
            bulk_g2s(smem_u32(ring + islot * mx_slot(FMT)), isrc, bytes, bar, pol);
        }
        isrc += n * kRows * mx_unit(FMT);
        ileft -= n;
        ++issued;
        if (++islot == S) islot = 0;
    };
    for (int s = 0; s < S; ++s) issue_one();

    // bounded wait for a counter
    auto wait_count = [&](const unsigned* p, unsigned want) {
        bool ok = true;
        if (lane == 0) {
            if (ld_acquire_gpu(p) < want) {
                const uint64_t t0 = globaltimer_ns();
                while (ld_acquire_gpu(p) < want) {
                    __nanosleep(64);
                    if (globaltimer_ns() - t0 > kMxWaitNs) {
                        ok = false;
                        break;
                    }
                }
            }
        }
        ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0) != 0;
        if (!ok) {
            dead = true;
            if (lane == 0 && A.err != nullptr) atomicExch(A.err, kErrWaitTimeout);
        }
        return ok;
    };

    const int hb = lane & 1, pl = lane >> 1, pp = pl & 3;
    const int my_row = 4 * hb + pp;                     // this lane's row of a tile after the butterfly
    const int qd = lane >> 3;                           // and its share of the tokens: m % 4

    while (!dead) {
        if (head == tail) issue_one();
        if (head == tail) break;
        const int t = __shfl_sync(0xffffffffu, fifo, static_cast<int>(head & 31u));
        ++head;
        if (t >= n1 && t < n1 + nq) {
            // -------------------------------------- quantize a piece of h
            const int pos = (t - n1) / nseg, seg = (t - n1) - pos * nseg;
            const int en = of_pos[pos];
            const int p = list[pos];
            if (!wait_count(done1 + en, static_cast<unsigned>(T1))) break;
            __syncwarp();
            const A8Scale ks = a8_scale(__uint_as_float(__ldcg(hmax + p)));
            const float4* hp = reinterpret_cast<const float4*>(A.h + static_cast<size_t>(p) * A.I);
            uint32_t* qp = reinterpret_cast<uint32_t*>(A.qh + static_cast<size_t>(p) * A.I);
            float4 v[kMxSeg / 128];
#pragma unroll
            for (int i = 0; i < kMxSeg / 128; ++i) {
                const int w = seg * (kMxSeg / 4) + 32 * i + lane;
                v[i] = w < A.I / 4 ? __ldcg(hp + w) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            const uint64_t rr = f2_pack(ks.r, ks.r);
            int sum = 0;
#pragma unroll
            for (int i = 0; i < kMxSeg / 128; ++i) {
                const int w = seg * (kMxSeg / 4) + 32 * i + lane;
                if (w < A.I / 4) {
                    uint32_t ok = 0xffffffffu;
                    uint32_t q = a8_pack4_fast2(v[i], rr, ok);
                    if (a8_needs_exact(ks) || (ok >> 31) == 0u) q = a8_pack4_exact(v[i], ks);
                    qp[w] = q;
                    sum = __dp4a(static_cast<int>(q), 0x01010101, sum);
                }
            }
            if (FMT == FMT_W4) {
                sum = __reduce_add_sync(0xffffffffu, sum);
                if (lane == 0) atomicAdd(hsum + p, sum);
            }
            __syncwarp();
            if (lane == 0) red_add_release_gpu(doneq + en, 1u);
            continue;
        }
        // ------------------------------------------------ a tile of weights
        const bool down = t >= n1;
        const int k = down ? t - n1 - nq : t;
        const int TT = down ? T2 : T1;
        const int en = k / TT, tile = k - en * TT;
        const int e = ent_e[en], pos0 = ent_off[en], cnt = min(kMxTok, static_cast<int>(off_s[e] + cnt_s[e]) - pos0);
        const int C = down ? C2 : C1;
        const int KK = down ? A.I : A.H;
        const int8_t* codes = (down ? A.qh : A.qx) + pl * 32;
        // this lane's row parameters, and its tokens' places in the codes
        float sw = 0.0f, bv = 0.0f;
        if (down) {
            const int row = 8 * tile + my_row;
            if (row < A.H) {
                sw = __ldg(A.s_dn + static_cast<size_t>(e) * A.H + row);
                if (A.b_dn != nullptr) bv = __ldg(A.b_dn + static_cast<size_t>(e) * A.H + row);
            }
            if (ld_volatile_s8(ready_s + en) == 0) {
                if (!wait_count(doneq + en, static_cast<unsigned>(cnt * nseg))) break;
                __syncwarp();
                __threadfence_block();
                if (lane == 0) ready_s[en] = 1;
            }
            __threadfence_block();
        } else {
            const int row = glu_param_row(8 * tile + my_row, A.I);
            if (row >= 0) {
                sw = __ldg(A.s_gu + static_cast<size_t>(e) * 2 * A.I + row);
                if (A.b_gu != nullptr) bv = __ldg(A.b_gu + static_cast<size_t>(e) * 2 * A.I + row);
            }
        }
        uint32_t off[kMxTok];
#pragma unroll
        for (int m = 0; m < kMxTok; ++m) {
            const int p = list[pos0 + min(m, cnt - 1)];
            off[m] = static_cast<uint32_t>(down ? p : p / slots) * static_cast<uint32_t>(KK);
        }
        int acc[kMxTok][4], accA[4][4];
#pragma unroll
        for (int m = 0; m < kMxTok; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[m][j] = 0;
                accA[m & 3][j] = 0;
            }
        for (int c = 0; c < C; c += kMxLines) {
            const uint32_t bar = bars + 8 * cslot;
            bool ok = __all_sync(0xffffffffu, mbar_test_wait(bar, cph));
            if (!ok) ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, cph, kMxWaitNs));
            if (!ok) {
                dead = true;
                if (lane == 0 && A.err != nullptr) atomicExch(A.err, kErrWaitTimeout);
                break;
            }
            if (c + pl < C) {
                const uint8_t* slot = ring + cslot * mx_slot(FMT);
                const int8_t* cp = codes + c * 32;
                if (cnt == 1) slice_dot<FMT, 1>(slot, pl, hb, pp, cp, off, cnt, acc, accA);
                else if (cnt == 2) slice_dot<FMT, 2>(slot, pl, hb, pp, cp, off, cnt, acc, accA);
                else if (cnt <= 4) slice_dot<FMT, 4>(slot, pl, hb, pp, cp, off, cnt, acc, accA);
                else slice_dot<FMT, 8>(slot, pl, hb, pp, cp, off, cnt, acc, accA);
            }
            if (++cslot == S) {
                cslot = 0;
                cph ^= 1u;
            }
            ++consumed;
            __syncwarp();
            if (issued - consumed < S) issue_one();
        }
        if (dead) break;
        // lanes of equal (hb, pp) add up, then the read permutation is undone:
        // lane l keeps row my_row of every token (four copies, by lane / 8)
#pragma unroll
        for (int m = 0; m < kMxTok; ++m) {
            if (m < cnt) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (FMT == FMT_W4 && m < 4) acc[m][j] += accA[m][j] >> 4;
                    acc[m][j] += __shfl_xor_sync(0xffffffffu, acc[m][j], 8);
                    acc[m][j] += __shfl_xor_sync(0xffffffffu, acc[m][j], 16);
                }
                acc[m][0] += __shfl_xor_sync(0xffffffffu, acc[m][2], 4);
                acc[m][1] += __shfl_xor_sync(0xffffffffu, acc[m][3], 4);
                acc[m][0] += __shfl_xor_sync(0xffffffffu, acc[m][1], 2);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = 4 * i + qd;                   // this lane's token
            if (4 * i >= cnt) break;
            int a = acc[4 * i][0];
#pragma unroll
            for (int q = 1; q < 4; ++q)
                if (qd == q) a = acc[4 * i + q][0];
            const bool have = m < cnt;
            const int p = list[pos0 + min(m, cnt - 1)];
            if (down) {
                if (FMT == FMT_W4) a -= 8 * __ldcg(hsum + p);
                const float sx = a8_scale(__uint_as_float(__ldcg(hmax + p))).s;
                const int row = 8 * tile + my_row;
                if (have && row < A.H)
                    A.part[static_cast<size_t>(p) * A.H + row] = __fmaf_rn(__fmul_rn(sw, sx), __int2float_rn(a), bv);
            } else {
                const int tok = p / slots;
                if (FMT == FMT_W4) a -= 8 * xsum_s[tok];
                const float v = __fmaf_rn(__fmul_rn(sw, __ldg(A.sx + tok)), __int2float_rn(a), bv);
                const float u = __shfl_xor_sync(0xffffffffu, v, 1);      // gate lanes are even, up lanes odd
                const int j = 4 * tile + pp;
                const bool out = have && hb == 0 && j < A.I;
                const float hv = out ? xa_glu(A.glu, v, u) : 0.0f;
                if (out) A.h[static_cast<size_t>(p) * A.I + j] = hv;
                unsigned bits = __float_as_uint(fabsf(hv));
                bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 2));
                bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 4));
                if (have && (lane & 7) == 0) atomicMax(hmax + p, bits);
            }
        }
        __syncwarp();
        if (!down) {
            if (lane == 0) red_add_release_gpu(done1 + en, 1u);
        } else {
            unsigned old = 0;
            if (lane == 0) {
                asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(done2 + tile), "r"(1u) : "memory");
            }
            old = __shfl_sync(0xffffffffu, old, 0);
            if (old == static_cast<unsigned>(NE - 1)) {
                __syncwarp();
                add_up(tile);
            }
        }
    }
    // after a wait that ran out: the copies in flight land before the block ends
    if (dead)
        for (int k = consumed; k < issued; ++k)
            if (!mbar_wait_bounded(bars + 8 * (k % S), static_cast<uint32_t>(k / S) & 1u, kMxWaitNs)) break;
}

__global__ void zero_words_kernel(unsigned* p, int n)
{
    pdl_launch_dependents();
    pdl_wait();
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) p[i] = 0u;
}

template <int FMT>
cudaError_t launch_experts_t(const MoeArgs& a, int grid, size_t smem, bool pdl, cudaStream_t s)
{
    auto kern = moe_experts_kernel<FMT>;
    static SmemLimit limit;
    cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), limit, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kMxThreads);
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

size_t moe_experts_smem(int fmt, int stages) { return static_cast<size_t>(mx_smem(fmt, stages).total); }

cudaError_t launch_moe_experts(int fmt, const MoeArgs& a, int grid, size_t smem, bool pdl, cudaStream_t s)
{
    return fmt == FMT_W4 ? launch_experts_t<FMT_W4>(a, grid, smem, pdl, s) : launch_experts_t<FMT_W8F>(a, grid, smem, pdl, s);
}

cudaError_t launch_zero_words(unsigned* p, int n, bool pdl, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n < 256 * 16 ? (n + 255) / 256 : 16));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = pdl ? attr : nullptr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, zero_words_kernel, p, n);
}

}  // namespace w4k
