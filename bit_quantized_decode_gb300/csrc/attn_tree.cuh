// What the attention kernels share: how a call's work is laid out over the
// grid, tensor-map copies, conversions of fragments.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attention.h"
#include "ptx.cuh"
#include "typed_io.cuh"

namespace w4k {

// Rows and cached places of sequence b that a call may touch, whatever the
// arrays hold: rows within [0, T), places within the page table.
struct SeqFacts {
    int q0, n;                // first row, rows
    int ctx, len;             // places before the drafts, and with them
};
__device__ __forceinline__ SeqFacts seq_facts(const AttnArgs& A, int b)
{
    SeqFacts f;
    const int cap = A.b.max_pages << A.c.lg;                  // at most 2^30 (the host's check)
    f.q0 = __ldg(A.b.q_start + b);
    f.n = __ldg(A.b.q_start + b + 1) - f.q0;
    if (f.q0 < 0 || f.q0 >= A.T) f.n = 0;
    f.n = max(0, min(min(f.n, A.b.max_tokens), A.T - f.q0));
    f.ctx = min(max(__ldg(A.b.ctx + b), 0), cap);
    f.len = min(f.ctx + f.n, cap);
    return f;
}
// Units of work of one (head, row tile), and such pairs, of a sequence.
__device__ __forceinline__ int seq_units(const SeqFacts& f, int unit) { return f.n > 0 ? (f.len + unit - 1) / unit : 0; }
__device__ __forceinline__ int seq_tiles(const AttnArgs& A, const SeqFacts& f, int rows) { return (f.n * A.G + rows - 1) / rows; }

// One (sequence, key head, tile of rows): its units are [u0, u0 + units) of the call's.
struct Segment {
    int u0;
    int units;
    int b, h, tile;
    SeqFacts f;
};

// How a call's units lie (fewer than 2^31 - 1024: the host's check): sequences one behind the other, in each its key heads,
// in each its tiles of rows.  Up to 32 sequences every warp holds them itself, one to a lane (one round of loads, no
// barrier); more lie as prefix sums in shared memory.  All calls are a whole warp's.
//
// Blocks take equal shares of the units, across segments.  A block that ends one segment and begins another pays twice
// for queries and joining (4.5 us of 10.7 for one token over 1000 places, since then 3).  So segments get blocks of their own
// instead, n for every segment of a sequence in near equal parts, where that makes no block's share longer by more than
// those 3 us.
struct Layout {
    const int* pre;           // [B + 1] in shared memory; null: in the lanes
    int mine;            // units before this lane's sequence
    SeqFacts f;               // this lane's sequence
    int total;
    int share;                // units of a block; 0: segments have blocks of their own
    int n, mine_b, blocks;    // those of each of this lane's segments, those before its sequence, of all
};
__device__ __forceinline__ int seq_cost(const AttnArgs& A, const SeqFacts& f, int rows, int unit)
{
    return A.c.Hkv * seq_tiles(A, f, rows) * seq_units(f, unit);
}
__device__ __forceinline__ int warp_scan(int v, int lane)
{
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += w;
    }
    return v;
}
__device__ __forceinline__ Layout lane_layout(const AttnArgs& A, int rows, int unit, int lane)
{
    Layout L;
    L.pre = nullptr;
    int v = 0, units = 0, segs = 0;
    L.f = SeqFacts{0, 0, 0, 0};
    if (lane < A.b.B) {
        L.f = seq_facts(A, lane);
        units = seq_units(L.f, unit);
        segs = A.c.Hkv * seq_tiles(A, L.f, rows);
        v = segs * units;
    }
    const int upto = warp_scan(v, lane);
    L.mine = upto - v;
    L.total = __shfl_sync(0xffffffffu, upto, 31);
    L.n = L.mine_b = L.blocks = 0;
    L.share = max((L.total + A.blocks - 1) / A.blocks, A.least);
    // the fewest units to a block with which all segments' parts find one, if that is not much more than an equal share
    auto fits = [&](int part) { return __reduce_add_sync(0xffffffffu, segs * ((units + part - 1) / part)) <= A.blocks; };
    if (__reduce_max_sync(0xffffffffu, segs) > A.blocks) return L;
    int hi = L.share;
    if (!fits(hi)) {                            // (each look costs some 0.1 us, so an even split comes first)
        hi += A.extra;
        if (!fits(hi)) return L;
        int lo = L.share + 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (fits(mid)) hi = mid;
            else lo = mid + 1;
        }
    }
    L.share = 0;
    L.n = (units + hi - 1) / hi;
    const int b = warp_scan(segs * L.n, lane);
    L.mine_b = b - segs * L.n;
    L.blocks = __shfl_sync(0xffffffffu, b, 31);
    return L;
}
// By the whole block of NT threads; pre needs kAtMaxSeq + 1 places, warp_s one for each warp.
template <int NT>
__device__ __forceinline__ Layout block_layout(const AttnArgs& A, int rows, int unit, int* pre, int* warp_s)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (A.b.B <= 32) return lane_layout(A, rows, unit, lane);
    int carry = 0;
    for (int base = 0; base < A.b.B; base += NT) {
        const int b = base + tid;
        const int v = warp_scan(b < A.b.B ? seq_cost(A, seq_facts(A, b), rows, unit) : 0, lane);
        if (lane == 31) warp_s[warp] = v;
        __syncthreads();
        int before = carry;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            if (w < warp) before += warp_s[w];
            carry += warp_s[w];
        }
        if (b < A.b.B) pre[b + 1] = before + v;
        __syncthreads();
    }
    if (tid == 0) pre[0] = 0;
    __syncthreads();
    Layout L;
    L.pre = pre;
    L.mine = 0;
    L.f = SeqFacts{0, 0, 0, 0};
    L.total = pre[A.b.B];
    L.share = max((L.total + A.blocks - 1) / A.blocks, A.least);
    L.n = L.mine_b = L.blocks = 0;
    return L;
}
__device__ __forceinline__ SeqFacts facts_of(const Layout& L, int b)
{
    SeqFacts f;
    f.q0 = __shfl_sync(0xffffffffu, L.f.q0, b);
    f.n = __shfl_sync(0xffffffffu, L.f.n, b);
    f.ctx = __shfl_sync(0xffffffffu, L.f.ctx, b);
    f.len = __shfl_sync(0xffffffffu, L.f.len, b);
    return f;
}
__device__ __forceinline__ Segment find_segment(const AttnArgs& A, const Layout& L, int u, int rows, int unit)
{
    Segment s;
    int first;
    if (L.pre == nullptr) {                     // the last sequence that begins at u or before
        const int lane = threadIdx.x & 31;
        s.b = __popc(__ballot_sync(0xffffffffu, lane < A.b.B && L.mine <= u)) - 1;
        s.f = facts_of(L, s.b);
        first = __shfl_sync(0xffffffffu, L.mine, s.b);
    } else {
        int lo = 0, hi = A.b.B;                 // pre[lo] <= u < pre[hi]
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (L.pre[m] <= u) lo = m;
            else hi = m;
        }
        s.b = lo;
        s.f = seq_facts(A, lo);
        first = L.pre[lo];
    }
    s.units = seq_units(s.f, unit);
    const int tiles = seq_tiles(A, s.f, rows);
    const int seg = (u - first) / s.units;
    s.h = seg / tiles;
    s.tile = seg - s.h * tiles;
    s.u0 = first + seg * s.units;
    return s;
}
// A block's piece of a segment that has blocks of its own: number j of n.
struct OwnPiece {
    int j, n, us, ue;
};
__device__ __forceinline__ OwnPiece own_piece(const Layout& L, const AttnArgs& A, int block, int unit)
{
    OwnPiece p = {0, 0, 0, 0};
    if (block >= L.blocks) return p;
    const int lane = threadIdx.x & 31;
    const int b = __popc(__ballot_sync(0xffffffffu, lane < A.b.B && L.mine_b <= block)) - 1;
    const SeqFacts f = facts_of(L, b);
    p.n = __shfl_sync(0xffffffffu, L.n, b);
    const int at = block - __shfl_sync(0xffffffffu, L.mine_b, b), units = seq_units(f, unit), seg = at / p.n;
    p.j = at - seg * p.n;
    const int u0 = __shfl_sync(0xffffffffu, L.mine, b) + seg * units;
    p.us = u0 + static_cast<int>(static_cast<long long>(units) * p.j / p.n);
    p.ue = u0 + static_cast<int>(static_cast<long long>(units) * (p.j + 1) / p.n);
    return p;
}
// The units [x, y) of a block.
__device__ __forceinline__ int2 block_units(const Layout& L, const AttnArgs& A, int block, int unit)
{
    if (L.share == 0) {
        const OwnPiece p = own_piece(L, A, block, unit);
        return make_int2(p.us, p.ue);
    }
    const int us = static_cast<int>(min(static_cast<long long>(block) * L.share, static_cast<long long>(L.total)));
    return make_int2(us, us + min(L.share, L.total - us));
}

// Of the host: blocks of a launch; units of one segment that a block takes at most, by the table's width (equal shares, or
// `extra` more where segments have blocks of their own).
inline int blocks_of(int sms) { return sms < kAtMaxBlocks ? sms : kAtMaxBlocks; }
inline long long piece_units(const AttnArgs& a, int blocks, int unit, int extra)
{
    const long long segment = (static_cast<long long>(a.b.max_pages) * a.c.page + unit - 1) / unit, share = a.units / blocks + 1 + extra;
    return segment < share ? segment : share;
}

// Box of a 3-D tensor map -> shared memory.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// Bulk copy without a cache hint.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// 2^x (within 2 ulp; results below 2^-126 are 0).
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Four int8 -> four bf16, exactly: the low seven bits on 128.0 (whose last place is 1), less 128 or, for a negative code,
// 256.
__device__ __forceinline__ void i8_to_bf16(uint32_t c, uint32_t& h01, uint32_t& h23)
{
    const uint32_t m = c & 0x7f7f7f7fu, n = c & 0x80808080u;
    const uint32_t a = __byte_perm(m, 0x43434343u, 0x4140), b = __byte_perm(m, 0x43434343u, 0x4342);
    const uint32_t s = __byte_perm(n, 0x43434343u, 0x4140), t = __byte_perm(n, 0x43434343u, 0x4342);
    const __nv_bfloat162 x = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&s));
    const __nv_bfloat162 y = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b), *reinterpret_cast<const __nv_bfloat162*>(&t));
    h01 = *reinterpret_cast<const uint32_t*>(&x);
    h23 = *reinterpret_cast<const uint32_t*>(&y);
}

// Probabilities in fp16 are made so much larger that the largest is near 2^15, and so are their sums (the quotient is the
// same): fp16's least step is 2^-24, and a long context's many small probabilities would vanish beside a large one while their
// sum counts them.  log2 of that factor, where a probability reaches 2^raise.
__host__ __device__ constexpr float prob_lift(int type, float raise) { return type == T_F16 ? 15.0f - raise : 0.0f; }

// Two fp32 as a pair of 16-bit numbers (the first in the low half), to nearest or towards zero, and back.
template <int T>
__device__ __forceinline__ uint32_t pair16(float a, float b)
{
    if constexpr (T == T_F16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <int T>
__device__ __forceinline__ uint32_t pair16_cut(float a, float b)
{
    uint32_t r;
    if constexpr (T == T_F16) asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
template <int T>
__device__ __forceinline__ float2 unpair16(uint32_t u)
{
    if constexpr (T == T_F16) return __half22float2(*reinterpret_cast<const __half2*>(&u));
    else return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// One 16-bit part of two probabilities, which become what is left of them; the last part is rounded.
//
// A value that a row sees may be infinite, and then every part times it has to be that infinity: a part that is 0 or of the
// other sign would make it a NaN.  So parts are cut towards zero and what is left counts a step of the last part more than it
// is (2^-23 of the probability, fp16 2^-21; against what the tensor cores cut from the sums: with the sum of the probabilities
// made as much larger, errors of 0.6e-6 to 3.8e-6 become 0.9e-6 to 3.9e-6): it has the probability's sign and is not 0 (down to
// 2^-87; fp16, whose least step is 2^-24, to 2^-13 of the largest and on the mma.sync kernel 2^-19).  An INT8 cache's codes are finite: its parts are
// rounded, and where a value's scale, which the probability has taken in, makes that infinite, the first part has it all
// (only_first).
template <int T, bool kCodes>
__device__ __forceinline__ uint32_t part16(float& x, float& y, bool last)
{
    if (kCodes || last) {
        const uint32_t w = pair16<T>(x, y);
        const float2 r = unpair16<T>(w);
        x -= r.x;
        y -= r.y;
        return w;
    }
    constexpr float more = T == T_F16 ? 1.0f + 1.0f / (1 << 21) : 1.0f + 1.0f / (1 << 23);
    const uint32_t w = pair16_cut<T>(x, y);
    const float2 r = unpair16<T>(w);
    x = __fmaf_rn(x, more, -r.x);
    y = __fmaf_rn(y, more, -r.y);
    return w;
}
// Scales from which a probability's product with them may pass fp32: one in a tile is looked for, not one in each product.
__device__ __forceinline__ bool vast(float scale) { return fabsf(scale) >= 1.2676506e30f; }      // 2^100
__device__ __forceinline__ uint32_t only_first(uint32_t w, bool first, bool second)
{
    return (first ? 0u : w & 0xffffu) | (second ? 0u : w & 0xffff0000u);
}

constexpr uint64_t kAtWaitNs = 250ull * 1000ull * 1000ull;
__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

}  // namespace w4k
