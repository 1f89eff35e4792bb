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

// Prefix sums of the sequences' units into pre[0 .. B], by the whole block; pre needs kAtMaxSeq + 1 places.
template <int NT>
__device__ __forceinline__ void seq_prefix(const AttnArgs& A, int rows, int unit, long long* pre, long long* warp_s)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kW = NT / 32;
    long long carry = 0;
    for (int base = 0; base < A.b.B; base += NT) {
        const int b = base + tid;
        long long v = 0;
        if (b < A.b.B) {
            const SeqFacts f = seq_facts(A, b);
            v = static_cast<long long>(A.c.Hkv) * seq_tiles(A, f, rows) * seq_units(f, unit);
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long w = __shfl_up_sync(0xffffffffu, v, off);
            if (lane >= off) v += w;
        }
        if (lane == 31) warp_s[warp] = v;
        __syncthreads();
        long long before = carry, all = 0;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            if (w < warp) before += warp_s[w];
            all += warp_s[w];
        }
        if (b < A.b.B) pre[b + 1] = before + v;
        carry += all;
        __syncthreads();
    }
    if (tid == 0) pre[0] = 0;
    __syncthreads();
}

// One (sequence, key head, tile of rows): its units are [u0, u0 + units) of the call's.
struct Segment {
    long long u0;
    int units;
    int b, h, tile;
    SeqFacts f;
};
__device__ __forceinline__ Segment find_segment(const AttnArgs& A, const long long* pre, long long u, int rows, int unit)
{
    int lo = 0, hi = A.b.B;                     // pre[lo] <= u < pre[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (pre[m] <= u) lo = m;
        else hi = m;
    }
    Segment s;
    s.b = lo;
    s.f = seq_facts(A, lo);
    s.units = seq_units(s.f, unit);
    const int tiles = seq_tiles(A, s.f, rows);
    const long long seg = (u - pre[lo]) / s.units;
    s.h = static_cast<int>(seg / tiles);
    s.tile = static_cast<int>(seg - static_cast<long long>(s.h) * tiles);
    s.u0 = pre[lo] + seg * s.units;
    return s;
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

constexpr uint64_t kAtWaitNs = 250ull * 1000ull * 1000ull;
__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

}  // namespace w4k
