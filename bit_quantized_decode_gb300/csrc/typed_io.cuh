// Typed loads and stores of the operators that take fp32, fp16 or bf16
// activations, and the conversions of int8 codes to fp16.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "operators.h"
#include "quant_a8.cuh"

namespace w4k {

// One lane of a converged warp.  The tensor-core and bulk-copy instructions
// take uniform registers: under an elected lane the compiler issues them
// once, where under "lane == 0" it loops over the lanes that might be active
// (550 against some 60 cycles for the four to five of a GEMM stage).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void zero8(float (&v)[8])
{
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.0f;
}

// Eight consecutive values from element `at` (a multiple of eight; the base
// is 16-byte aligned) as fp32.
template <int T>
__device__ __forceinline__ void load8(const void* base, size_t at, float (&v)[8])
{
    if constexpr (T == T_F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
        const float4 a = __ldg(p), b = __ldg(p + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (T == T_F16) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                v[2 * k] = f.x;
                v[2 * k + 1] = f.y;
            } else {                                   // bf16: the upper half of an fp32
                v[2 * k] = __uint_as_float(w[k] << 16);
                v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
            }
        }
    }
}

// One value, rounded to the output type (to nearest even).
__device__ __forceinline__ void store_typed(void* y, int type, size_t at, float v)
{
    if (type == T_F32) static_cast<float*>(y)[at] = v;
    else if (type == T_F16) static_cast<__half*>(y)[at] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
}

// Eight INT8 codes of fp32 values, in order.
__device__ __forceinline__ uint2 quant8(const float (&t)[8], const A8Scale& ks)
{
    const float4 a = make_float4(t[0], t[1], t[2], t[3]), b = make_float4(t[4], t[5], t[6], t[7]);
    const uint64_t rr = f2_pack(ks.r, ks.r);
    uint32_t ok0 = 0xffffffffu, ok1 = 0xffffffffu;
    uint2 q = make_uint2(a8_pack4_fast2(a, rr, ok0), a8_pack4_fast2(b, rr, ok1));
    const bool all = a8_needs_exact(ks);
    if (all || (ok0 >> 31) == 0u) q.x = a8_pack4_exact(a, ks);
    if (all || (ok1 >> 31) == 0u) q.y = a8_pack4_exact(b, ks);
    return q;
}

// The experts kernel's workspace (MoeFill), by the whole grid.
__device__ __forceinline__ void moe_fill(const MoeFill& f)
{
    const unsigned head = kMxHead / 4, n = f.p != nullptr ? head + f.values : 0u;
    for (unsigned i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) {
        const unsigned v = i < head ? 0u : kMxNoValue;
        f.p[i] = make_uint4(v, v, v, v);
    }
}

// Four int8 -> four fp16, exactly: q + 128 as the low byte of the fp16 number
// 1024 + (q + 128), less 1152.
__device__ __forceinline__ void i8_to_f16(uint32_t c, uint32_t& h01, uint32_t& h23)
{
    const uint32_t u = c ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));   // 1152
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
    h01 = *reinterpret_cast<const uint32_t*>(&x);
    h23 = *reinterpret_cast<const uint32_t*>(&y);
}

__device__ __forceinline__ uint4 codes_f16(const uint2 q)
{
    uint4 h;
    i8_to_f16(q.x, h.x, h.y);
    i8_to_f16(q.y, h.z, h.w);
    return h;
}

}  // namespace w4k
