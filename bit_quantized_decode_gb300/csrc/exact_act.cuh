// The logistic function and the gated activations to one fp32 rounding.
//
// The experts' hidden values are quantized again, and the router's sigmoid
// scores choose experts, so a value that differs in its last bit can change an
// integer code or a choice.  These functions therefore evaluate in pairs of
// fp32 (an unevaluated sum hi + lo, about 2^-42 of the value) and round once:
// two correct implementations agree but for values within that distance of a
// rounding boundary (about one in 2^17), and then by one step.
//
// exp(-t), t >= 0: table-driven reduction (P. T. P. Tang, "Table-driven
// implementation of the exponential function in IEEE floating-point
// arithmetic", ACM TOMS 15(2), 1989): t = N ln2 / 32 + r, |r| <= ln2 / 64,
// exp(-t) = 2^-(N / 32) 2^(-(N mod 32) / 32) exp(-r), the last by its Taylor
// series with the terms up to r^2 in pairs.  ln2 / 32 is a sum of three fp32,
// the first with nine bits so that N times it is exact.  Results that are
// subnormal in fp32 may flush to zero.
#pragma once
#include <cmath>
#include <cstdint>

#include "internal.h"

namespace w4k {

struct F2 {
    float h, l;
};

#ifdef __CUDA_ARCH__
__device__ __forceinline__ float xa_fma(float a, float b, float c) { return __fmaf_rn(a, b, c); }
__device__ __forceinline__ float xa_mul(float a, float b) { return __fmul_rn(a, b); }
__device__ __forceinline__ float xa_add(float a, float b) { return __fadd_rn(a, b); }
__device__ __forceinline__ float xa_div(float a, float b) { return __fdiv_rn(a, b); }
#define XA_TABLE __device__ const
#else
inline float xa_fma(float a, float b, float c) { return std::fmaf(a, b, c); }
inline float xa_mul(float a, float b) { return a * b; }
inline float xa_add(float a, float b) { return a + b; }
inline float xa_div(float a, float b) { return a / b; }
#define XA_TABLE static const
#endif

// 2^(-j / 32) as hi + lo.
XA_TABLE float kXaPow[32][2] = {
    {1.0f, 0.0f}, {0.978572071f, -8.51090221e-09f}, {0.957603276f, 4.92266405e-09f}, {0.93708384f, -2.33150281e-08f},
    {0.917004049f, -5.61963898e-09f}, {0.897354543f, -5.70752245e-09f}, {0.878126085f, -4.61788519e-09f}, {0.859309673f, -2.4248088e-08f},
    {0.840896428f, -1.23776633e-08f}, {0.822877765f, -2.56248605e-08f}, {0.805245161f, 4.91810859e-09f}, {0.787990451f, -2.83051271e-08f},
    {0.771105409f, 4.03545242e-09f}, {0.754582226f, -1.24796866e-08f}, {0.738413095f, -2.25044943e-08f}, {0.722590387f, 1.66209997e-08f},
    {0.707106769f, 1.21016175e-08f}, {0.69195497f, -2.93778868e-08f}, {0.677127779f, -5.06167463e-09f}, {0.662618339f, -1.74818666e-08f},
    {0.648419797f, -2.00949977e-08f}, {0.634525478f, 7.09666659e-10f}, {0.620928884f, 2.24841905e-08f}, {0.607623696f, -1.63369744e-08f},
    {0.594603539f, 1.89881764e-08f}, {0.58186245f, -2.02572075e-08f}, {0.56939429f, 2.69311116e-08f}, {0.557193398f, -2.71777001e-08f},
    {0.545253873f, -6.53876997e-09f}, {0.53357023f, -2.96687599e-08f}, {0.522136867f, 2.41673508e-08f}, {0.510948598f, -2.40577993e-08f}};

// a + b exactly (Knuth), and with |a| >= |b| (Dekker).
__host__ __device__ inline F2 xa_sum(float a, float b)
{
    const float s = xa_add(a, b);
    const float bp = xa_add(s, -a);
    return F2{s, xa_add(xa_add(a, -xa_add(s, -bp)), xa_add(b, -bp))};
}
__host__ __device__ inline F2 xa_fast(float a, float b)
{
    const float s = xa_add(a, b);
    return F2{s, xa_add(b, -xa_add(s, -a))};
}
__host__ __device__ inline F2 xa_prod(float a, float b)
{
    const float p = xa_mul(a, b);
    return F2{p, xa_fma(a, b, -p)};
}
__host__ __device__ inline F2 xa_prod(F2 a, F2 b)
{
    const F2 p = xa_prod(a.h, b.h);
    return xa_fast(p.h, xa_fma(a.h, b.l, xa_fma(a.l, b.h, p.l)));
}

// exp(-t), t >= 0.
__host__ __device__ inline F2 xa_exp_neg(F2 t)
{
    if (!(t.h < 87.0f)) return F2{t.h == t.h ? 0.0f : t.h, 0.0f};        // (NaN stays)
    const float N = std::rint(xa_mul(t.h, 0x1.715476p+5f));
    const float d = xa_fma(-N, 0x1.63p-6f, t.h);                     // exact
    const F2 p = xa_prod(N, -0x1.bd0106p-18f);
    const F2 s = xa_sum(d, -p.h);
    const F2 r = xa_sum(s.h, xa_add(xa_add(s.l, -p.l), t.l));        // (t.l may pass s.h; the series wants a small low part)
    const float qh = -r.h;
    const float ql = -xa_fma(-N, 0x1.cf79acp-45f, r.l);
    const F2 q2 = xa_prod(qh, qh);
    const float q3 = xa_mul(xa_mul(q2.h, qh), xa_fma(qh, xa_fma(qh, 0x1.111112p-7f, 0x1.555556p-5f), 0x1.555556p-3f));
    const F2 a = xa_fast(qh, xa_mul(0.5f, q2.h));
    const float lo = xa_add(xa_add(a.l, ql), xa_add(xa_fma(qh, ql, xa_mul(0.5f, q2.l)), q3));
    const F2 one = xa_fast(1.0f, a.h);
    const int n = static_cast<int>(N);
    const float* T = kXaPow[n & 31];
    const F2 e = xa_prod(F2{T[0], T[1]}, xa_fast(one.h, xa_add(one.l, lo)));
    union {
        uint32_t u;
        float f;
    } scale;
    scale.u = static_cast<uint32_t>(127 - (n >> 5)) << 23;           // n >> 5 <= 125
    return F2{xa_mul(e.h, scale.f), xa_mul(e.l, scale.f)};
}

// 1 / (1 + exp(-t)).
__host__ __device__ inline F2 xa_sigmoid(F2 t)
{
    const bool neg = t.h < 0.0f;
    const F2 e = xa_exp_neg(neg ? F2{-t.h, -t.l} : t);
    const F2 s = xa_fast(1.0f, e.h);
    const F2 den = xa_fast(s.h, xa_add(s.l, e.l));
    const F2 num = neg ? e : F2{1.0f, 0.0f};
    const float q = xa_div(num.h, den.h);
    const float r = xa_add(xa_fma(-q, den.h, num.h), xa_fma(-q, den.l, num.l));
    return xa_fast(q, xa_div(r, den.h));
}

// The gated activation act(g) u, rounded once.
__host__ __device__ inline float xa_glu(int kind, float g, float u)
{
    F2 t = F2{g, 0.0f};
    if (kind == GLU_GELU_TANH) {
        // g / 2 (1 + tanh z) = g / (1 + exp(-2 z)), 2 z = 2 sqrt(2 / pi) (g + 0.044715 g^3)
        const F2 k = xa_prod(F2{0x1.6e4e26p-5f, 0x1.a9003ep-30f}, xa_prod(g, g));
        const F2 s = xa_sum(1.0f, k.h);
        t = xa_prod(xa_prod(F2{0x1.988454p+0f, -0x1.857936p-25f}, F2{g, 0.0f}), xa_fast(s.h, xa_add(s.l, k.l)));
        if (!(fabsf(t.h) < 3.0e38f)) t = F2{g < 0.0f ? -100.0f : 100.0f, 0.0f};   // g^3 past fp32
    }
    const F2 y = xa_prod(xa_prod(g, u), xa_sigmoid(t));
    return xa_add(y.h, y.l);
}

// The logistic function, rounded once.
__host__ __device__ inline float xa_logistic(float v)
{
    const F2 s = xa_sigmoid(F2{v, 0.0f});
    return xa_add(s.h, s.l);
}

}  // namespace w4k
