// The logistic function and the gated activations to one fp32 rounding.
//
// The experts' hidden values are quantized again, and the router's sigmoid
// scores choose experts, so a value that differs in its last bit can change an
// integer code or a choice.  These functions therefore evaluate in pairs of
// fp32 (an unevaluated sum hi + lo) and round once.  The exponential, the
// quotient and the products are within 2^-41.5 of their values together, the
// tanh-GELU's argument t within |t| 2^-43.5, so two correct implementations
// agree but for values that close to a rounding boundary, and then by one step
// (2 million random values of each function against 64-bit mantissas: none
// differed).  Exponents are carried as integers up to the last operation: the
// products overflow and underflow where the result does.  A subnormal result
// is rounded twice, to 24 bits and to its step.
//
// exp(-t), t >= 0: table-driven reduction (P. T. P. Tang, "Table-driven
// implementation of the exponential function in IEEE floating-point
// arithmetic", ACM TOMS 15(2), 1989): t = N ln2 / 32 + r, |r| <= ln2 / 64,
// exp(-t) = 2^-(N / 32) 2^(-(N mod 32) / 32) exp(-r), the last by its Taylor
// series with the terms up to r^2 in pairs.  ln2 / 32 is a sum of three fp32,
// the first with nine bits so that N times it is exact.
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

// A pair m times 2^-n.
struct XaScaled {
    F2 m;
    int n;
};

// y 2^k, |y| below 8 (past fp32: infinity; subnormal: rounded once more).
__host__ __device__ inline float xa_scale(float y, int k)
{
    k = k < -252 ? -252 : k > 254 ? 254 : k;                         // 0, or infinity, at the ends
    const int k1 = k / 2;
    union {
        uint32_t u;
        float f;
    } a, b;
    a.u = static_cast<uint32_t>(127 + k1) << 23;
    b.u = static_cast<uint32_t>(127 + k - k1) << 23;
    return xa_mul(xa_mul(y, a.f), b.f);
}

// |v| in [1, 2) with v's sign, and its exponent; v is neither 0 nor infinite.
__host__ __device__ inline float xa_split(float v, int& e)
{
    union {
        uint32_t u;
        float f;
    } a;
    a.f = v;
    e = -127;
    if ((a.u & 0x7f800000u) == 0u) {
        a.f = xa_mul(v, 0x1p+64f);
        e -= 64;
    }
    e += static_cast<int>((a.u >> 23) & 0xffu);
    a.u = (a.u & 0x807fffffu) | 0x3f800000u;
    return a.f;
}

// exp(-t), t >= 0; 0 from t = 400 on, where no product of fp32 numbers with it reaches 2^-149.
__host__ __device__ inline XaScaled xa_exp_neg(F2 t)
{
    if (!(t.h < 400.0f)) return XaScaled{F2{t.h == t.h ? 0.0f : t.h, 0.0f}, 0};        // (NaN stays)
    const float N = std::rint(xa_mul(t.h, 0x1.715476p+5f));          // below 2^15
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
    return XaScaled{xa_prod(F2{T[0], T[1]}, xa_fast(one.h, xa_add(one.l, lo))), n >> 5};
}

// 1 / (1 + exp(-t)).
__host__ __device__ inline XaScaled xa_sigmoid(F2 t)
{
    const bool neg = t.h < 0.0f;
    const XaScaled e = xa_exp_neg(neg ? F2{-t.h, -t.l} : t);
    // the exponential beside 1: nothing below 2^-64
    union {
        uint32_t u;
        float f;
    } scale;
    scale.u = e.n < 64 ? static_cast<uint32_t>(127 - e.n) << 23 : 0u;
    const F2 s = xa_fast(1.0f, xa_mul(e.m.h, scale.f));
    const F2 den = xa_fast(s.h, xa_fma(e.m.l, scale.f, s.l));
    const F2 num = neg ? e.m : F2{1.0f, 0.0f};
    const float q = xa_div(num.h, den.h);
    const float r = xa_add(xa_fma(-q, den.h, num.h), xa_fma(-q, den.l, num.l));
    return XaScaled{xa_fast(q, xa_div(r, den.h)), neg ? e.n : 0};
}

// The gated activation act(g) u, rounded once.
__host__ __device__ inline float xa_glu(int kind, float g, float u)
{
    const float big = 0x1.fffffep+127f;
    if (!(fabsf(g) <= big) || !(fabsf(u) <= big) || g == 0.0f || u == 0.0f)
        return g < -big ? xa_add(g, -g) : xa_mul(g, u);              // (-infinity times 0: NaN)
    F2 t = F2{g, 0.0f};
    if (kind == GLU_GELU_TANH) {
        // g / 2 (1 + tanh z) = g / (1 + exp(-2 z)), 2 z = 2 sqrt(2 / pi) (g + 0.044715 g^3)
        const F2 k = xa_prod(F2{0x1.6e4e26p-5f, 0x1.a9003ep-30f}, xa_prod(g, g));
        const F2 s = xa_sum(1.0f, k.h);
        t = xa_prod(xa_prod(F2{0x1.988454p+0f, -0x1.857936p-25f}, F2{g, 0.0f}), xa_fast(s.h, xa_add(s.l, k.l)));
        if (fabsf(g) > 64.0f) t = F2{g < 0.0f ? -1000.0f : 1000.0f, 0.0f};            // past the exponential's range
    }
    // the exponents apart: the product of the three may be in range where that of two is not
    int eg, eu;
    const float gm = xa_split(g, eg), um = xa_split(u, eu);
    const XaScaled s = xa_sigmoid(t);
    const F2 y = xa_prod(xa_prod(gm, um), s.m);
    return xa_scale(xa_add(y.h, y.l), eg + eu - s.n);
}

// The logistic function, rounded once.
__host__ __device__ inline float xa_logistic(float v)
{
    const XaScaled s = xa_sigmoid(F2{v, 0.0f});
    return xa_scale(xa_add(s.m.h, s.m.l), -s.n);
}

}  // namespace w4k
