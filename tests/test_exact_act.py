"""The logistic function and the gated activations (exact_act.cuh), compiled for the host, over the whole fp32 range.

One rounding is half a step of the result.  In front of it a product of two pairs is off by at most 2^-45.5 of its value
(the product of the low parts, two roundings of 24 bits in them), so the exponential, the quotient and the two products add
up to 2^-41.5, and the tanh-GELU's argument t (four such products) to |t| 2^-43.5, which its exponential takes over.  In
steps (2^-24 of a value at least): 2^-17, and |t| 2^-19.5.  Subnormal results are rounded to 24 bits first: 2^-24 of the
value more.  The 64-bit values are off by |t| 2^-51 at most."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_decode_gb300", "csrc")
SOURCE = """
#include "exact_act.cuh"
extern "C" void glu(int kind, int n, const float* g, const float* u, float* y)
{
    for (int i = 0; i < n; ++i) y[i] = w4k::xa_glu(kind, g[i], u[i]);
}
extern "C" void logistic(int n, const float* v, float* y)
{
    for (int i = 0; i < n; ++i) y[i] = w4k::xa_logistic(v[i]);
}
"""
SILU, GELU = 1, 2
F32, F64 = np.float32, np.float64
FLT_MAX = float(np.finfo(F32).max)


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from bit_quantized_decode_gb300 import build
    d = tmp_path_factory.mktemp("exact_act")
    (d / "a.cpp").write_text(SOURCE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    cmd = [shutil.which("g++"), "-std=c++17", "-O2", "-ffp-contract=off", "-fno-fast-math", "-shared", "-fPIC", "-I", CSRC,
           "-I", cuda, str(d / "a.cpp"), "-o", str(d / "a.so")]
    subprocess.run(cmd, check=True)
    return ctypes.CDLL(str(d / "a.so"))


def _p(a):
    return a.ctypes.data_as(ctypes.c_void_p)


def _glu(lib, kind, g, u):
    g, u = np.ascontiguousarray(g, F32), np.ascontiguousarray(u, F32)
    y = np.empty_like(g)
    lib.glu(kind, g.size, _p(g), _p(u), _p(y))
    return y


def _logistic(lib, v):
    v = np.ascontiguousarray(v, F32)
    y = np.empty_like(v)
    lib.logistic(v.size, _p(v), _p(y))
    return y


def _argument(kind, g):
    g = g.astype(F64)
    return g if kind == SILU else 2.0 * np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3)


def _want(kind, g, u):
    with np.errstate(over="ignore"):
        return g.astype(F64) / (1.0 + np.exp(-_argument(kind, g))) * u.astype(F64)


def _check(y, want, extra):
    """y: fp32 results, want: 64 bits, extra: steps beyond the half."""
    size = np.maximum(np.abs(want), 2.0 ** -126)
    step = 2.0 ** (np.floor(np.log2(size)) - 23)
    tol = (0.5 + extra) * step + np.where(np.abs(want) < 2.0 ** -126, 2.0 ** -24 * np.abs(want), 0.0)
    edge = FLT_MAX + 2.0 ** 103                                     # from here on a value rounds to infinity
    over, y64 = np.abs(want) >= edge, y.astype(F64)
    sure = over & (np.abs(want) > edge * (1 + 2.0 ** -30))
    assert np.array_equal(y[sure], np.where(want[sure] > 0, np.inf, -np.inf).astype(F32))
    with np.errstate(invalid="ignore"):
        ok = over | (np.abs(y64 - want) <= tol)
    bad = ~ok
    assert not bad.any(), (int(bad.sum()), y[bad][:4], want[bad][:4])


def _values(n, seed, low, high):
    """Both signs, the exponent spread evenly over 2^low .. 2^high."""
    g = np.random.default_rng(seed)
    return (g.choice([-1.0, 1.0], n) * g.uniform(1.0, 2.0, n) * 2.0 ** g.uniform(low, high, n)).astype(F32)


@pytest.mark.parametrize("kind", [SILU, GELU])
@pytest.mark.parametrize("g_range,u_range", [((1, 2.2), (-10, 10))])
def test_gated_activations_round_once(lib, kind, g_range, u_range):
    n = 200000
    g, u = _values(n, 11, *g_range), _values(n, 12, *u_range)
    t = np.minimum(np.abs(_argument(kind, g)), 400.0)
    _check(_glu(lib, kind, g, u), _want(kind, g, u), 2.0 ** -17 + (t * 2.0 ** -19.5 if kind == GELU else 0.0))
