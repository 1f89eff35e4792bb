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
@pytest.mark.parametrize("g_range,u_range", [((1, 2.2), (-10, 10)), ((-20, 3), (-10, 10)), ((3, 7.5), (-10, 10)), ((4, 8), (90, 127)), ((-149, -20), (-149, 127)),
                                             ((40, 127), (-149, 127)), ((-149, 127), (-149, 127))])
def test_gated_activations_round_once(lib, kind, g_range, u_range):
    n = 200000
    g, u = _values(n, 11, *g_range), _values(n, 12, *u_range)
    t = np.minimum(np.abs(_argument(kind, g)), 400.0)
    _check(_glu(lib, kind, g, u), _want(kind, g, u), 2.0 ** -17 + (t * 2.0 ** -19.5 if kind == GELU else 0.0))


@pytest.mark.parametrize("kind,g,u", [(SILU, -88, 1), (SILU, -88, 1000), (SILU, -50, 1e37), (SILU, 1e20, 1e20), (SILU, -110, 1e38),
                                      (SILU, -180, 3e38), (SILU, 1e30, -1e30), (SILU, 2.0, 2.5e38), (SILU, 1e-30, 1e-10),
                                      (SILU, 1e-40, 1e20), (GELU, -10.2, 1000), (GELU, -10.2, 1), (GELU, 1e20, 1), (GELU, 1e20, 1e20),
                                      (GELU, -13, 3e38), (GELU, -1e20, 1e38), (GELU, 3e-39, 1e30), (GELU, 5.0, 3.4e38)])
def test_the_ends_of_the_range(lib, kind, g, u):
    g, u = np.array([g], F32), np.array([u], F32)
    t = np.minimum(np.abs(_argument(kind, g)), 400.0)
    _check(_glu(lib, kind, g, u), _want(kind, g, u), 2.0 ** -17 + t * 2.0 ** -19.5)


@pytest.mark.parametrize("kind", [SILU, GELU])
def test_zeros_infinities_and_nan(lib, kind):
    inf, nan = np.inf, np.nan
    rows = [(0.0, 5.0, 0.0), (-0.0, 5.0, -0.0), (3.0, 0.0, 0.0), (-3.0, 0.0, -0.0), (200.0, 1.0, 200.0), (-1000.0, 1.0, 0.0),
            (inf, 2.0, inf), (inf, -2.0, -inf), (1.0, inf, inf), (-1.0, inf, -inf), (1.0, -inf, -inf),
            (nan, 1.0, nan), (1.0, nan, nan), (inf, 0.0, nan), (0.0, inf, nan), (nan, 0.0, nan), (-inf, 1.0, nan)]
    y = _glu(lib, kind, [r[0] for r in rows], [r[1] for r in rows])
    assert np.array_equal(y, np.array([r[2] for r in rows], F32), equal_nan=True), y


def test_logistic_rounds_once_to_the_smallest_values(lib):
    v = np.concatenate([_values(400000, 3, -30, 7.5), np.linspace(-104, -86, 40001, dtype=F32), np.linspace(-88, 88, 200001, dtype=F32)])
    want = 1.0 / (1.0 + np.exp(-v.astype(F64)))
    _check(_logistic(lib, v), want, 2.0 ** -17)
    y = _logistic(lib, [np.inf, -np.inf, 0.0, np.nan, 1000.0, -1000.0])
    assert np.array_equal(y, np.array([1.0, 0.0, 0.5, np.nan, 1.0, 0.0], F32), equal_nan=True)


def test_far_logits_keep_their_order(lib):
    """Scores below 2^-126 are numbers like others: a larger logit has no smaller score, and those apart differ."""
    v = np.linspace(-103, -86, 2000, dtype=F32)
    y = _logistic(lib, v)
    assert (np.diff(y.astype(F64)) >= 0).all() and y[0] > 0
    assert _logistic(lib, [-88.0])[0] > _logistic(lib, [-90.0])[0] > _logistic(lib, [-100.0])[0] > 0
