"""The INT8 linear where its product runs on pairs of blocks (more than one round of 128 x 128 tiles, past 128 tokens): the
quantizer's codes in half tiles, norm, residual and the residual updated in place, and long runs.  Shapes named "pairs" give
pairs on 152 SMs; the others are the single blocks' in-place updates.  Tolerances: test_gpu_w8a8."""
import numpy as np
import pytest

import ops_reference as ref
from bit_quantized_decode_gb300 import workloads as wl
from helpers import cuda_ok, dev, host
from test_gpu_w8a8 import _check, _dtype, _repacked, _workspace

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

PAIRS = [(1000, 2560, 1536), (1100, 2500, 96), (2000, 4608, 544), (300, 20000, 800), (1030, 3001, 1376), (129, 20000, 96)]


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_decode_gb300 import _lib
    _lib.load()
    _lib.clear_device_error()
    yield _lib
    assert _lib.device_error() == 0


def _case(M, N, K, xt, norm):
    g = wl.rng(M + 3 * N + K + norm)
    x = dev(wl.residual_stream(g, M, K)).to(_dtype(xt))
    x[M // 2] = 0.0                                               # an all-zero token: scale 0, y = b
    gamma, b = wl.norm_weight(g, K), wl.bias(g, N)
    w, sw = wl.int_codes(g, (N, K), -127, 127), wl.positive_scales(g, N, 1e-4, 1e-3)
    xf = host(x.float())
    q, s = ref.codes(ref.rmsnorm(xf, gamma, 1e-6) if norm else xf)
    return x, gamma, b, w, sw, q, s, wl.residual_stream(g, M, N)


@pytest.mark.parametrize("xt,yt,norm", [("float32", "float32", True), ("bfloat16", "bfloat16", False), ("float16", "float16", True)])
@pytest.mark.parametrize("M,N,K", PAIRS)
def test_pairs_match_64_bits(lib, M, N, K, xt, yt, norm):
    import torch
    x, gamma, b, w, sw, q, s, _ = _case(M, N, K, xt, norm)
    y = torch.full((M * N + 257,), 3.25, dtype=_dtype(yt), device="cuda")
    qx, sx = torch.empty((M, K), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    lib.w8a8_linear(_repacked(lib, w), dev(sw), dev(b), x, y[:M * N].view(M, N), qx, sx, _workspace(lib, M, N, K),
                    dev(gamma) if norm else None, 1e-6)
    assert np.array_equal(host(sx).astype(np.float64), s) and np.array_equal(host(qx).astype(np.float64), q)
    assert (y[M * N:] == 3.25).all()                              # nothing behind the last token
    want, _ = ref.linear(q, s, w, sw, b)
    prod, _ = ref.linear(q, s, w, sw)
    _check(y[:M * N].view(M, N), want, np.abs(prod), yt)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("M,N,K", PAIRS[:4] + [(16, 130, 1536), (40, 392, 1120), (70, 264, 96), (128, 257, 2048), (9, 20000, 96),
                                               (100, 3584, 512), (200, 520, 1536)])
def test_residual_in_place(lib, M, N, K, norm):
    """y = residual + ..., the residual another tensor or y itself, with dependent launches behind what wrote x and y."""
    import torch
    x, gamma, b, w, sw, q, s, res = _case(M, N, K, "float32", norm)
    wd, sd, bd, gd, ws, sx = _repacked(lib, w), dev(sw), dev(b), dev(gamma), _workspace(lib, M, N, K), torch.empty(M, device="cuda")
    y, r = torch.full((M, N), float("nan"), device="cuda"), dev(res)
    lib.w8a8_linear(wd, sd, bd, x, y, None, sx, ws, gd if norm else None, 1e-6, r)
    want, _ = ref.linear(q, s, w, sw, b)
    prod, _ = ref.linear(q, s, w, sw)
    _check(y, want + res, np.abs(prod), "float32", np.abs(want))
    z, x2 = r.clone(), torch.empty_like(x)
    for _ in range(3):
        z.copy_(r)
        x2.copy_(x)
        lib.w8a8_linear(wd, sd, bd, x2, z, None, sx, ws, gd if norm else None, 1e-6, z, flags=lib.W4_FLAG_PDL)
        assert torch.equal(z, y)


@pytest.mark.parametrize("M,N,K,calls", [(300, 20000, 800, 4000), (2000, 4608, 544, 3000), (1100, 2500, 96, 6000), (1030, 3001, 1376, 3000)])
def test_long_runs_on_pairs_repeat_every_bit(lib, M, N, K, calls):
    """Thousands of calls, each compared: odd numbers of stages, one to three rounds of tiles, ragged rows and tokens, dependent
    launches back to back."""
    import torch
    from bit_quantized_decode_gb300 import QuantLinear
    g = torch.Generator(device="cuda").manual_seed(3)
    lin = QuantLinear.from_float("w8", [torch.randn(N, K, device="cuda", generator=g)])
    x = torch.randn(M, K, device="cuda", generator=g)
    want = torch.cat([lin(x[m:m + 4].contiguous()) for m in range(0, M, 4)])
    ws, sx = lin.workspace(M), torch.empty(M, device="cuda")
    ys = [torch.empty((M, N), device="cuda") for _ in range(8)]
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(calls // len(ys)):
        for y in ys:
            lin(x, y, None, sx, workspace=ws, flags=lib.W4_FLAG_PDL)
        for y in ys:
            wrong += (y != want).any()
    assert int(wrong) == 0 and lib.device_error() == 0
