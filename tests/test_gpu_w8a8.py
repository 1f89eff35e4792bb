"""The INT8 x INT8 linear for any number of tokens (w8a8_matmul, w8a8_linear, QuantLinear("w8")).

Integer sums are exact, so y differs from the 64-bit value by four roundings at most: the fp32 conversion of the sum
(2^-24 of the product), the fused multiply-add (2^-24 of y), the residual's add (2^-24 of y) and the output type's half
step.  Codes and scales are compared for equality."""
import numpy as np
import pytest

import ops_reference as ref
from bit_quantized_decode_gb300 import workloads as wl
from helpers import cuda_ok, dev, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]
U = 2.0 ** -24


@pytest.fixture(scope="module")
def lib():
    from bit_quantized_decode_gb300 import _lib
    _lib.load()
    _lib.clear_device_error()
    yield _lib
    assert _lib.device_error() == 0


def _dtype(name):
    import torch
    return getattr(torch, name)


def _repacked(lib, q):
    import torch
    w = torch.full((lib.w8_repacked_bytes(*q.shape),), 0xAB, dtype=torch.uint8, device="cuda")
    lib.w8_repack([dev(q)], q.shape[1], w)
    return w


def _workspace(lib, M, N, K):
    import torch
    return torch.full((lib.w8a8_workspace_bytes(M, N, K),), 0xFF, dtype=torch.uint8, device="cuda")   # fp16 NaN


def _check(y, want, prod, typ, extra=0.0):
    """y against the 64-bit `want`; prod: |s_w s_x acc|; extra: roundings relative to the sum before the residual."""
    y = host(y.float()).astype(np.float64)
    big = np.abs(want)
    bound = 1.01 * (U * prod + 2 * U * (big + extra) + (ref.EPS[typ] * big if typ != "float32" else 0.0)) + ref.TINY[typ]
    bad = np.abs(y - want) > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), y[bad][:4], want[bad][:4])


SHAPES = [  # M, N, K
    (1, 1, 32), (1, 4608, 3584), (2, 130, 64), (3, 128, 1024), (5, 127, 1056), (8, 512, 3584), (9, 264, 96),
    (15, 129, 2080), (16, 1000, 512), (17, 300, 1536), (31, 8, 160), (33, 640, 1088), (64, 384, 18944), (100, 257, 2016),
    (127, 136, 992), (128, 256, 2048), (129, 255, 1536), (130, 1, 3584), (257, 1000, 480), (300, 392, 1120),
    (513, 4000, 1536), (1000, 2560, 1536),
    # more tiles than SMs: pairs of blocks, with ragged tokens, rows and K, several rounds of tiles
    (1100, 2500, 96), (770, 5000, 1056), (2000, 4608, 544), (4001, 3333, 32), (200, 40000, 160),
]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul_matches_64_bits(lib, M, N, K):
    import torch
    g = wl.rng(M * 7919 + N * 31 + K)
    w, q = wl.int_codes(g, (N, K), -128, 127), wl.int_codes(g, (M, K), -127, 127)
    sw, sx, b = wl.positive_scales(g, N), wl.positive_scales(g, M), wl.bias(g, N)
    wd = _repacked(lib, w)
    for bias, typ in ((None, "float32"), (b, "bfloat16"), (b, "float16")):
        y = torch.full((M, N), float("nan"), dtype=_dtype(typ), device="cuda")
        lib.w8a8_matmul(wd, dev(sw), None if bias is None else dev(bias), dev(q), dev(sx), y, _workspace(lib, M, N, K))
        want, _ = ref.linear(q, sx, w, sw, bias)
        prod, _ = ref.linear(q, sx, w, sw)
        if typ == "float16":
            want = np.clip(want, -60000, 60000)
            y = y.clamp(-60000, 60000)
        _check(y, want, np.abs(prod), typ)


@pytest.mark.parametrize("M", [1, 4, 16, 40, 200])
def test_largest_magnitudes_stay_exact(lib, M):
    """Every product at its largest, K past what one fp32 accumulator holds exactly: with unit scales y is fp32(acc)."""
    import torch
    K, N = 18944, 136
    q = np.full((M, K), 127, np.int8)
    q[1::2] = -127
    w = np.full((N, K), -128, np.int8)
    w[1::3] = 127
    w[2::3, ::2] = 127                       # sums that cancel to the last bit
    w[5, 17] = 126
    one = lambda n: np.ones(n, np.float32)   # noqa: E731
    y = torch.empty((M, N), device="cuda")
    lib.w8a8_matmul(_repacked(lib, w), dev(one(N)), None, dev(q), dev(one(M)), y, _workspace(lib, M, N, K))
    acc = q.astype(np.int64) @ w.astype(np.int64).T
    assert np.array_equal(host(y), acc.astype(np.float32))


@pytest.mark.parametrize("xt,yt", [("float32", "float32"), ("bfloat16", "bfloat16"), ("float16", "float32"),
                                   ("float32", "float16")])
@pytest.mark.parametrize("M,N,K", [(1, 500, 3584), (7, 384, 512), (16, 130, 1536), (70, 264, 96), (333, 392, 3584),
                                   (3, 136, 20512)])
@pytest.mark.parametrize("norm", [False, True])
def test_linear_matches_64_bits(lib, M, N, K, xt, yt, norm):
    import torch
    g = wl.rng(M + 3 * N + K + norm)
    x = dev(wl.residual_stream(g, M, K)).to(_dtype(xt))
    if M > 2:
        x[2] = 0.0                                                # an all-zero token: scale 0, y = b
    gamma, b, res = wl.norm_weight(g, K), wl.bias(g, N), wl.residual_stream(g, M, N)
    w = wl.int_codes(g, (N, K), -127, 127)
    sw = wl.positive_scales(g, N, 1e-4, 1e-3)
    xf = host(x.float())
    q, s = ref.codes(ref.rmsnorm(xf, gamma, 1e-6) if norm else xf)
    residual = res if yt == "float32" else None
    y = torch.full((M, N), float("nan"), dtype=_dtype(yt), device="cuda")
    qx, sx = torch.empty((M, K), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    lib.w8a8_linear(_repacked(lib, w), dev(sw), dev(b), x, y, qx, sx, _workspace(lib, M, N, K),
                    dev(gamma) if norm else None, 1e-6, None if residual is None else dev(residual))
    assert np.array_equal(host(sx).astype(np.float64), s)
    assert np.array_equal(host(qx).astype(np.float64), q)
    want, _ = ref.linear(q, s, w, sw, b)
    prod, _ = ref.linear(q, s, w, sw)
    extra = np.abs(want)
    if residual is not None:
        want = want + residual
    _check(y, want, np.abs(prod), yt, extra)


def test_a_token_is_the_same_in_every_batch(lib):
    """Row m of a call does not depend on the other rows, nor on how many there are."""
    import torch
    g = wl.rng(5)
    N, K, M = 520, 1536, 200
    w, sw = wl.int_codes(g, (N, K), -127, 127), wl.positive_scales(g, N)
    from bit_quantized_decode_gb300 import QuantLinear
    lin = QuantLinear.from_canonical("w8", [dev(w)], K, [dev(sw)])
    x = dev(wl.activations(g, M, K, outliers=True))
    whole = lin(x)
    for m0, m1 in ((0, 1), (3, 5), (10, 17), (20, 36), (40, 73), (100, 200)):
        assert torch.equal(lin(x[m0:m1].contiguous()), whole[m0:m1]), (m0, m1)


def test_linear_without_outputs_or_tokens(lib):
    import torch
    x = torch.randn(3, 64, device="cuda")
    qx, sx = torch.empty((3, 64), dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
    empty = torch.empty(0, dtype=torch.uint8, device="cuda")
    lib.w8a8_linear(empty, torch.empty(0, device="cuda"), None, x, torch.empty((3, 0), device="cuda"), qx, sx,
                    _workspace(lib, 3, 0, 64))
    q, s = ref.codes(host(x))
    assert np.array_equal(host(qx).astype(np.float64), q) and np.array_equal(host(sx).astype(np.float64), s)
    w = torch.zeros(lib.w8_repacked_bytes(8, 64), dtype=torch.uint8, device="cuda")
    lib.w8a8_linear(w, torch.ones(8, device="cuda"), None, x[:0], torch.empty((0, 8), device="cuda"), None,
                    sx[:0], empty)


def test_rows_behind_the_last_token_stay(lib):
    """Nothing past [M][N] of y is written, nothing past M of sx."""
    import torch
    g = wl.rng(11)
    for M, N, K in ((5, 130, 96), (20, 70, 64), (131, 129, 64)):
        w, sw = wl.int_codes(g, (N, K), -127, 127), wl.positive_scales(g, N)
        y = torch.full((M * N + 257,), 3.25, device="cuda")
        sx = torch.full((M + 9,), 3.25, device="cuda")
        x = dev(wl.activations(g, M, K))
        lib.w8a8_linear(_repacked(lib, w), dev(sw), None, x, y[:M * N].view(M, N), None, sx[:M], _workspace(lib, M, N, K))
        assert (y[M * N:] == 3.25).all() and (sx[M:] == 3.25).all()


def test_captured_and_replayed_on_another_stream(lib):
    import torch
    from bit_quantized_decode_gb300 import QuantLinear
    g = wl.rng(6)
    N, K, M = 392, 1536, 50
    lin = QuantLinear.from_float("w8", [dev(wl.weights(g, 200, K)), dev(wl.weights(g, 192, K))])
    x = dev(wl.activations(g, M, K))
    bufs, ws = lin.buffers(M), lin.workspace(M)
    want = [lin(x * k).clone() for k in (1.0, -2.0)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        lin(x, *bufs, workspace=ws)
    graph.replay()
    assert torch.equal(bufs[0], want[0])
    x.mul_(-2.0)
    graph.replay()
    assert torch.equal(bufs[0], want[1])
    x.mul_(-0.5)
    side.wait_stream(torch.cuda.current_stream())
    y = torch.empty((M, N), device="cuda")
    with torch.cuda.stream(side):
        lin(x, y, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(y, want[0])
