"""The INT8 linear and the expert layer as programs use them beyond a single call: streams given to a call, buffers and
workspaces shared by consecutive dependent launches, inputs updated in place.  All outputs are compared bit for bit with
those of separate calls."""
import numpy as np
import pytest

from bit_quantized_decode_gb300 import workloads as wl
from helpers import cuda_ok, dev

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module")
def bq():
    import bit_quantized_decode_gb300 as pkg
    pkg._lib.load()
    pkg._lib.clear_device_error()
    yield pkg
    assert pkg._lib.device_error() == 0


def _moe(bq, fmt, g, H, I, E, k):
    router = bq.MoeRouter(dev((g.standard_normal((E, H)) * 0.03).astype(np.float32)), k, norm=dev(wl.norm_weight(g, H)))
    gu = (dev(wl.weights(g, 2 * I, H)) for _ in range(E))
    dn = (dev(wl.weights(g, H, I)) for _ in range(E))
    return bq.MoeLayer.from_float(fmt, router, gu, dn)


@pytest.mark.parametrize("M", [1, 12, 300])
def test_linear_on_a_given_stream_makes_its_own_tensors(bq, M):
    """Temporaries of a call on another stream are not handed to the current stream's work while that call runs."""
    import torch
    g = wl.rng(M)
    lin = bq.QuantLinear.from_float("w8", [dev(wl.weights(g, 520, 2048))])
    xs = [dev(wl.activations(g, M, 2048)) for _ in range(4)]
    want = [lin(x).clone() for x in xs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ys = []
    for i in range(24):
        ys.append(lin(xs[i % 4], stream=side))
        torch.full((M * 2048 + 1 << 10,), 255, dtype=torch.uint8, device="cuda")       # reuses what the current stream freed
        torch.full((M,), float("nan"), device="cuda")
    torch.cuda.synchronize()
    for i, y in enumerate(ys):
        assert torch.equal(y, want[i % 4])


@pytest.mark.parametrize("fmt", ["w4", "w8"])
def test_expert_layer_on_a_given_stream_and_in_place(bq, fmt):
    import torch
    g = wl.rng(5)
    H = 512
    layer = _moe(bq, fmt, g, H, 256, 12, 3)
    side = torch.cuda.Stream()
    for M in (1, 2, 7, 16):
        x = dev(wl.residual_stream(g, M, H))
        want = layer(x, residual=x).clone()
        torch.cuda.synchronize()
        ys = [layer(x, residual=x, stream=side) for _ in range(6)]
        torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for y in ys:
            assert torch.equal(y, want)
        # x, the residual and y in one tensor
        b = layer.buffers(M)
        b.y.copy_(x)
        layer(b.y, b, residual=b.y)
        assert torch.equal(b.y, want)


def test_dependent_launches_share_buffers_and_workspaces(bq):
    """Consecutive calls of different token counts on one workspace, each a dependent launch of the one before."""
    import torch
    g = wl.rng(8)
    K, N, H = 1536, 1000, 512
    lin = bq.QuantLinear.from_float("w8", [dev(wl.weights(g, N, K))])
    layer = _moe(bq, "w4", g, H, 256, 12, 3)
    counts = (1, 200, 2, 16, 7, 130, 1, 64)
    xs = [dev(wl.activations(g, M, K)) for M in counts]
    ts = [dev(wl.residual_stream(g, min(M, 16), H)) for M in counts]
    want, wmoe = [lin(x).clone() for x in xs], [layer(t, residual=t).clone() for t in ts]
    ws = lin.workspace(max(counts))
    bufs = {t.shape[0]: layer.buffers(t.shape[0]) for t in ts}
    shared = layer.buffers(16).workspace
    for b in bufs.values():
        b.workspace = shared
    ys, zs = [torch.empty_like(w) for w in want], [torch.empty_like(w) for w in wmoe]
    F = bq.W4_FLAG_PDL

    def step():
        for x, y, t, z in zip(xs, ys, ts, zs):
            lin(x, y, workspace=ws, flags=F)
            b = bufs[t.shape[0]]
            layer(t, b, residual=t, flags=F)
            layer(t, b, residual=t, flags=F)
            z.copy_(b.y)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(5):
        for v in ys + zs:
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(ys + zs, want + wmoe):
            assert torch.equal(got, w)


@pytest.mark.parametrize("fmt", ["w4", "w8"])
def test_many_small_expert_calls_all_finish(bq, fmt):
    """Blocks that take their tickets one at a time get them in order: thousands of small calls, each of them complete."""
    import torch
    g = wl.rng(9)
    H = 512
    layer = _moe(bq, fmt, g, H, 256, 12, 3)
    for M, calls in ((1, 6000), (2, 2000), (7, 1000)):
        x = dev(wl.residual_stream(g, M, H))
        want = layer(x, residual=x).clone()
        b = layer.buffers(M)
        wrong = torch.zeros((), dtype=torch.int64, device="cuda")
        for _ in range(calls):
            b.y.fill_(float("nan"))
            layer(x, b, residual=x)
            wrong += (b.y != want).any()
        assert int(wrong) == 0 and bq._lib.device_error() == 0


@pytest.mark.parametrize("fmt,M,H,I,E,k", [("w4", 16, 8192, 64, 4, 2), ("w8", 16, 16384, 64, 4, 2), ("w4", 9, 96, 4160, 3, 2),
                                           ("w8", 16, 2080, 2976, 3, 3), ("w4", 16, 2080, 2976, 3, 3), ("w4", 16, 32, 32, 2, 1)])
def test_batches_equal_single_tokens(bq, fmt, M, H, I, E, k):
    """Every way to batch an expert's tokens gives each of them the bits that it has alone: codes that do not fit shared
    memory, several entries to an expert, odd numbers of tiles, slices that end early, one line."""
    import torch
    g = wl.rng(M + H)
    layer = _moe(bq, fmt, g, H, I, E, k)
    x = dev(wl.residual_stream(g, M, H))
    y = layer(x).clone()
    for m in range(M):
        assert torch.equal(layer(x[m:m + 1].contiguous()), y[m:m + 1])


@pytest.mark.parametrize("M,N,K", [(16, 20000, 3584), (12, 19999, 1056), (40, 20500, 544), (9, 41000, 32), (100, 19600, 1120)])
def test_many_rows_equal_few_token_calls(bq, M, N, K):
    """Several tiles to a block: the codes that stay in shared memory serve all of them."""
    import torch
    g = wl.rng(M + K)
    lin = bq.QuantLinear.from_float("w8", [dev(wl.weights(g, N, K))])
    x = dev(wl.activations(g, M, K))
    for _ in range(2):
        y = lin(x)
        for m in range(0, M, 4):
            assert torch.equal(lin(x[m:m + 4].contiguous()), y[m:m + 4])


@pytest.mark.parametrize("M,N,K,calls", [(128, 3584, 18944, 6000), (100, 640, 7168, 4000), (16, 40000, 1024, 4000), (48, 5000, 3584, 4000)])
def test_long_runs_of_the_linear_repeat_every_bit(bq, M, N, K, calls):
    """Thousands of calls, whatever the order in which copies land: odd and even numbers of stages, split K or not."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    lin = bq.QuantLinear.from_float("w8", [torch.randn(N, K, device="cuda", generator=g)])
    x = torch.randn(M, K, device="cuda", generator=g)
    want = torch.cat([lin(x[m:m + 4].contiguous()) for m in range(0, M, 4)])
    ws, sx = lin.workspace(M), torch.empty(M, device="cuda")
    ys = [torch.empty((M, N), device="cuda") for _ in range(8)]
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(calls // len(ys)):
        for y in ys:
            lin(x, y, None, sx, workspace=ws, flags=bq.W4_FLAG_PDL)
        for y in ys:
            wrong += (y != want).any()
    assert int(wrong) == 0 and bq._lib.device_error() == 0
