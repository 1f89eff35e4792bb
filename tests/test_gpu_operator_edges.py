"""Ends of the ranges of the expert router and the expert layer: scores and gates far out, infinities, the largest codes."""
import numpy as np
import pytest

import ops_reference as ref
from bit_quantized_decode_gb300 import workloads as wl
from helpers import cuda_ok, dev, host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]
U = 2.0 ** -24


@pytest.fixture(scope="module")
def bq():
    import bit_quantized_decode_gb300 as pkg
    pkg._lib.load()
    pkg._lib.clear_device_error()
    yield pkg
    assert pkg._lib.device_error() == 0


def _stored(fmt, q):
    import oracle
    return dev(oracle.pack_int4(q).view(np.int32)) if fmt == "w4" else dev(q)


@pytest.mark.parametrize("E", [6, 70])
def test_sigmoid_scores_far_below_one_keep_their_order(bq, E):
    """Logits below -87, whose scores are subnormal: a larger one comes first, and its weight is the larger."""
    K, k = 64, 4
    l = -100.0 + 12.5 * np.linspace(0.0, 1.0, E)                   # the last expert leads
    x = np.zeros((2, K), np.float32)
    x[:, 3] = 1.0
    w = np.zeros((E, K), np.float32)
    w[:, 3] = l
    ids, weights = bq.MoeRouter(dev(w), k, score="sigmoid", renormalize=False)(dev(x))
    want, ww = ref.route(ref.logits(x, w), k, "sigmoid", None, False, 1.0)
    assert np.array_equal(host(ids), want) and host(ids)[0].tolist() == list(range(E - 1, E - 1 - k, -1))
    # one rounding of the value, to a subnormal's step and 24 bits; the product with 1 adds none
    assert (np.abs(host(weights).astype(np.float64) - ww) <= 2.0 ** -150 + U * ww).all()


@pytest.mark.parametrize("fmt", ["w4", "w8"])
@pytest.mark.parametrize("act,gate,up", [("silu", (-60.0, -50.0), 1e37), ("silu", (-92.0, -88.0), 1e3), ("silu", (1e18, 4e18), 5e18),
                                         ("gelu_tanh", (-10.6, -10.2), 1e4), ("gelu_tanh", (-12.2, -11.8), 1e37), ("silu", (1e-30, 4e-30), 1e-5)])
@pytest.mark.parametrize("M", [1, 2, 9])
def test_far_gates(bq, fmt, act, gate, up, M):
    """Gates whose activation is tiny beside a large up value, or whose product passes fp32 before the sigmoid: the layer's y
    is the definition's."""
    import torch
    H = I = 64
    top = 7 if fmt == "w4" else 127
    g = wl.rng(M)
    gu = np.zeros((2 * I, H), np.int8)
    gu[:I, 0] = top if gate[0] > 0 else -top
    gu[I:, 0] = g.choice([-top, top], I)
    size = np.concatenate([g.uniform(abs(gate[0]), abs(gate[1]), I) if gate[0] > 0 else g.uniform(abs(gate[1]), abs(gate[0]), I),
                           up * g.uniform(1.0, 2.0, I)])
    s_gu = (size / top).astype(np.float32)
    dn = wl.int_codes(g, (H, I), -top, top)
    s_dn = wl.positive_scales(g, H, 1e-3, 1e-2)
    x = np.zeros((M, H), np.float32)
    x[:, 0] = 1.0                                                   # code 127, scale 1 / 127
    q, s = ref.codes(x)
    ids, w = np.zeros((M, 1), np.int32), np.ones((M, 1), np.float32)
    layer = bq.MoeLayer.from_canonical(fmt, bq.MoeRouter(torch.zeros(1, H, device="cuda"), 1), [_stored(fmt, gu)], dev(s_gu[None]),
                                       [_stored(fmt, dn)], dev(s_dn[None]), act)
    y = torch.empty((M, H), device="cuda")
    layer.experts(dev(q.astype(np.int8)), dev(s.astype(np.float32)), dev(ids), dev(w), y)
    want, room = ref.experts(q, s, ids, w, [gu], s_gu[None], [dn], s_dn[None], act)
    assert np.isfinite(want).all() and (np.abs(want).max(axis=1) > 0).all()
    bound = 1.05 * (room + U * np.abs(want)) + 2.0 ** -148
    assert (np.abs(host(y).astype(np.float64) - want) <= bound).all()


@pytest.mark.parametrize("E,k", [(6, 3), (70, 9), (300, 16)])
def test_infinite_logits_lead_or_trail(bq, E, k):
    """A logit that passes fp32 is an infinity of its sign, not a NaN: it is the first choice, or (negative) comes after every
    finite one, and its sigmoid score is 1 or 0."""
    K = 96
    g = wl.rng(E)
    w = (g.standard_normal((E, K)) * 0.05).astype(np.float32)
    w[:, 5] = np.where(np.arange(E) % 3 == 0, -3.0, 2.0)
    w[E - 1, 5] = 5.0
    x = wl.activations(g, 5, K)
    x[0, 5], x[1, 5] = np.inf, -np.inf                      # infinite for every expert
    x[2, 5] = 1e38                                          # past fp32 for the last expert only
    x[3, 5] = -1.2e38                                       # past fp32 for the last (negative) and for every third
    with np.errstate(over="ignore"):
        l = ref.logits(x, w)
    assert np.isinf(l[:2]).all() and np.isposinf(l[2, -1]) and np.isneginf(l[3, -1]) and np.isposinf(l[3, 0]) and np.isfinite(l[4]).all()
    for score in ("softmax", "sigmoid"):
        ids, weights = bq.MoeRouter(dev(w), k, score=score, renormalize=False)(dev(x))
        with np.errstate(over="ignore", invalid="ignore"):
            want, ww = ref.route(l, k, score, None, False, 1.0)
        assert np.array_equal(host(ids), want), (host(ids), want)
        if score == "sigmoid":
            assert (np.abs(host(weights).astype(np.float64) - ww) <= U * ww + 2.0 ** -150).all()
        else:                                               # an infinite logit has no softmax
            assert np.isfinite(host(weights)[4]).all()


def test_weights_that_moved_are_found(bq):
    """New storage behind the same tensors (a reload, an update by swapping .data): the next call reads the new one."""
    import torch
    g = wl.rng(2)
    N, K, H, I, E = 72, 128, 64, 32, 3
    a, b = (bq.QuantLinear.from_float("w8", [dev(wl.weights(g, N, K))]) for _ in range(2))
    layers = [bq.MoeLayer.from_float("w4", bq.MoeRouter(dev(wl.weights(g, E, H)), 2), [dev(wl.weights(g, 2 * I, H)) for _ in range(E)],
                                     [dev(wl.weights(g, H, I)) for _ in range(E)]) for _ in range(2)]
    x, t = dev(wl.activations(g, 3, K)), dev(wl.activations(g, 2, H))
    wants = [q(x).clone() for q in (a, b)], [m(t).clone() for m in layers]
    assert not torch.equal(*wants[0]) and not torch.equal(*wants[1])
    tensors = [(a.w, b.w), (a.s_w, b.s_w)]
    for d0, d1 in ((layers[0].desc, layers[1].desc), (layers[0].router.desc, layers[1].router.desc)):
        tensors += [(p, q) for p, q in zip(d0._tensors, d1._tensors) if p is not None]
    for p, q in tensors:
        p.data, q.data = q.data, p.data
    assert torch.equal(a(x), wants[0][1]) and torch.equal(b(x), wants[0][0])
    assert torch.equal(layers[0](t), wants[1][1]) and torch.equal(layers[1](t), wants[1][0])


def _streams_of(tensors):
    """The stream whose pool holds each tensor's memory, as the allocator keeps it."""
    import torch
    segments = torch.cuda.memory_snapshot()

    def of(t):
        return next(s["stream"] for s in segments if s["address"] <= t.data_ptr() < s["address"] + s["total_size"])
    return [of(t) for t in tensors]


def test_a_call_on_a_stream_takes_its_memory_from_that_streams_pool(bq, monkeypatch):
    """Every tensor that a call makes itself, outputs and temporaries: memory that the allocator orders with the given stream."""
    import torch
    g = wl.rng(12)
    N, K, H, I, E, k = 520, 2048, 64, 32, 6, 2
    lin = bq.QuantLinear.from_float("w8", [dev(wl.weights(g, N, K))])
    router = bq.MoeRouter(dev(wl.weights(g, E, H)), k)
    layer = bq.MoeLayer.from_float("w4", router, [dev(wl.weights(g, 2 * I, H)) for _ in range(E)], [dev(wl.weights(g, H, I)) for _ in range(E)])
    made, empty = [], torch.empty

    def recording(*args, **kw):
        t = empty(*args, **kw)
        if t.is_cuda:
            made.append(t)
        return t

    side = torch.cuda.Stream()
    xs = {M: dev(wl.activations(g, M, K)) for M in (1, 12, 300)}
    codes = {M: (torch.ones((M, K), dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda"), torch.zeros((M, N), device="cuda")) for M in (1, 12, 300)}
    t = dev(wl.residual_stream(g, 5, H))
    b, y = layer.buffers(5), torch.zeros((5, H), device="cuda")
    router(t, bq.moe.RouteBuffers(b.ids, b.weights), b.qx, b.sx)
    calls = [(lambda s, x=x: lin(x, stream=s), 3) for x in xs.values()]
    calls += [(lambda s, c=c: lin.gemv(*c, stream=s), 1) for c in codes.values()]
    calls += [(lambda s: router(t, stream=s), 2), (lambda s: layer(t, stream=s), 6),
              (lambda s: layer.experts(b.qx, b.sx, b.ids, b.weights, y, stream=s), 1)]
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "empty", recording)
    for stream, handle in ((side, side.cuda_stream), (None, torch.cuda.current_stream().cuda_stream)):
        for call, count in calls:
            made.clear()
            call(stream)
            assert len(made) == count and _streams_of(made) == [handle] * count
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["w4", "w8"])
@pytest.mark.parametrize("M,H,I", [(1, 3584, 2976), (2, 3584, 2976), (16, 3584, 2976), (16, 1056, 4128)])
def test_largest_magnitudes_of_the_experts(bq, fmt, M, H, I):
    """Codes of +-127 against weights at both ends of their range, in both halves of the layer: each integer sum at its largest
    or cancelling to the last bit, one rounding in the epilogue."""
    import torch
    lo, top = (-8, 7) if fmt == "w4" else (-128, 127)

    def rows(n, K):
        w = np.full((n, K), lo, np.int8)
        w[1::4] = top
        w[2::4, ::2] = top                                         # sums that nearly cancel
        w[3::4, 1::2] = top
        w[:, 17] = np.arange(n) % (top - lo + 1) + lo              # and differ in one weight
        return w

    # gates at the top, ups at both ends with scales that make them alike: every code of h is +-127
    gu, dn = [np.full((2 * I, H), top, np.int8) for _ in range(2)], [rows(H, I) for _ in range(2)]
    for w in gu:
        w[I::2] = lo
    q = np.full((M, H), 127, np.int8)
    q[1::3] = -127
    q[2::3, ::2] = -126
    s = np.full(M, 2.0 ** -7)
    s_gu = np.full((2, 2 * I), 2.0 ** -2 / (H * top), np.float32)
    s_gu[:, I::2] = 2.0 ** -2 / (H * -lo)
    s_dn = np.full((2, H), 2.0 ** -9, np.float32)
    h = ref.act("silu", *np.split(ref.linear(q[:2], s[:2], gu[1], s_gu[1])[1], 2, axis=1))
    assert (np.abs(ref.codes(h)[0]) == 127).all()
    layer = bq.MoeLayer.from_canonical(fmt, bq.MoeRouter(torch.zeros(2, H, device="cuda"), 1), [_stored(fmt, w) for w in gu], dev(s_gu),
                                       [_stored(fmt, w) for w in dn], dev(s_dn))
    ids, w = np.ones((M, 1), np.int32), np.ones((M, 1), np.float32)
    y = torch.empty((M, H), device="cuda")
    layer.experts(dev(q), dev(s.astype(np.float32)), dev(ids), dev(w), y)
    want, room = ref.experts(q, s, ids, w, gu, s_gu, dn, s_dn, "silu")
    assert (np.abs(want).max(axis=1) > 0).all()
    assert (np.abs(host(y).astype(np.float64) - want) <= 1.05 * (room + U * np.abs(want))).all()
