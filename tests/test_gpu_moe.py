"""The expert router, the experts and the whole mixture-of-experts layer for 1 to 16 tokens.

Choices and codes are compared for equality.  Router weights: an exponential of the CUDA library is off by at most two
steps (2^-22 relative) and its argument by 2^-24 of its magnitude, in the numerator and in the sum; the sum has at most
E / 32 + 5 additions, then a division and a product.  The layer's y: per slot the fp32 conversion of the integer sum and
one fused multiply-add, then one rounding of the running sum per slot (ops_reference.experts counts them), the
residual's add and the output type's half step."""
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


def _dtype(name):
    import torch
    return getattr(torch, name)


def _weights_close(w, want, l, E, renorm):
    span = float((l.max(axis=1) - l.min(axis=1)).max()) + float(np.abs(l).max())
    rel = 2 * (2 ** -22 + (span + 1) * U) + (E / 32 + 5 + 4) * U
    assert (np.abs(host(w).astype(np.float64) - want) <= rel * np.abs(want) + 1e-38).all()


# --------------------------------------------------------------- router
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,top_k,K,xt", [
    (1, 1, 1, 32, "float32"), (1, 64, 8, 3584, "float32"), (2, 2, 2, 96, "bfloat16"), (3, 60, 4, 1536, "float16"),
    (4, 64, 1, 512, "float32"), (5, 65, 16, 2048, "bfloat16"), (7, 8, 8, 7168, "float32"), (16, 256, 6, 1536, "bfloat16"),
    (9, 1000, 10, 64, "float32"), (16, 1024, 16, 3584, "float32"), (3, 33, 5, 20480, "float32"), (2, 16, 4, 40960, "float16"),
])
def test_route_matches_64_bits(bq, M, E, top_k, K, xt, score):
    import torch
    g = wl.rng(M * 131 + E * 7 + K)
    x = dev(wl.residual_stream(g, M, K)).to(_dtype(xt))
    w = (g.standard_normal((E, K)) * 0.03).astype(np.float32)
    gamma, bias = wl.norm_weight(g, K), (0.1 * g.standard_normal(E)).astype(np.float32)
    for norm, renorm, scale in ((True, True, 1.0), (True, False, 2.5), (False, True, 0.5)):
        b = bias if score == "sigmoid" and renorm else None
        r = bq.MoeRouter(dev(w), top_k, None if b is None else dev(b), score, renorm, scale, dev(gamma) if norm else None, 1e-5)
        qx, sx = torch.empty((M, K), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        ids, weights = r(x, qx=qx, sx=sx)
        xn = host(x.float()).astype(np.float64)
        if norm:
            xn = ref.rmsnorm(xn, gamma, 1e-5)
        q, s = ref.codes(xn)
        assert np.array_equal(host(qx).astype(np.float64), q) and np.array_equal(host(sx).astype(np.float64), s)
        l = ref.logits(xn * 1.0, w)
        want_ids, want_w = ref.route(l, top_k, score, b, renorm, scale)
        assert np.array_equal(host(ids), want_ids)
        _weights_close(weights, want_w, l, E, renorm)
        again, _ = r(x)                                    # without codes
        assert torch.equal(again, ids)


def test_equal_scores_take_the_lowest_index(bq):
    import torch
    g = wl.rng(3)
    K, E = 256, 96
    w = (g.standard_normal((E, K)) * 0.05).astype(np.float32)
    w[40:80] = w[7]                                        # forty equal experts, ties within and across lanes
    w[90] = 0.0
    w[91] = -0.0
    x = wl.activations(g, 3, K)
    x[0] = 3.0 * w[7] / np.abs(w[7]).max()                 # the equal ones lead
    x[1] = 0.0                                             # every logit 0
    for score, bias in (("softmax", None), ("sigmoid", None), ("sigmoid", np.zeros(E, np.float32))):
        ids, weights = bq.MoeRouter(dev(w), 12, None if bias is None else dev(bias), score)(dev(x))
        want, ww = ref.route(ref.logits(x, w), 12, score, bias, True, 1.0)
        assert np.array_equal(host(ids), want)
        assert host(ids)[0].tolist() == [7] + list(range(40, 51)) and host(ids)[1].tolist() == list(range(12))
        assert np.allclose(host(weights), ww, rtol=1e-6)
    assert torch.isfinite(weights).all()


def test_ids_are_valid_whatever_the_input(bq):
    import torch
    K, E, k = 64, 40, 8
    w = torch.randn(E, K, device="cuda")
    x = torch.randn(6, K, device="cuda")
    x[0] = float("nan")
    x[1, 3] = float("inf")
    x[2] = 1e38
    x[3, 5] = float("-inf")
    w[11] = float("nan")
    for score in ("softmax", "sigmoid"):
        ids, _ = bq.MoeRouter(w, k, score=score)(x)
        for row in host(ids):
            assert len(set(row.tolist())) == k and row.min() >= 0 and row.max() < E
        assert 11 not in host(ids)[4:].ravel().tolist()    # a NaN score is the last choice


# -------------------------------------------------------------- experts
def _experts(bq, fmt, n, H, I, seed, biased=False):
    g = wl.rng(seed)
    top = 7 if fmt == "w4" else 127
    lo = -top - 1
    gu = [wl.int_codes(g, (2 * I, H), lo, top) for _ in range(n)]
    dn = [wl.int_codes(g, (H, I), lo, top) for _ in range(n)]
    sgu = np.stack([wl.positive_scales(g, 2 * I, 0.2 / top / np.sqrt(H), 1.0 / top / np.sqrt(H)) for _ in range(n)])
    sdn = np.stack([wl.positive_scales(g, H, 0.2 / top / np.sqrt(I), 1.0 / top / np.sqrt(I)) for _ in range(n)])
    bgu = np.stack([wl.bias(g, 2 * I) for _ in range(n)]) if biased else None
    bdn = np.stack([wl.bias(g, H) for _ in range(n)]) if biased else None
    return gu, dn, sgu, sdn, bgu, bdn


def _stored(fmt, q):
    import oracle
    return dev(oracle.pack_int4(q).view(np.int32)) if fmt == "w4" else dev(q)


def _layer(bq, fmt, router, ex, act, shared):
    gu, dn, sgu, sdn, bgu, bdn = ex
    return bq.MoeLayer.from_canonical(fmt, router, [_stored(fmt, q) for q in gu], dev(sgu), [_stored(fmt, q) for q in dn],
                                      dev(sdn), act, shared, None if bgu is None else dev(bgu), None if bdn is None else dev(bdn))


def _check_y(y, want, room, typ, res):
    y = host(y.float()).astype(np.float64)
    bound = 1.05 * (room + U * np.abs(want) * (2 if res else 1) + (ref.EPS[typ] * np.abs(want) if typ != "float32" else 0.0))
    bound += ref.TINY[typ] + 1e-30
    bad = np.abs(y - want) > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), y[bad][:4], want[bad][:4], bound[bad][:4])


CASES = [  # fmt, M, H, I, E, shared, top_k, act, biased, y type, residual
    ("w4", 1, 32, 32, 1, 0, 1, "silu", False, "float32", False),
    ("w4", 1, 1536, 768, 8, 0, 4, "gelu_tanh", False, "float32", True),
    ("w4", 2, 544, 1120, 6, 1, 2, "silu", True, "bfloat16", False),
    ("w4", 3, 96, 2368, 4, 0, 3, "silu", False, "float16", False),
    ("w4", 5, 3584, 96, 5, 2, 2, "gelu_tanh", True, "float32", True),
    ("w4", 16, 512, 544, 7, 0, 3, "silu", False, "float32", False),
    ("w4", 16, 256, 256, 40, 1, 6, "silu", True, "float32", True),
    ("w8", 1, 64, 32, 3, 0, 2, "silu", False, "float32", False),
    ("w8", 2, 1536, 768, 6, 1, 4, "silu", False, "bfloat16", False),
    ("w8", 7, 160, 1120, 9, 0, 5, "gelu_tanh", True, "float32", True),
    ("w8", 16, 512, 256, 3, 4, 2, "silu", False, "float16", False),
]


@pytest.mark.parametrize("fmt,M,H,I,E,shared,top_k,act,biased,yt,res", CASES)
def test_experts_match_64_bits(bq, fmt, M, H, I, E, shared, top_k, act, biased, yt, res):
    import torch
    ex = _experts(bq, fmt, E + shared, H, I, M + H + I + E, biased)
    gu, dn, sgu, sdn, bgu, bdn = ex
    layer = _layer(bq, fmt, bq.MoeRouter(torch.zeros(E, H, device="cuda"), min(top_k, E)), ex, act, shared)
    g = wl.rng(17 * M + E)
    q, s = ref.codes(wl.activations(g, M, H))
    patterns = [np.stack([g.permutation(E)[:top_k] for _ in range(M)])]
    patterns.append(np.full((M, top_k), E - 1))            # every slot the same expert: duplicates in a token
    mixed = g.integers(-2, E + 2, size=(M, top_k))         # empty slots on both sides of the range
    mixed[0] = -1                                          # a token without any expert
    mixed[-1, -1] = 2 ** 31 - 1
    patterns.append(mixed)
    patterns.append(np.full((M, top_k), -7))               # no expert at all
    for ids in patterns:
        w = g.uniform(-0.5, 1.0, size=(M, top_k)).astype(np.float32)
        r = wl.residual_stream(g, M, H) if res else None
        y = torch.full((M, H), float("nan"), dtype=_dtype(yt), device="cuda")
        ws = torch.full((layer.buffers(M).workspace.numel() if top_k == layer.router.top_k else
                         bq._lib.w4_moe_workspace_bytes(layer.desc, M, top_k),), 0xFF, dtype=torch.uint8, device="cuda")
        layer.experts(dev(q.astype(np.int8)), dev(s.astype(np.float32)), dev(ids.astype(np.int32)), dev(w), y, ws,
                      None if r is None else dev(r))
        want, room = ref.experts(q, s, ids, w, gu, sgu, dn, sdn, act, shared, bgu, bdn)
        _check_y(y, want if r is None else want + r, room, yt, res)


@pytest.mark.parametrize("fmt,M,E,shared,top_k,score,act,xt,yt,res", [
    ("w4", 1, 16, 0, 4, "softmax", "silu", "float32", "float32", True),
    ("w4", 4, 64, 0, 8, "softmax", "gelu_tanh", "bfloat16", "bfloat16", False),
    ("w4", 16, 24, 1, 6, "sigmoid", "silu", "float32", "float32", True),
    ("w8", 3, 12, 2, 2, "sigmoid", "silu", "float16", "float32", True),
    ("w8", 16, 8, 0, 8, "softmax", "silu", "bfloat16", "float16", False),
])
def test_layer_matches_64_bits(bq, fmt, M, E, shared, top_k, score, act, xt, yt, res):
    import torch
    H, I = 768, 416
    g = wl.rng(M * E + top_k)
    ex = _experts(bq, fmt, E + shared, H, I, 5 * M + E)
    gamma, rw = wl.norm_weight(g, H), (g.standard_normal((E, H)) * 0.03).astype(np.float32)
    bias = (0.1 * g.standard_normal(E)).astype(np.float32) if score == "sigmoid" else None
    router = bq.MoeRouter(dev(rw), top_k, None if bias is None else dev(bias), score, True, 1.5, dev(gamma), 1e-6)
    layer = _layer(bq, fmt, router, ex, act, shared)
    x = dev(wl.residual_stream(g, M, H)).to(_dtype(xt))
    r = wl.residual_stream(g, M, H) if res else None
    b = layer.buffers(M, _dtype(yt))
    layer(x, b, None if r is None else dev(r))
    xn = ref.rmsnorm(host(x.float()), gamma, 1e-6)
    q, s = ref.codes(xn)
    l = ref.logits(xn, rw)
    ids, w = ref.route(l, top_k, score, bias, True, 1.5)
    assert np.array_equal(host(b.ids), ids) and np.array_equal(host(b.qx).astype(np.float64), q)
    _weights_close(b.weights, w, l, E, True)
    # the layer's own fp32 weights: their error is the router's, bounded above
    want, room = ref.experts(q, s, ids, host(b.weights).astype(np.float64), ex[0], ex[2], ex[1], ex[3], act, shared)
    _check_y(b.y, want if r is None else want + r, room, yt, res)


def test_from_float_quantizes_as_the_row_quantizers(bq):
    import torch
    g = wl.rng(8)
    H, I, E = 64, 32, 3
    for fmt, quant, top in (("w4", bq._lib.w4_quantize_rows, 7), ("w8", bq._lib.w8_quantize_rows, 127)):
        gu = [dev(wl.weights(g, 2 * I, H)) for _ in range(E)]
        dn = [dev(wl.weights(g, H, I)) for _ in range(E)]
        router = bq.MoeRouter(dev(wl.weights(g, E, H)), 2)
        a = bq.MoeLayer.from_float(fmt, router, gu, dn)
        codes = lambda W: np.clip(np.rint(host(W) / np.float32(1) / (np.abs(host(W)).max(1, keepdims=True) / np.float32(top))), -top, top)  # noqa: E731
        scale = lambda W: np.abs(host(W)).max(1) / np.float32(top)                  # noqa: E731
        b = bq.MoeLayer.from_canonical(fmt, router, [_stored(fmt, codes(W).astype(np.int8)) for W in gu],
                                       dev(np.stack([scale(W) for W in gu])), [_stored(fmt, codes(W).astype(np.int8)) for W in dn],
                                       dev(np.stack([scale(W) for W in dn])))
        x = dev(wl.activations(g, 2, H))
        assert torch.equal(a(x), b(x))


def test_repeats_other_tokens_and_the_batch_change_nothing(bq):
    """The same bits from every call, alone or in a batch, in place on the residual or not, and from two streams at once."""
    import torch
    H, I, E, k = 1536, 768, 24, 4
    g = wl.rng(21)
    router = bq.MoeRouter(dev((g.standard_normal((E, H)) * 0.03).astype(np.float32)), k, norm=dev(wl.norm_weight(g, H)))
    layers = [_layer(bq, fmt, router, _experts(bq, fmt, E, H, I, 31), "silu", 0) for fmt in ("w4", "w8")]
    x = dev(wl.residual_stream(g, 16, H))
    for layer in layers:
        want = layer(x, residual=x).clone()
        for _ in range(10):
            assert torch.equal(layer(x, residual=x), want)
        for m0, m1 in ((0, 1), (3, 5), (8, 16)):
            assert torch.equal(layer(x[m0:m1].contiguous(), residual=x[m0:m1].contiguous()), want[m0:m1])
        b = layer.buffers(16)
        b.y.copy_(x)
        layer(x, b, residual=b.y)                           # the residual stream updated in place
        assert torch.equal(b.y, want)
    wants = [layer(x).clone() for layer in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    bufs = [layer.buffers(16) for layer in layers]
    torch.cuda.synchronize()
    for _ in range(8):
        for layer, st, b in zip(layers, streams, bufs):
            with torch.cuda.stream(st):
                layer(x, b)
    torch.cuda.synchronize()
    for b, want in zip(bufs, wants):
        assert torch.equal(b.y, want)


def test_decoder_block_captured_with_dependent_launches(bq):
    """INT8 projections and the expert layer as a decode step runs them: norm and q/k/v, the output projection added to the
    residual stream, the expert layer added to it, captured once and replayed on new tokens."""
    import torch
    H, I, E, k, M = 1024, 512, 16, 4, 6
    g = wl.rng(44)
    N = H + 256
    wq, wo = wl.int_codes(g, (N, H), -127, 127), wl.int_codes(g, (H, H), -127, 127)
    sq, so = wl.positive_scales(g, N, 1e-4, 6e-4), wl.positive_scales(g, H, 1e-4, 6e-4)
    g1, g2 = wl.norm_weight(g, H), wl.norm_weight(g, H)
    qkv = bq.QuantLinear.from_canonical("w8", [dev(wq)], H, [dev(sq)])
    out = bq.QuantLinear.from_canonical("w8", [dev(wo)], H, [dev(so)])
    rw = (g.standard_normal((E, H)) * 0.03).astype(np.float32)
    ex = _experts(bq, "w4", E, H, I, 91)
    layer = _layer(bq, "w4", bq.MoeRouter(dev(rw), k, norm=dev(g2)), ex, "silu", 0)
    F = bq.W4_FLAG_PDL
    h = torch.zeros((M, H), device="cuda")
    a = torch.zeros((M, H), device="cuda")
    y1, _, s1 = qkv.buffers(M)
    s2 = torch.empty(M, device="cuda")
    w1, w2, b, gd = qkv.workspace(M), out.workspace(M), layer.buffers(M), dev(g1)

    def step():
        qkv(h, y1, None, s1, norm=gd, workspace=w1, flags=F)
        a.copy_(y1[:, :H])
        out(a, h, None, s2, residual=h, workspace=w2)
        layer(h, b, residual=h, flags=F)

    graph = torch.cuda.CUDAGraph()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        x = wl.residual_stream(wl.rng(seed), M, H)
        h.copy_(dev(x))
        graph.replay()
        torch.cuda.synchronize()
        q, s = ref.codes(ref.rmsnorm(x, g1, 1e-6))
        _, v = ref.linear(q, s, wq, sq)
        assert np.array_equal(host(y1).astype(np.float64), v)
        q, s = ref.codes(v[:, :H])
        want = ref.one(x + ref.linear(q, s, wo, so)[1])
        assert np.array_equal(host(h).astype(np.float64), want)
        xn = ref.rmsnorm(want, g2, 1e-6)
        ids, _ = ref.route(ref.logits(xn, rw), k, "softmax", None, True, 1.0)
        assert np.array_equal(host(b.ids), ids)
        q, s = ref.codes(xn)
        y, room = ref.experts(q, s, ids, host(b.weights).astype(np.float64), ex[0], ex[2], ex[1], ex[3], "silu")
        _check_y(b.y, y + want, room, "float32", True)
