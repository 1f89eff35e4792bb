"""What the calls of the INT8 linear, the router and the expert layer hand to the library when a weight's memory has moved
(a new storage in place, a reload, another device): the addresses of the call, checked again.  No GPU: the tensors pass for
CUDA tensors and the library's entry points record their arguments."""
import types

import pytest
import torch

from bit_quantized_decode_gb300 import QuantLinear, _lib, build


@pytest.fixture
def calls(monkeypatch):
    build.build()
    real = _lib.load()
    seen = []

    def record(name):
        def fn(*args):
            seen.append((name, args))
            return 0
        return fn

    fake = types.SimpleNamespace(**{n: record(n) for n in ("w8a8_linear", "w8a8_matmul", "w4_moe_route", "w4_moe_experts", "w4_moe_layer")},
                                 w8_repacked_bytes=real.w8_repacked_bytes, w4_repacked_bytes=real.w4_repacked_bytes,
                                 w4_glu_repacked_bytes=real.w4_glu_repacked_bytes)
    monkeypatch.setattr(_lib, "load", lambda: fake)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: getattr(t, "at", 0))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(_lib, "_raw_stream", lambda stream, device: 0)
    return seen


def _swap(t, other=None):
    """A new storage behind the same tensor; the old one stays alive, so that the address is another."""
    old = t.data
    t.data = old.clone() if other is None else other
    assert t.data_ptr() != old.data_ptr()
    return old


def test_linear_takes_the_addresses_of_the_call(calls):
    N, K, M = 8, 64, 3
    lin = QuantLinear("w8", N, K, torch.zeros(_lib.w8_repacked_bytes(N, K), dtype=torch.uint8), torch.zeros(N), torch.zeros(N), None)
    x, y, sx, ws = torch.zeros(M, K), torch.zeros(M, N), torch.zeros(M), torch.zeros(1 << 14, dtype=torch.uint8)
    call = lambda: lin(x, y, None, sx, workspace=ws)                   # noqa: E731
    expect = lambda: (lin.w.data_ptr(), lin.s_w.data_ptr(), lin.bias.data_ptr())   # noqa: E731
    call()
    assert calls[-1][1][:3] == expect()
    keep = []
    for t in (lin.w, lin.s_w, lin.bias):
        keep.append(_swap(t))
        call()
        assert calls[-1][1][:3] == expect()
    lin.s_w = torch.ones(N)                                             # another tensor
    call()
    assert calls[-1][1][:3] == expect()
    n = len(calls)
    for t, bad in ((lin.w, torch.zeros(64, dtype=torch.uint8)), (lin.s_w, torch.zeros(N - 1)), (lin.bias, torch.zeros(N, dtype=torch.float64))):
        old = _swap(t, bad)                                             # too small, of another shape or type
        with pytest.raises(ValueError):
            call()
        t.data = old
    assert len(calls) == n
    call()


def _experts(E, H, I):
    w_gu = torch.zeros(E * _lib.w4_glu_repacked_bytes(I, H), dtype=torch.uint8)
    w_dn = torch.zeros(E * _lib.w4_repacked_bytes(H, I), dtype=torch.uint8)
    return _lib.moe_experts("w4", w_gu, torch.zeros(E, 2 * I), w_dn, torch.zeros(E, H), E, 0, H, I, _lib.W4_GLU_SILU,
                            torch.zeros(E, 2 * I), torch.zeros(E, H))


def test_descriptors_take_the_addresses_of_the_call(calls):
    E, H, I, M, k = 4, 64, 32, 2, 2
    r = _lib.moe_router(torch.zeros(E, H), k, torch.zeros(E), "sigmoid", norm=torch.zeros(H))
    e = _experts(E, H, I)
    x, ids, w = torch.zeros(M, H), torch.zeros(M, k, dtype=torch.int32), torch.zeros(M, k)
    qx, sx, y, ws = torch.zeros(M, H, dtype=torch.int8), torch.zeros(M), torch.zeros(M, H), torch.zeros(1 << 16, dtype=torch.uint8)

    def layer():
        _lib.w4_moe_layer(r, e, x, ids, w, qx, sx, y, ws)
        a = calls[-1][1]
        return a[0]._obj, a[1]._obj

    def right(dr, de):
        assert (dr.w, dr.select_bias, dr.norm_weight) == tuple(t.data_ptr() for t in r._tensors)
        assert (de.w_gu, de.s_gu, de.b_gu, de.w_dn, de.s_dn, de.b_dn) == tuple(t.data_ptr() for t in e._tensors)

    right(*layer())
    keep = []
    for t in (*r._tensors, *e._tensors):
        keep.append(_swap(t))
        right(*layer())
    keep.append(_swap(r._tensors[0]))
    _lib.w4_moe_route(r, x, ids, w)
    assert calls[-1][1][0]._obj.w == r._tensors[0].data_ptr()
    keep.append(_swap(e._tensors[0]))
    _lib.w4_moe_experts(e, qx, sx, ids, w, y, ws)
    assert calls[-1][1][0]._obj.w_gu == e._tensors[0].data_ptr()
    n = len(calls)
    for t, bad in ((r._tensors[0], torch.zeros(E, H - 32)), (e._tensors[0], torch.zeros(16, dtype=torch.uint8)), (e._tensors[4], torch.zeros(E, H, dtype=torch.float64))):
        old = _swap(t, bad)
        with pytest.raises(ValueError):
            layer()
        t.data = old
    assert len(calls) == n
    right(*layer())


@pytest.mark.parametrize("fmt", ["w8", "w8a32", "q4_0"])
def test_a_chain_takes_int4_rows_only(calls, fmt):
    """A chain reads its weights as per-row INT4: the INT8 linear's bytes would be taken for twice as many of them."""
    from bit_quantized_decode_gb300 import LinearChain
    N, K = 8, 64
    lin = QuantLinear(fmt, N, K, torch.zeros(_lib.w8_repacked_bytes(N, K), dtype=torch.uint8), torch.zeros(N), None, None)
    x, y = torch.zeros(1, K), torch.zeros(1, N)
    with pytest.raises(ValueError, match="per-row INT4"):
        LinearChain([(lin, x, y, torch.zeros((1, K), dtype=torch.int8), torch.zeros(1))], 1)


def test_every_imported_function_is_public():
    import bit_quantized_decode_gb300 as bq
    names = {n for n, v in vars(bq).items() if not n.startswith("_") and not isinstance(v, types.ModuleType)}
    assert names - {"annotations"} == set(bq.__all__)


def test_a_smaller_tensor_at_the_same_address_is_checked(calls):
    """A part of the old storage, or another type in it: the address alone does not show it."""
    N, K, M, E, H, I = 8, 64, 3, 4, 64, 32
    lin = QuantLinear("w8", N, K, torch.zeros(_lib.w8_repacked_bytes(N, K), dtype=torch.uint8), torch.zeros(N), torch.zeros(N), None)
    r, e = _lib.moe_router(torch.zeros(E, H), 2, torch.zeros(E), "sigmoid", norm=torch.zeros(H)), _experts(E, H, I)
    x, y, sx, ws = torch.zeros(M, K), torch.zeros(M, N), torch.zeros(M), torch.zeros(1 << 16, dtype=torch.uint8)
    ids, w, qx, z = torch.zeros(M, 2, dtype=torch.int32), torch.zeros(M, 2), torch.zeros(M, H, dtype=torch.int8), torch.zeros(M, H)
    linear = lambda: lin(x, y, None, sx, workspace=ws)                          # noqa: E731
    layer = lambda: _lib.w4_moe_layer(r, e, x, ids, w, qx, sx, z, ws)           # noqa: E731
    for call, tensors in ((linear, (lin.w, lin.s_w, lin.bias)), (layer, (*r._tensors, *e._tensors))):
        call()
        for t in tensors:
            whole = t.data
            for part in (whole[:-1], whole.view(torch.int8)[..., : whole.shape[-1]] if whole.element_size() > 1 else whole[: 1]):
                assert part.data_ptr() == whole.data_ptr()
                t.data = part
                n = len(calls)
                with pytest.raises(ValueError):
                    call()
                assert len(calls) == n
                t.data = whole
            call()
