"""Host-side refusals of the INT8 x INT8 linear, the expert router and the mixture-of-experts layer: every bad argument
comes back as a status (C ABI) or a ValueError (tensors) before any device query or launch, and empty calls succeed."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x1000)       # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x1004)        # 4-byte but not 16-byte aligned
ODD2 = ctypes.c_void_p(0x1002)       # 2-byte aligned
OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3
BIG = 1 << 40                        # workspace bytes that suffice
by = ctypes.byref


@pytest.fixture(scope="module")
def L():
    from bit_quantized_decode_gb300 import _lib, build
    build.build()
    _lib.load()
    return _lib


def call(fn, base, **change):
    """fn with `base`'s arguments in order, some of them changed."""
    assert set(change) <= set(base)
    return fn(*{**base, **change}.values())


MATMUL = dict(w=FAKE, s_w=FAKE, bias=None, qx=FAKE, sx=FAKE, M=20, N=8, K=64, y=FAKE, y_type=0, ws=FAKE, ws_bytes=BIG, s=None)
LINEAR = dict(w=FAKE, s_w=FAKE, bias=None, x=FAKE, x_type=0, M=20, N=8, K=64, y=FAKE, y_type=0, qx=None, sx=FAKE, f=None,
              flags=0, ws=FAKE, ws_bytes=BIG, s=None)

SHAPES = [(dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID), (dict(K=-32), INVALID), (dict(K=48), SHAPE),
          (dict(K=131072 + 32), SHAPE), (dict(M=(1 << 20) + 1), SHAPE), (dict(N=1 << 30), SHAPE),
          (dict(M=1 << 20, N=1 << 29), SHAPE)]


@pytest.mark.parametrize("change,status", SHAPES + [
    (dict(w=None), INVALID), (dict(s_w=None), INVALID), (dict(qx=None), INVALID), (dict(sx=None), INVALID),
    (dict(y=None), INVALID), (dict(ws=None), INVALID), (dict(y_type=3), INVALID), (dict(y_type=-1), INVALID),
    (dict(ws_bytes=0), SHAPE), (dict(w=ODD), MISALIGNED), (dict(qx=ODD), MISALIGNED), (dict(ws=ODD), MISALIGNED),
    (dict(s_w=ODD2), MISALIGNED), (dict(sx=ODD2), MISALIGNED), (dict(bias=ODD2), MISALIGNED), (dict(y=ODD2), MISALIGNED),
    (dict(y=ctypes.c_void_p(0x1001), y_type=2), MISALIGNED), (dict(M=0, w=None, y=None, ws=None), OK),
    (dict(N=0, w=None, y=None, ws=None), OK)])
def test_matmul_arguments(L, change, status):
    assert call(L.load().w8a8_matmul, MATMUL, **change) == status


@pytest.mark.parametrize("change,status", SHAPES + [
    (dict(w=None), INVALID), (dict(s_w=None), INVALID), (dict(x=None), INVALID), (dict(sx=None), INVALID),
    (dict(y=None), INVALID), (dict(ws=None), INVALID), (dict(x_type=3), INVALID), (dict(y_type=7), INVALID),
    (dict(flags=2), INVALID), (dict(ws_bytes=0), SHAPE), (dict(w=ODD), MISALIGNED), (dict(x=ODD), MISALIGNED),
    (dict(qx=ODD), MISALIGNED), (dict(ws=ODD), MISALIGNED), (dict(sx=ODD2), MISALIGNED), (dict(y=ODD2), MISALIGNED),
    (dict(M=0, x=None, w=None, sx=None), OK)])
def test_linear_arguments(L, change, status):
    assert call(L.load().w8a8_linear, LINEAR, **change) == status


@pytest.mark.parametrize("fields,status", [
    ((None, 0.0, 1, None), SHAPE), ((None, 0.0, 2, None), SHAPE), ((None, 0.0, 3, None), INVALID), ((None, 0.0, -1, None), INVALID),
    ((0x1000, 0.0, 0, None), INVALID), ((0x1000, -1.0, 0, None), INVALID), ((0x1000, float("inf"), 0, None), INVALID),
    ((0x1000, float("nan"), 0, None), INVALID), ((0x1004, 1e-6, 0, None), MISALIGNED), ((None, 0.0, 0, 0x1002), MISALIGNED)])
def test_linear_fused_operators(L, fields, status):
    f = L.Fusion(*fields)
    assert call(L.load().w8a8_linear, LINEAR, f=by(f)) == status


def test_linear_workspace_sizes(L):
    n = L.w8a8_workspace_bytes
    assert n(0, 8, 64) == 0 and n(1, 8, 48) == 0 and n(-1, 8, 64) == 0 and n(1, 8, 131072 + 32) == 0
    assert n((1 << 20) + 1, 8, 64) == 0
    for M in (1, 8, 16, 17, 129, 4096, 1 << 20):
        # the codes as fp16 in tiles of a multiple of 16 tokens, at most 192 of them
        assert M * 2 * 64 <= n(M, 8, 64) <= (M + 192) * 2 * 64
        assert call(L.load().w8a8_matmul, MATMUL, M=M, ws_bytes=n(M, 8, 64) - 1) == SHAPE


ROUTE = dict(x=FAKE, x_type=0, M=1, K=64, ids=FAKE, weights=FAKE, qx=None, sx=None, flags=0, s=None)


def router(L, **change):
    base = dict(norm_weight=None, norm_eps=0.0, w=0x1000, select_bias=None, E=8, top_k=2, score=0, renormalize=1, scale=1.0)
    assert set(change) <= set(base)
    return L.Router(*{**base, **change}.values())


@pytest.mark.parametrize("change,status", [
    (dict(E=0), INVALID), (dict(E=-1), INVALID), (dict(top_k=0), INVALID), (dict(top_k=9), INVALID), (dict(score=2), INVALID),
    (dict(select_bias=0x1000), INVALID), (dict(norm_weight=0x1000), INVALID), (dict(norm_weight=0x1000, norm_eps=float("inf")), INVALID),
    (dict(E=1025), SHAPE), (dict(E=64, top_k=17), SHAPE), (dict(w=None), INVALID), (dict(w=0x1004), MISALIGNED),
    (dict(norm_weight=0x1004, norm_eps=1e-6), MISALIGNED), (dict(score=1, select_bias=0x1002), MISALIGNED)])
def test_router_descriptors(L, change, status):
    r = router(L, **change)
    assert L.load().w4_moe_route(by(r), *ROUTE.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INVALID), (dict(M=17), SHAPE), (dict(K=0), INVALID), (dict(K=40), SHAPE), (dict(K=131072 + 32), SHAPE),
    (dict(x=None), INVALID), (dict(ids=None), INVALID), (dict(weights=None), INVALID), (dict(x_type=3), INVALID),
    (dict(flags=2), INVALID), (dict(qx=FAKE), INVALID), (dict(sx=FAKE), INVALID), (dict(x=ODD), MISALIGNED),
    (dict(ids=ODD2), MISALIGNED), (dict(weights=ODD2), MISALIGNED), (dict(qx=ODD, sx=FAKE), MISALIGNED),
    (dict(qx=FAKE, sx=ODD2), MISALIGNED), (dict(M=0, x=None, ids=None, weights=None), OK)])
def test_route_arguments(L, change, status):
    r = router(L)
    assert call(lambda *a: L.load().w4_moe_route(by(r), *a), ROUTE, **change) == status
    assert L.load().w4_moe_route(None, *ROUTE.values()) == INVALID


def experts(L, **change):
    base = dict(fmt=0, E=8, n_shared=1, H=64, I=96, glu=1, w_gu=0x1000, s_gu=0x1000, b_gu=None, w_dn=0x1000, s_dn=0x1000,
                b_dn=None)
    assert set(change) <= set(base)
    return L.Experts(*{**base, **change}.values())


DESCRIPTORS = [
    (dict(fmt=1), INVALID), (dict(fmt=4), INVALID), (dict(E=0), INVALID), (dict(n_shared=-1), INVALID), (dict(H=0), INVALID),
    (dict(I=-32), INVALID), (dict(glu=0), INVALID), (dict(glu=3), INVALID), (dict(n_shared=5), SHAPE), (dict(E=1024), SHAPE),
    (dict(H=72), SHAPE), (dict(I=100), SHAPE), (dict(H=131072 + 32), SHAPE), (dict(I=131072 + 32), SHAPE)]
EXPERTS = dict(qx=FAKE, sx=FAKE, ids=FAKE, weights=FAKE, M=2, top_k=2, residual=None, y=FAKE, y_type=0, ws=FAKE, ws_bytes=BIG,
               flags=0, s=None)
LAYER = dict(x=FAKE, x_type=0, M=2, ids=FAKE, weights=FAKE, qx=FAKE, sx=FAKE, residual=None, y=FAKE, y_type=0, ws=FAKE,
             ws_bytes=BIG, flags=0, s=None)


@pytest.mark.parametrize("change,status", DESCRIPTORS + [
    (dict(w_gu=None), INVALID), (dict(s_gu=None), INVALID), (dict(w_dn=None), INVALID), (dict(s_dn=None), INVALID),
    (dict(w_gu=0x1008), MISALIGNED), (dict(w_dn=0x1004), MISALIGNED), (dict(s_gu=0x1002), MISALIGNED),
    (dict(s_dn=0x1001), MISALIGNED), (dict(b_gu=0x1002), MISALIGNED), (dict(b_dn=0x1002), MISALIGNED)])
def test_expert_descriptors(L, change, status):
    e, r = experts(L, **change), router(L, E=change.get("E", 8), top_k=min(2, max(1, change.get("E", 8))))
    assert L.load().w4_moe_experts(by(e), *EXPERTS.values()) == status
    assert L.load().w4_moe_layer(by(r), by(e), *LAYER.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INVALID), (dict(M=17), SHAPE), (dict(top_k=0), INVALID), (dict(top_k=17), SHAPE), (dict(qx=None), INVALID),
    (dict(sx=None), INVALID), (dict(ids=None), INVALID), (dict(weights=None), INVALID), (dict(y=None), INVALID),
    (dict(ws=None), INVALID), (dict(y_type=3), INVALID), (dict(flags=4), INVALID), (dict(ws_bytes=0), SHAPE),
    (dict(qx=ODD), MISALIGNED), (dict(ws=ODD), MISALIGNED), (dict(sx=ODD2), MISALIGNED), (dict(ids=ODD2), MISALIGNED),
    (dict(weights=ODD2), MISALIGNED), (dict(residual=ODD2), MISALIGNED), (dict(y=ODD2), MISALIGNED),
    (dict(M=0, qx=None, ids=None, y=None, ws=None), OK)])
def test_experts_arguments(L, change, status):
    e = experts(L)
    assert call(lambda *a: L.load().w4_moe_experts(by(e), *a), EXPERTS, **change) == status
    assert L.load().w4_moe_experts(None, *EXPERTS.values()) == INVALID


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INVALID), (dict(M=17), SHAPE), (dict(x=None), INVALID), (dict(ids=None), INVALID), (dict(weights=None), INVALID),
    (dict(qx=None), INVALID), (dict(sx=None), INVALID), (dict(qx=None, sx=None), INVALID), (dict(y=None), INVALID),
    (dict(ws=None), INVALID), (dict(x_type=5), INVALID), (dict(y_type=3), INVALID), (dict(flags=2), INVALID),
    (dict(ws_bytes=64), SHAPE), (dict(x=ODD), MISALIGNED), (dict(qx=ODD), MISALIGNED), (dict(ws=ODD), MISALIGNED),
    (dict(residual=ODD2), MISALIGNED), (dict(M=0, x=None, y=None, ws=None), OK)])
def test_layer_arguments(L, change, status):
    r, e = router(L), experts(L)
    assert call(lambda *a: L.load().w4_moe_layer(by(r), by(e), *a), LAYER, **change) == status
    assert L.load().w4_moe_layer(None, by(e), *LAYER.values()) == INVALID
    assert L.load().w4_moe_layer(by(r), None, *LAYER.values()) == INVALID
    other = router(L, E=7)
    assert L.load().w4_moe_layer(by(other), by(e), *LAYER.values()) == INVALID      # not these experts' router


def test_experts_workspace_sizes(L):
    e = experts(L)
    n = L.w4_moe_workspace_bytes
    assert n(e, 0, 2) == 0 and n(e, 17, 2) == 0 and n(e, 1, 0) == 0 and n(experts(L, H=72), 1, 2) == 0
    assert L.load().w4_moe_workspace_bytes(None, 1, 2) == 0
    # at least h (fp32), its codes and the slots' outputs of every pair
    for M in (1, 16):
        assert n(e, M, 2) >= M * 3 * (96 * 4 + 96 + 64 * 4)
        assert call(lambda *a: L.load().w4_moe_experts(by(e), *a), EXPERTS, M=M, ws_bytes=n(e, M, 2) - 1) == SHAPE
    # past 32 bits: 16 tokens, 20 slots, the largest sizes
    large = experts(L, n_shared=4, H=131072, I=131072)
    assert n(large, 16, 16) >= 16 * 20 * (131072 * 4 + 131072 + 131072 * 4)


def test_paired_int8_layout_arguments(L):
    lib = L.load()
    assert lib.w8_glu_repacked_bytes(3, 64) == 8 * 64 and lib.w8_glu_repacked_bytes(8, 64) == 16 * 64
    assert lib.w8_glu_repacked_bytes(8, 48) == 0 and lib.w8_glu_repacked_bytes(-1, 64) == 0
    assert lib.w8_repack_glu(FAKE, None, 8, 64, FAKE, 1 << 20, None) == INVALID
    assert lib.w8_repack_glu(FAKE, FAKE, 8, 64, FAKE, 16, None) == SHAPE
    assert lib.w8_repack_glu(FAKE, FAKE, 8, 64, ODD, 1 << 20, None) == MISALIGNED
    assert lib.w8_repack_glu(FAKE, FAKE, 0, 64, None, 0, None) == OK


def test_host_tensors_and_names_are_refused(L):
    from bit_quantized_decode_gb300 import MoeLayer, MoeRouter, QuantLinear
    w, x = torch.zeros((8, 64)), torch.zeros((1, 64))
    with pytest.raises(ValueError, match="CUDA device"):
        MoeRouter(w, 2)
    with pytest.raises(ValueError, match="score"):
        MoeRouter(w, 2, score="relu")
    with pytest.raises(ValueError, match="CUDA device"):
        L.w8a8_linear(torch.zeros(512, dtype=torch.uint8), torch.zeros(8), None, x, torch.zeros((1, 8)), None, torch.zeros(1),
                      torch.zeros(1 << 12, dtype=torch.uint8))
    q = QuantLinear("w8", 8, 64, torch.zeros(512, dtype=torch.uint8), torch.zeros(8), None, None)
    with pytest.raises(ValueError, match="columns"):
        q(torch.zeros((1, 32)))
    with pytest.raises(ValueError, match="glu"):
        q(x, glu=L.W4_GLU_SILU)

    class R:
        E, K = 2, 64
    codes = [torch.zeros((64, 8), dtype=torch.int32)] * 2, [torch.zeros((64, 4), dtype=torch.int32)] * 2
    s = torch.zeros((2, 64)), torch.zeros((2, 64))
    for fmt, act, n in (("q4_0", "silu", 0), ("w4", "relu", 0), ("w4", "silu", 1)):
        with pytest.raises(ValueError):
            MoeLayer.from_canonical(fmt, R, codes[0], s[0], codes[1], s[1], act, n)
    with pytest.raises(ValueError):
        MoeLayer.from_float("q4_0", R, [], [])
    with pytest.raises(ValueError):
        L.moe_experts("w5", None, None, None, None, 2, 0, 64, 32, 1)
