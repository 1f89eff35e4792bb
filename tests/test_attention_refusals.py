"""What the attention refuses, it refuses before the cache is written; arguments at the ends of their ranges.  No GPU."""
import ctypes
import types

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from bit_quantized_decode_gb300 import _lib, build
    build.build()
    _lib.load()
    return _lib


@pytest.fixture
def calls(L, monkeypatch):
    """The entry points that ran, on host tensors that pass for the GPU's."""
    ran, real = [], L.load()
    fake = types.SimpleNamespace(**{n: (lambda *a, n=n: ran.append(n) or 0) for n in ("w4_kv_append", "w4_tree_attention")},
                                 w4_tree_attention_workspace_bytes=real.w4_tree_attention_workspace_bytes)
    monkeypatch.setattr(L, "load", lambda: fake)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(L, "_raw_stream", lambda stream, device: 0)
    return ran


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def test_a_refused_attention_leaves_the_cache(L, calls):
    import bit_quantized_decode_gb300 as bq
    k = torch.zeros((40, 2, 16, 64), dtype=torch.float16)
    cache = bq.KVCache(k, k.clone())
    att, T = bq.CachedAttention(cache, 4), 3
    batch, prompt = (bq.KVBatch(i32(1, 30), i32(1), i32(2), max_tokens=n) for n in (T, 65))
    qkv = torch.zeros((T, 8 * 64))
    b = att.buffers(T, batch)
    att(qkv, batch, buffers=b)
    assert calls == ["w4_kv_append", "w4_tree_attention"]
    calls.clear()
    change = lambda **f: type(b)(**{**b.__dict__, **f})                         # noqa: E731
    odd = torch.zeros(b.workspace.numel() + 8, dtype=torch.uint8)
    at = 4 if odd.data_ptr() % 16 == 0 else 0
    for call in (lambda: att(qkv, prompt), lambda: att(qkv, prompt, buffers=b),
                 lambda: att(qkv, batch, buffers=change(workspace=b.workspace[:-1])),
                 lambda: att(qkv, batch, buffers=change(workspace=odd[at: at + b.workspace.numel()])),
                 lambda: att(qkv, batch, buffers=change(y=b.y[:2])), lambda: att(qkv, batch, buffers=change(y=b.y.double())),
                 lambda: att(qkv, batch, buffers=change(q=b.q.to(torch.bfloat16))),
                 lambda: att(qkv, batch, mask=torch.zeros(T, dtype=torch.int32), buffers=b),
                 lambda: att(qkv, batch, mask=torch.zeros(T - 1, dtype=torch.int64), buffers=b),
                 lambda: bq.CachedAttention(cache, 4, scale=-1.0)(qkv, batch, buffers=b),
                 lambda: bq.CachedAttention(cache, 4, scale=float("nan"))(qkv, batch, buffers=b)):
        with pytest.raises((ValueError, L.W4Error)):
            call()
        assert calls == []


def test_a_workspace_for_a_refused_call_is_an_error(L, calls):
    import bit_quantized_decode_gb300 as bq
    k = torch.zeros((40, 2, 16, 64), dtype=torch.float16)
    att = bq.CachedAttention(bq.KVCache(k, k.clone()), 4)
    batch = lambda B=1, n=4: bq.KVBatch(i32(B, 30), i32(B), i32(B + 1), max_tokens=n)          # noqa: E731
    assert att.workspace(4, batch()).numel() > 0
    assert att.workspace(0, batch()).numel() == 0 and att.workspace(4, batch(0)).numel() == 0   # empty calls
    for T, b in ((100, batch(n=65)), (-1, batch()), ((1 << 20) + 1, batch()), (4, batch(1025))):
        with pytest.raises(L.W4Error):
            att.workspace(T, b)
        with pytest.raises((L.W4Error, RuntimeError)):
            att.buffers(T, b)


def test_histories_that_32_bits_do_not_count_are_refused(L):
    u = L.LogitRulesDesc(V=100, S=1, ids=0x1000, cap=(1 << 28) + 1, length=0x1000)
    call = lambda: L.load().w4_logits_adjust(ctypes.byref(u), 0x1000, 0, 100, 1, None, None, None, None, 0x1000, 100, 0, None)  # noqa: E731
    assert call() == L.W4_UNSUPPORTED_SHAPE
    u.cap, u.length = 1 << 28, 0x1002            # the longest: refused for its misaligned lengths, only
    assert call() == L.W4_MISALIGNED


def test_scales_that_pass_fp32_times_log2_e_are_refused(L):
    c = L.KVCacheDesc(k=0x1000, v=0x1000, type=2, pages=10, page_size=16, Hkv=2, D=64)
    b = L.KVBatchDesc(table=0x1000, ctx=0x1000, q_start=0x1000, B=2, max_pages=4, max_tokens=4)
    f = lambda scale, y: L.load().w4_tree_attention(ctypes.byref(c), ctypes.byref(b), 0x1000, 2, 3, 4, None, scale, y, 0, 0x1000,  # noqa: E731
                                                    1 << 40, 0, None)
    assert f(2.5e38, 0x1000) == L.W4_INVALID_ARG and f(1.9e38, 0x1004) == L.W4_MISALIGNED


@pytest.mark.parametrize("scaling", [{}, {"trained": 0}, {"trained": float("nan")}, {"trained": 4096, "slow": 32.0}, {"trained": 4096, "slow": -1.0},
                                     {"trained": 4096, "fast": 0.5}])
def test_scaling_by_parts_that_says_too_little(scaling):
    from bit_quantized_decode_gb300 import RopeTable
    with pytest.raises(ValueError):
        RopeTable.frequencies(64, 1e4, {"kind": "by_parts", "factor": 4.0, **scaling})
