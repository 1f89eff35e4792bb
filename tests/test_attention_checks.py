"""Host-side refusals of the cache append, the tree attention and the logit rules: every bad argument comes back as a status
(C ABI) or a ValueError (tensors) before any launch, and empty calls succeed.  No GPU."""
import ctypes

import pytest
import torch

FAKE = ctypes.c_void_p(0x1000)       # 16-byte aligned, never dereferenced
ODD = ctypes.c_void_p(0x1004)        # 4-byte but not 16-byte aligned
ODD2 = ctypes.c_void_p(0x1002)       # 2-byte aligned
OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3
BIG = 1 << 40
by = ctypes.byref


@pytest.fixture(scope="module")
def L():
    from bit_quantized_decode_gb300 import _lib, build
    build.build()
    _lib.load()
    return _lib


def cache(L, **change):
    return L.KVCacheDesc(**{**dict(k=0x1000, v=0x1000, k_scale=None, v_scale=None, type=2, pages=10, page_size=16, Hkv=2, D=64), **change})


def batch(L, **change):
    return L.KVBatchDesc(**{**dict(table=0x1000, ctx=0x1000, q_start=0x1000, B=2, max_pages=4, max_tokens=4), **change})


def rope(L, **change):
    return L.RopeDesc(**{**dict(turns=0x1000, positions=100, rot=64, layout=0), **change})


APPEND = dict(qkv=FAKE, x_type=0, ld=512, T=3, Hq=4, positions=None, q_norm=None, k_norm=None, eps=1e-6, q=FAKE, q_type=2, flags=0,
              s=None)
ATTEND = dict(q=FAKE, q_type=2, T=3, Hq=4, mask=None, scale=0.125, y=FAKE, y_type=0, ws=FAKE, ws_bytes=BIG, flags=0, s=None)
INT8 = dict(type=3, k_scale=0x1000, v_scale=0x1000)
# (fields of the cache, of the batch, status): both calls refuse them
CALLS = [(dict(type=0), {}, INVALID), (dict(type=4), {}, INVALID), (dict(pages=0), {}, INVALID), (dict(Hkv=0), {}, INVALID),
         (dict(D=0), {}, INVALID), (dict(D=96), {}, SHAPE), (dict(D=512), {}, SHAPE), (dict(page_size=0), {}, INVALID),
         (dict(page_size=8), {}, SHAPE), (dict(page_size=48), {}, SHAPE), (dict(page_size=512), {}, SHAPE),
         (dict(pages=1 << 30, Hkv=2), {}, SHAPE), (dict(k=None), {}, INVALID), (dict(v=None), {}, INVALID),
         (dict(k_scale=0x1000), {}, INVALID), (dict(type=3), {}, INVALID), (dict(type=3, k_scale=0x1000), {}, INVALID),
         (dict(k=0x1008), {}, MISALIGNED), (dict(v=0x1004), {}, MISALIGNED), ({**INT8, "k_scale": 0x1004}, {}, MISALIGNED),
         ({}, dict(B=-1), INVALID), ({}, dict(B=1025), SHAPE), ({}, dict(max_pages=0), INVALID), ({}, dict(max_tokens=0), INVALID),
         ({}, dict(max_pages=(1 << 26) + 1), SHAPE), ({}, dict(table=None), INVALID), ({}, dict(ctx=None), INVALID),
         ({}, dict(q_start=None), INVALID), ({}, dict(table=0x1002), MISALIGNED), ({}, dict(q_start=0x1001), MISALIGNED)]


@pytest.mark.parametrize("c,b,status", CALLS)
def test_caches_and_batches(L, c, b, status):
    lib = L.load()
    assert lib.w4_kv_append(by(cache(L, **c)), by(batch(L, **b)), by(rope(L)), *APPEND.values()) == status
    assert lib.w4_tree_attention(by(cache(L, **c)), by(batch(L, **b)), *ATTEND.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(T=(1 << 20) + 1), SHAPE), (dict(Hq=0), INVALID), (dict(Hq=3, ld=512), SHAPE), (dict(Hq=2048, ld=1 << 20), SHAPE),
    (dict(x_type=3), INVALID), (dict(q_type=0), INVALID), (dict(q_type=3), INVALID), (dict(flags=2), INVALID), (dict(ld=511), INVALID),
    (dict(ld=514), MISALIGNED), (dict(qkv=None), INVALID), (dict(q=None), INVALID), (dict(qkv=ODD), MISALIGNED), (dict(q=ODD), MISALIGNED),
    (dict(positions=ODD2), MISALIGNED), (dict(q_norm=ODD), MISALIGNED), (dict(k_norm=ODD), MISALIGNED),
    (dict(q_norm=FAKE, eps=0.0), INVALID), (dict(k_norm=FAKE, eps=float("nan")), INVALID), (dict(q_norm=FAKE, eps=float("inf")), INVALID),
    (dict(T=0, qkv=None, q=None), OK)])
def test_append_arguments(L, change, status):
    assert L.load().w4_kv_append(by(cache(L)), by(batch(L)), by(rope(L)), *{**APPEND, **change}.values()) == status


@pytest.mark.parametrize("fields,status", [
    (dict(rot=-8), INVALID), (dict(rot=12), SHAPE), (dict(rot=72), SHAPE), (dict(positions=0), INVALID), (dict(layout=2), INVALID),
    (dict(layout=-1), INVALID), (dict(turns=None), INVALID), (dict(turns=0x1008), MISALIGNED)])
def test_rotations(L, fields, status):
    assert L.load().w4_kv_append(by(cache(L)), by(batch(L)), by(rope(L, **fields)), *APPEND.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(T=(1 << 20) + 1), SHAPE), (dict(Hq=0), INVALID), (dict(Hq=5), SHAPE), (dict(Hq=2048), SHAPE),
    (dict(q_type=1), INVALID), (dict(q_type=0), INVALID), (dict(y_type=3), INVALID), (dict(y_type=-1), INVALID), (dict(flags=4), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(q=None), INVALID), (dict(y=None), INVALID), (dict(ws=None), INVALID), (dict(ws_bytes=1000), SHAPE), (dict(q=ODD), MISALIGNED),
    (dict(y=ODD), MISALIGNED), (dict(ws=ODD), MISALIGNED), (dict(mask=ODD), MISALIGNED), (dict(T=0, q=None, y=None, ws=None), OK)])
def test_attention_arguments(L, change, status):
    assert L.load().w4_tree_attention(by(cache(L)), by(batch(L)), *{**ATTEND, **change}.values()) == status


def test_attention_limits(L):
    lib = L.load()
    assert lib.w4_tree_attention(by(cache(L)), by(batch(L, max_tokens=65)), *ATTEND.values()) == SHAPE
    assert lib.w4_tree_attention(by(cache(L)), by(batch(L, B=0)), *ATTEND.values()) == OK
    assert lib.w4_tree_attention(None, by(batch(L)), *ATTEND.values()) == INVALID
    assert lib.w4_tree_attention(by(cache(L)), None, *ATTEND.values()) == INVALID
    assert lib.w4_kv_append(by(cache(L)), None, None, *APPEND.values()) == INVALID
    # an int8 cache takes queries of either 16-bit type and no others
    for t in (0, 3):
        assert lib.w4_tree_attention(by(cache(L, **INT8)), by(batch(L)), *{**ATTEND, "q_type": t}.values()) == INVALID
    # units of work are counted in 32 bits
    assert lib.w4_tree_attention(by(cache(L, Hkv=64)), by(batch(L, B=1024, max_pages=1 << 22)), *{**ATTEND, "Hq": 64}.values()) == SHAPE


def test_workspace_sizes(L):
    n = lambda c=None, b=None, T=3, Hq=4: L.w4_tree_attention_workspace_bytes(cache(L, **(c or {})), batch(L, **(b or {})), T, Hq)  # noqa: E731
    assert n(T=0) == 0 and n(Hq=3) == 0 and n(dict(D=80)) == 0 and n(b=dict(max_tokens=65)) == 0 and n(b=dict(B=0)) == 0
    assert L.load().w4_tree_attention_workspace_bytes(None, by(batch(L)), 1, 4) == 0
    # two partial results for each block: maxima, sums and rows of D; no more rows than a call has, nor than a tile
    assert n(T=1) >= 152 * 2 * 2 * (64 + 2) * 4
    assert n(T=64, Hq=64, b=dict(max_tokens=64)) >= 152 * 2 * 128 * (64 + 2) * 4
    assert n(T=64, Hq=64, b=dict(max_tokens=64)) == n(T=64, Hq=32, b=dict(max_tokens=64))
    need = n()
    assert L.load().w4_tree_attention(by(cache(L)), by(batch(L)), *{**ATTEND, "ws_bytes": need - 1}.values()) == SHAPE


def test_rope_table_and_values_arguments(L):
    lib = L.load()
    f = lib.w4_rope_table
    assert f(FAKE, 1.0, 1.0, -1, 64, FAKE, None) == INVALID and f(FAKE, 1.0, 1.0, 10, -8, FAKE, None) == INVALID
    assert f(FAKE, 0.0, 1.0, 10, 64, FAKE, None) == INVALID and f(FAKE, 1.0, float("nan"), 10, 64, FAKE, None) == INVALID
    assert f(FAKE, 1.0, 1.0, 10, 12, FAKE, None) == SHAPE and f(FAKE, 1.0, 1.0, 10, 264, FAKE, None) == SHAPE
    assert f(None, 1.0, 1.0, 10, 64, FAKE, None) == INVALID and f(FAKE, 1.0, 1.0, 10, 64, None, None) == INVALID
    assert f(ODD, 1.0, 1.0, 10, 64, FAKE, None) == MISALIGNED and f(FAKE, 1.0, 1.0, 10, 64, ODD, None) == MISALIGNED
    assert f(None, 1.0, 1.0, 0, 64, None, None) == OK
    g = lib.w4_kv_values
    assert g(None, 0, FAKE, None) == INVALID and g(by(cache(L)), 0, FAKE, None) == INVALID       # a 16-bit cache is its own values
    assert g(by(cache(L, **INT8)), 2, FAKE, None) == INVALID and g(by(cache(L, **INT8)), 0, None, None) == INVALID
    assert g(by(cache(L, **INT8)), 1, ODD, None) == MISALIGNED and g(by(cache(L, **{**INT8, "D": 100})), 1, FAKE, None) == SHAPE


RULES = dict(V=100, S=2, ids=0x1000, cap=8, length=0x1000, prompt=None, repetition=None, frequency=None, presence=None, bias_ids=None,
             bias=None, n_bias=0)
LOGITS = dict(logits=FAKE, type=0, ld=100, R=3, row_start=None, drafts=None, mask=None, allowed=None, out=FAKE, ld_out=100, flags=0,
              s=None)


@pytest.mark.parametrize("rules,change,status", [
    (dict(V=-1), {}, INVALID), (dict(S=-1), {}, INVALID), (dict(cap=-1), {}, INVALID), (dict(n_bias=-1), {}, INVALID),
    (dict(n_bias=1025, bias_ids=0x1000, bias=0x1000), {}, SHAPE), (dict(V=(1 << 24) + 1), dict(ld=1 << 25, ld_out=1 << 25), SHAPE),
    (dict(ids=None), {}, INVALID), (dict(length=None), {}, INVALID), (dict(n_bias=1), {}, INVALID),
    (dict(n_bias=1, bias_ids=0x1000), {}, INVALID), (dict(ids=0x1002), {}, MISALIGNED), (dict(prompt=0x1001), {}, MISALIGNED),
    (dict(repetition=0x1002), {}, MISALIGNED), (dict(frequency=0x1002), {}, MISALIGNED), (dict(presence=0x1002), {}, MISALIGNED),
    ({}, dict(R=-1), INVALID), ({}, dict(R=(1 << 20) + 1), SHAPE), ({}, dict(type=3), INVALID), ({}, dict(flags=2), INVALID),
    ({}, dict(ld=99), INVALID), ({}, dict(ld_out=99), INVALID), ({}, dict(drafts=FAKE), INVALID),
    ({}, dict(mask=FAKE, row_start=FAKE), INVALID), ({}, dict(logits=None), INVALID), ({}, dict(out=None), INVALID),
    ({}, dict(logits=ODD2), MISALIGNED), ({}, dict(out=ODD2), MISALIGNED), ({}, dict(type=2, out=ctypes.c_void_p(0x1001)), MISALIGNED),
    ({}, dict(row_start=ODD2), MISALIGNED), ({}, dict(allowed=ODD2), MISALIGNED), ({}, dict(ld_out=104), INVALID),
    ({}, dict(row_start=FAKE, drafts=FAKE, mask=ODD), MISALIGNED), ({}, dict(R=0, logits=None, out=None), OK),
    (dict(V=0), dict(logits=None, out=None, ld=0, ld_out=0), OK), (dict(S=0), dict(logits=None, out=None), OK)])
def test_logit_arguments(L, rules, change, status):
    u = L.LogitRulesDesc(**{**RULES, **rules})
    assert L.load().w4_logits_adjust(by(u), *{**LOGITS, **change}.values()) == status
    assert L.load().w4_logits_adjust(None, *LOGITS.values()) == INVALID


def test_host_tensors_and_names_are_refused(L, monkeypatch):
    import bit_quantized_decode_gb300 as bq
    k = torch.zeros((4, 2, 16, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA device"):
        bq.KVCache(k, k)
    with pytest.raises(ValueError, match="scales"):
        bq.KVCache(k.to(torch.int8), k.to(torch.int8))
    with pytest.raises(ValueError, match="scales"):
        bq.KVCache(k, k, torch.zeros(4, 2, 16), torch.zeros(4, 2, 16))
    with pytest.raises(ValueError, match="page_size"):
        bq.KVCache(k[0], k[0])
    with pytest.raises(ValueError, match="pages"):
        bq.KVBatch(torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), 1)
    with pytest.raises(ValueError, match="layout"):
        bq.RopeTable(torch.zeros(4, 32, 2), "spiral")
    with pytest.raises(ValueError, match="turns"):
        bq.RopeTable(torch.zeros(4, 32))
    for bad in (dict(rot=12), dict(rot=64, scaling={"kind": "magic"}), dict(rot=64, scaling={"kind": "linear", "factor": 0.5}),
                dict(rot=64, scaling={"kind": "linear", "factor": 2.0, "trained": 5})):
        with pytest.raises(ValueError):
            bq.RopeTable.frequencies(**bad)
    with pytest.raises(ValueError, match="together"):
        bq.LogitRules(10, torch.zeros((1, 4), dtype=torch.int32))
    with pytest.raises(ValueError, match="together"):
        bq.LogitRules(10, bias_ids=torch.zeros((1, 4), dtype=torch.int32))
    with pytest.raises(ValueError, match="sequences"):
        bq.LogitRules(10)
    # what the tensors of a call must be, on tensors that pass for the GPU's
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(L, "_raw_stream", lambda stream, device: 0)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)                          # noqa: E731
    with pytest.raises(ValueError, match="v: "):
        bq.KVCache(k, k[:2])
    with pytest.raises(ValueError, match="v: "):
        bq.KVCache(k, k.to(torch.bfloat16))
    with pytest.raises(ValueError, match="k: "):
        bq.KVCache(k.float(), k.float())
    with pytest.raises(ValueError, match="contiguous"):
        bq.KVCache(k.transpose(1, 2), k.transpose(1, 2))
    with pytest.raises(ValueError, match="q_start"):
        bq.KVBatch(i32(2, 4), i32(2), i32(2), 1)
    with pytest.raises(ValueError, match="ctx"):
        bq.KVBatch(i32(2, 4), i32(2).long(), i32(3), 1)
    c, b = bq.KVCache(k, k), bq.KVBatch(i32(1, 4), i32(1), i32(2), 1)
    with pytest.raises(ValueError, match="evenly"):
        bq.CachedAttention(c, 3)
    with pytest.raises(ValueError, match="queries"):
        bq.CachedAttention(c, 4, q_dtype=torch.bfloat16)
    att = bq.CachedAttention(c, 4)
    q, qkv = torch.zeros((3, 4, 64), dtype=torch.float16), torch.zeros((3, 8 * 64))
    for call in (lambda: att.append(qkv[:, :-1], b), lambda: att.append(qkv.double(), b), lambda: att.append(qkv.t(), b),
                 lambda: att.append(qkv[:1].expand(3, 512), b), lambda: att.append(qkv, b, q=q[:2]), lambda: att.append(qkv, b, i32(2)),
                 lambda: att.append(qkv, b, i32(3).long()), lambda: att.attend(q, b, i32(3)), lambda: att.attend(q.float(), b),
                 lambda: att.attend(q, b, y=torch.zeros(3, 4, 32)), lambda: att.attend(q[..., :32], b),
                 lambda: att.attend(q, b, workspace=torch.zeros(10))):
        with pytest.raises(ValueError):
            call()
    u = bq.LogitRules(64, sequences=3)
    x = torch.zeros((3, 64))
    for call in (lambda: u(x[:, :63]), lambda: u(x.double()), lambda: u(x, torch.zeros((3, 64), dtype=torch.float16)), lambda: u(x, x[:2]),
                 lambda: u(x, allowed=i32(3, 1)), lambda: u(x, row_start=i32(3)), lambda: u(x, row_start=i32(4), drafts=i32(2)),
                 lambda: u(x, row_start=i32(4), drafts=i32(3), mask=i32(3))):
        with pytest.raises(ValueError):
            call()
    for bad in (dict(ids=i32(3), length=i32(3)), dict(ids=i32(3, 4), length=i32(2)), dict(repetition=torch.zeros(3, dtype=torch.float64)),
                dict(bias_ids=i32(3, 4), bias_values=torch.zeros(3, 5))):
        with pytest.raises(ValueError):
            bq.LogitRules(64, **bad)


def test_scaled_frequencies():
    """The scaled angles per position: linear, a raised base, and by parts between the slowest and the fastest pairs."""
    import math

    from bit_quantized_decode_gb300 import RopeTable
    inv, one = RopeTable.frequencies(128, 1e6)
    assert one == 1.0 and inv.dtype == torch.float64 and float(inv[0]) == 1.0 and abs(float(inv[63]) - 1e6 ** (-126 / 128)) < 1e-18
    lin, _ = RopeTable.frequencies(128, 1e6, {"kind": "linear", "factor": 4.0})
    assert torch.allclose(lin * 4, inv, rtol=1e-15, atol=0)
    raised, _ = RopeTable.frequencies(128, 1e6, {"kind": "base", "factor": 4.0})
    assert float(raised[0]) == 1.0 and abs(float(raised[63]) * 4 / float(inv[63]) - 1) < 1e-12
    parts, scale = RopeTable.frequencies(128, 1e6, {"kind": "by_parts", "factor": 4.0, "trained": 4096})
    turns = 4096 * inv / (2 * math.pi)
    assert torch.equal(parts[turns > 32], inv[turns > 32]) and torch.allclose(parts[turns < 1] * 4, inv[turns < 1], rtol=1e-15, atol=0)
    mid = (turns > 1) & (turns < 32)
    assert bool(((parts < inv) & (parts * 4 > inv))[mid].all()) and abs(scale - (0.1 * math.log(4) + 1)) < 1e-15
    assert RopeTable.frequencies(128, 1e6, {"kind": "by_parts", "factor": 4.0, "trained": 4096, "attention": 1.0})[1] == 1.0


def test_memory_that_moved_is_checked_again(L, monkeypatch):
    """A cache, a batch or rules whose tensors got other memory behind them: the addresses of the call, checked again."""
    import types

    import bit_quantized_decode_gb300 as bq
    seen = []
    fake = types.SimpleNamespace(**{n: (lambda *a, n=n: seen.append((n, a)) or 0) for n in ("w4_kv_append", "w4_tree_attention", "w4_logits_adjust")},
                                 w4_tree_attention_workspace_bytes=L.load().w4_tree_attention_workspace_bytes)
    monkeypatch.setattr(L, "load", lambda: fake)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: getattr(t, "at", 0))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(L, "_raw_stream", lambda stream, device: 0)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)                          # noqa: E731
    k = torch.zeros((4, 2, 16, 64), dtype=torch.float16)
    c, b = bq.KVCache(k, k.clone()), bq.KVBatch(i32(1, 4), i32(1), i32(2), 1)
    att, rules = bq.CachedAttention(c, 4, rope=bq.RopeTable(torch.zeros(8, 32, 2))), bq.LogitRules(64, i32(1, 8), i32(1), repetition=torch.ones(1))
    q, ws, x = torch.zeros((1, 4, 64), dtype=torch.float16), torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros((1, 64))
    def calls():                                                                # noqa: E306
        att.append(torch.zeros(1, 8 * 64), b, q=q)
        att.attend(q, b, y=q, workspace=ws)
        rules(x, x)
    calls()
    assert [n for n, _ in seen] == ["w4_kv_append", "w4_tree_attention", "w4_logits_adjust"]
    keep = []
    for t, desc, field in ((c.k, c.desc, "k"), (c.v, c.desc, "v"), (b.desc._tensors[1], b.desc, "ctx"), (att.rope.turns, att.rope.desc, "turns"),
                           (rules.desc._tensors[0], rules.desc, "ids")):
        keep.append(t.data)
        t.data = t.data.clone()
        calls()
        assert getattr(desc, field) == t.data_ptr()
    n = len(seen)
    for t, bad in ((c.k, k[:2].clone()), (c.v, torch.zeros_like(k, dtype=torch.bfloat16)), (b.desc._tensors[0], i32(2, 4)),
                   (att.rope.turns, torch.zeros(8, 16, 2))):
        old, t.data = t.data, bad
        with pytest.raises(ValueError):
            calls()
        t.data = old
    with pytest.raises(AttributeError):
        c.k = k
    assert all(name == "w4_kv_append" for name, _ in seen[n:]) or len(seen) == n
