"""The cache append, the tree attention and the logit rules as programs use them: captured and replayed with lengths that move
on the device, on given streams, with shared workspaces, on caches past 32-bit offsets, over long contexts, again and again."""
import random

import pytest
import torch

import attention_reference as ref
from helpers import cuda_ok
from test_gpu_attention import BF16, F16, F32, I8, check_attention, make_cache, on_gpu, units

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module")
def bq():
    import bit_quantized_decode_gb300 as pkg
    pkg._lib.load()
    pkg._lib.clear_device_error()
    yield pkg
    assert pkg._lib.device_error() == 0


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


# ------------------------------------ the tensor-core kernel's own ways (more than 16 rows to a key head)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("Hq,dtype", [(8, BF16), (20, BF16), (20, F16), (80, F16), (20, I8)])
def test_hidden_infinities_in_tiles_of_many_rows(bq, Hq, dtype, bad):
    """As for few rows: drafts of other paths, places behind the last; drafts on both sides of a tile's border."""
    D, Hkv, page, n = 128, 2, 32, 8
    for ctx in (0, 3, 60, 200):
        lay = ref.Paged(5, [n], [ctx], page)
        tensors, k64, v64 = make_cache(lay, Hkv, D, dtype, 5)
        for p in [ctx + 1, ctx + 5] + list(range(ctx + n, len(lay.table[0]) * page)):
            pg, off = lay.table[0][p // page], p % page
            if dtype == I8:
                tensors[2][pg, :, off], tensors[3][pg, :, off] = bad, bad
            else:
                tensors[0][pg, :, off], tensors[1][pg, :, off] = bad, bad
        masks = [0b00000001, 0b00000011, 0b00000101, 0b00001101, 0, 0b00100000, 0b01000101, 0b10000000]
        q = torch.randn((n, Hq, D), generator=torch.Generator().manual_seed(1)).to(F16 if dtype == F16 else BF16)
        cache, batch = on_gpu(bq, lay, tensors)
        y = bq.CachedAttention(cache, Hq).attend(q.cuda(), batch, ref.as_int64(masks).cuda(), torch.empty((n, Hq, D), device="cuda")).cpu()
        want, bound = ref.attend(lay, q.double(), k64, v64, masks, D ** -0.5, *units(dtype, F32), rounded_scales=dtype == I8)
        for t in (0, 2, 3, 4, 6, 7):
            assert bool(((y[t].double() - want[t]).abs() <= bound[t] + 1e-30).all()), (ctx, t)
        assert not bool(torch.isfinite(y[1]).any()) and not bool(torch.isfinite(y[5]).any())
        if ctx == 0:
            assert bool((y[4] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, I8])
def test_missing_pages_in_tiles_of_many_rows(bq, dtype):
    D, Hq, Hkv, page, n, ctx = 64, 16, 2, 16, 5, 150
    lay = ref.Paged(1, [n], [ctx], page)
    tensors, k64, v64 = make_cache(lay, Hkv, D, dtype, 1)
    q = torch.randn((n, Hq, D), generator=torch.Generator().manual_seed(1)).to(BF16)
    table, c, s = lay.tensors()
    for lost in ([1], [0, 1, 2, 3], [5, 7]):
        t = table.clone()
        for k, p in enumerate(lost):
            t[0, p] = (-1, lay.pages, 2 ** 31 - 1, -2 ** 31)[k]
        cache = bq.KVCache(*[None if x is None else x.cuda() for x in tensors])
        y = bq.CachedAttention(cache, Hq).attend(q.cuda(), bq.KVBatch(t.cuda(), c.cuda(), s.cuda(), n),
                                                 y=torch.empty((n, Hq, D), device="cuda")).cpu()
        for i in range(n):
            keep = [p for p in range(ctx + i + 1) if p // page not in lost]
            K, V = (lay.gather(x, 0, ctx + n)[:, keep] for x in (k64, v64))
            w = torch.softmax(torch.einsum("hgd,hld->hgl", q[i].double().view(Hkv, -1, D), K) * D ** -0.5, -1)
            want = torch.einsum("hgl,hld->hgd", w, V).reshape(Hq, D)
            # (three bf16 parts and fp32 sums of numbers up to some units: far below 2^-13)
            assert float((y[i].double() - want).abs().max()) <= 2.0 ** -13


def test_arrays_beyond_their_ranges_with_many_rows(bq):
    lay = ref.Paged(3, [1, 1], [20, 20], 16)
    tensors, _, _ = make_cache(lay, 2, 128, BF16, 3)
    cache = bq.KVCache(tensors[0].cuda(), tensors[1].cuda())
    table, _, _ = lay.tensors()
    q = torch.randn((2, 64, 128), generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    att = bq.CachedAttention(cache, 64)
    for ctxs, starts in (([-5, 1 << 30], [0, 1, 2]), ([20, 20], [0, 1, 100]), ([20, 20], [5, 6, 7]), ([2 ** 31 - 1, 3], [0, 2, 2]),
                         ([20, 20], [0, -3, 2]), ([20, 20], [-4, 1, 2]), ([20, 20], [2, 1, 0]), ([20, 20], [0, 0, 0])):
        batch = bq.KVBatch(table.cuda(), i32(ctxs), i32(starts), 2)
        y = torch.full((4, 64, 128), 3.0, device="cuda")
        att.attend(q, batch, y=y[1:3])
        assert bool((y[0] == 3.0).all()) and bool((y[3] == 3.0).all())
    assert bool((y == 3.0).all())                               # (the last: no rows at all)
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows_per_token", [1, 2, 4, 14, 16, 33, 64])
@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, I8), (256, F16)])
def test_groups_of_every_size(bq, rows_per_token, D, dtype):
    """Tiles of rows that end inside a token's heads, one to five tiles to a key head."""
    n = 9
    masks = ref.tree(random.Random(2), n)[0]
    check_attention(bq, 12, [n, 1], [140, 70], 64, rows_per_token, 1, D, dtype, F32, masks + [1])


def test_scores_that_grow_along_the_context(bq):
    """Keys that grow with their place: the running maximum is raised again and again, by more than the lazy margin."""
    for dtype, Hq in ((BF16, 14), (F16, 14), (BF16, 64)):
        lay = ref.Paged(4, [2], [1500], 32)
        (k, v, _, _), _, _ = make_cache(lay, 2, 64, dtype, 4)
        for p in range(1502):
            k[lay.table[0][p // 32], :, p % 32] *= 0.02 * p ** 1.0 / 4
        q = torch.randn((2, Hq, 64), generator=torch.Generator().manual_seed(2)).to(dtype)
        cache, batch = on_gpu(bq, lay, (k, v, None, None))
        y = bq.CachedAttention(cache, Hq).attend(q.cuda(), batch, y=torch.empty((2, Hq, 64), device="cuda")).cpu()
        want, bound = ref.attend(lay, q.double(), k.double(), v.double(), [1, 3], 0.125, *units(dtype, F32))
        assert bool(((y.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("n,Hq,Hkv,D,dtype", [(1, 28, 4, 128, BF16), (16, 28, 4, 128, BF16), (5, 8, 1, 256, I8), (2, 4, 2, 64, F16)])
def test_long_contexts(bq, n, Hq, Hkv, D, dtype):
    masks = ref.tree(random.Random(1), n)[0]
    check_attention(bq, 5, [n], [131071], 64, Hq, Hkv, D, dtype, F32, masks)


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, F16), (128, I8), (256, BF16)])
def test_long_sums_keep_their_precision(bq, D, dtype):
    """Some hundred tiles to a block, fp32 outputs, against 64 bits on the GPU: what the tensor cores cut from a sum at each
    step (2^-23 at most, 12 steps a tile) must not add up over more than the 16 tiles after which sums are taken out."""
    Hkv, Hq, n, page = 16, 256, 2, 64
    ctx = 60000 * 64 // D
    lay = ref.Paged(3, [n], [ctx], page)
    shape = (lay.pages, Hkv, page, D)
    g = torch.Generator(device="cuda").manual_seed(3)
    if dtype == I8:
        k, v = (torch.randint(-127, 128, shape, generator=g, dtype=torch.int8, device="cuda") for _ in range(2))
        ks, vs = (torch.full(shape[:3], s, device="cuda") for s in (0.004, 0.03))
    else:
        k, v = ((s * torch.randn(shape, generator=g, device="cuda")).to(dtype) for s in (0.3, 1.0))
        ks = vs = None
    v = v.abs() if dtype != I8 else v.abs().clamp(max=127)      # all of one sign: sums that only grow
    q = torch.randn((n, Hq, D), generator=g, device="cuda").to(F16 if dtype == F16 else BF16)
    cache = bq.KVCache(k, v, ks, vs)
    batch = bq.KVBatch(*[t.cuda() for t in lay.tensors()], max_tokens=n)
    y = bq.CachedAttention(cache, Hq).attend(q, batch, y=torch.empty((n, Hq, D), device="cuda"))
    table = torch.tensor(lay.table[0], device="cuda")
    want = torch.empty((n, Hq, D), dtype=torch.float64, device="cuda")
    for h in range(Hkv):
        K, V = (t[table, h].reshape(-1, D).double()[: ctx + n] for t in (k, v))
        if dtype == I8:
            K, V = K * ks[0, 0, 0].double(), V * vs[0, 0, 0].double()
        for i in range(n):
            s = (q[i, 16 * h: 16 * h + 16].double() @ K[: ctx + i + 1].T) * D ** -0.5
            want[i, 16 * h: 16 * h + 16] = torch.softmax(s, -1) @ V[: ctx + i + 1]
    off = float((y.double() - want).norm() / want.norm())
    # 16 tiles of 12 steps; scores and exponentials (2^-19 in all at these sizes); the parts of a probability (2^-17)
    assert off <= 192 * 2.0 ** -24 + 2.0 ** -19 + 2.0 ** -17, off


# ----------------------------------------------------------------- 32 bits
@pytest.mark.parametrize("dtype,pages", [(I8, 70000), (BF16, 36000)])
def test_caches_past_32_bit_offsets(bq, dtype, pages):
    """Pages at the far end of a cache of more than 2^32 bytes (2^31 elements and more) give what they give in a small one."""
    D, Hkv, page, n = 256, 1, 256, 3
    lay = ref.Paged(2, [n, n], [700, 200], page)
    tensors, _, _ = make_cache(lay, Hkv, D, dtype, 2)
    big = bq.KVCache.empty(pages, page, Hkv, D, dtype)
    small = bq.KVCache(*[None if t is None else t.cuda() for t in tensors])
    at = pages - lay.pages
    for a, b in ((big.k, small.k), (big.v, small.v), (big.k_scale, small.k_scale), (big.v_scale, small.v_scale)):
        if a is not None:
            a[at:] = b
    assert big.k.numel() * big.k.element_size() > 2 ** 32
    table, ctx, q_start = lay.tensors()
    far = torch.where(table >= 0, table + at, table)
    g = torch.Generator().manual_seed(4)
    for Hq in (4, 16):
        qkv = torch.randn((2 * n, (Hq + 2) * D), generator=g).cuda()
        ys = []
        for cache, t in ((small, table), (big, far)):
            att = bq.CachedAttention(cache, Hq, rope=bq.RopeTable.build(1000, 128))
            batch = bq.KVBatch(t.cuda(), ctx.cuda(), q_start.cuda(), n)
            ys.append(att(qkv, batch))
        assert torch.equal(*ys)
        assert torch.equal(big.k[at:], small.k) and torch.equal(big.v[at:], small.v)
    del big
    torch.cuda.empty_cache()


# ------------------------------------------------------- streams and graphs
@pytest.mark.parametrize("Hq", [8, 40])
def test_captured_steps_follow_the_lengths_on_the_device(bq, Hq):
    """A captured step, replayed while contexts, pages and inputs change in place, gives what an eager step gives; two graphs
    share one workspace."""
    Hkv, D, page, B, n = 2, 128, 16, 3, 2
    g = torch.Generator().manual_seed(1)
    caches = [bq.KVCache.empty(64, page, Hkv, D, BF16) for _ in range(3)]
    rope = bq.RopeTable.build(256, D)
    table = i32([list(range(16 * b, 16 * b + 16)) for b in range(B)])
    ctx, q_start = i32([0] * B), i32([n * b for b in range(B + 1)])
    batch = bq.KVBatch(table, ctx, q_start, n)
    qkv, mask = torch.zeros((n * B, (Hq + 2 * Hkv) * D), device="cuda"), ref.as_int64([1, 3] * B).cuda()
    atts = [bq.CachedAttention(c, Hq, rope=rope) for c in caches]
    shared = atts[0].buffers(n * B, batch)
    outs, graphs = [], []
    for att in atts[:2]:
        b = type(shared)(torch.empty_like(shared.q), torch.empty_like(shared.y), shared.workspace)
        att(qkv, batch, None, mask, b)                          # (sets kernels up before the capture)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            att(qkv, batch, None, mask, b)
        graphs.append(graph)
        outs.append(b.y)
    for c in caches:
        c.k.zero_()
        c.v.zero_()
    for step in range(30):
        qkv.copy_(torch.randn(qkv.shape, generator=g))
        for graph in graphs:
            graph.replay()
        y = atts[2](qkv, batch, None, mask)
        assert torch.equal(outs[0], y) and torch.equal(outs[1], y), step
        assert torch.equal(caches[0].k, caches[2].k) and torch.equal(caches[1].v, caches[2].v)
        ctx += i32([1, 2, step % 3])


@pytest.mark.parametrize("Hq", [8, 40])
def test_calls_on_a_given_stream_make_their_own_tensors(bq, Hq):
    D, Hkv = 128, 2
    lay = ref.Paged(1, [4, 2], [900, 3], 16)
    tensors, _, _ = make_cache(lay, Hkv, D, BF16, 1)
    cache, batch = on_gpu(bq, lay, tensors)
    att = bq.CachedAttention(cache, Hq)
    qkvs = [torch.randn((6, (Hq + 2 * Hkv) * D), generator=torch.Generator().manual_seed(s)).cuda() for s in range(3)]
    x = torch.randn((2, 9000), device="cuda")
    rules = bq.LogitRules(9000, i32([[1, 2, 2, 3], [7, 7, 7, 7]]), i32([4, 4]), frequency=torch.ones(2, device="cuda"))
    lw = rules(x).clone()
    want = [att(q, batch).clone() for q in qkvs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for i in range(12):
        got.append((att(qkvs[i % 3], batch, stream=side), rules(x, stream=side)))
        torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")             # reuses what the current stream freed
    torch.cuda.synchronize()
    for i, (y, l) in enumerate(got):
        assert torch.equal(y, want[i % 3]) and torch.equal(l, lw)


def test_two_streams_at_once_and_many_repetitions(bq):
    """Calls of both kernels on two streams, each with its own workspace, thousands of times: always the same bits."""
    runs = []
    for seed, (ns, ctxs, Hq, Hkv, D, dtype) in enumerate([([1], [3000], 28, 4, 128, BF16), ([16], [1111], 28, 4, 128, BF16),
                                                          ([1] * 40, [100 + 37 * b for b in range(40)], 8, 2, 64, F16),
                                                          ([5, 9], [2000, 70], 8, 1, 256, I8), ([64, 3], [100, 800], 14, 2, 128, I8)]):
        lay = ref.Paged(seed, ns, ctxs, 16)
        tensors, _, _ = make_cache(lay, Hkv, D, dtype, seed)
        cache, batch = on_gpu(bq, lay, tensors)
        att = bq.CachedAttention(cache, Hq)
        q = torch.randn((lay.T, Hq, D), generator=torch.Generator().manual_seed(seed)).to(att.q_dtype).cuda()
        m = ref.as_int64([m for n in ns for m in ref.tree(random.Random(seed), n)[0]]).cuda()
        y = [torch.empty((lay.T, Hq, D), device="cuda") for _ in range(2)]
        runs.append((att, q, batch, m, y, [att.workspace(lay.T, batch) for _ in range(2)], att.attend(q, batch, m, torch.empty_like(y[0])).clone()))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for rep in range(60):
        for k in range(10):
            for j, s in enumerate(streams):
                att, q, batch, m, y, ws, _ = runs[(k + j + rep) % len(runs)]
                att.attend(q, batch, m, y[j], ws[j], stream=s)
        torch.cuda.synchronize()
        for _, _, _, _, y, _, want in runs:
            assert torch.equal(y[0], want) and torch.equal(y[1], want), rep
    assert bq._lib.device_error() == 0


def test_consecutive_calls_share_a_workspace(bq):
    """Calls of different shapes behind each other on one workspace: each result is that of a call by itself."""
    todo = []
    for seed, (n, ctx, Hq) in enumerate([(1, 2000, 8), (16, 500, 8), (1, 30, 8), (5, 1800, 16), (64, 100, 8), (2, 1000, 2)]):
        lay = ref.Paged(seed, [n, n], [ctx, ctx // 2], 16)
        tensors, _, _ = make_cache(lay, 2, 128, F16, seed)
        cache, batch = on_gpu(bq, lay, tensors)
        att = bq.CachedAttention(cache, Hq)
        q = torch.randn((lay.T, Hq, 128), generator=torch.Generator().manual_seed(seed)).to(F16).cuda()
        todo.append((att, q, batch, att.attend(q, batch).clone()))
    ws = torch.empty(max(t[0].workspace(t[1].shape[0], t[2]).numel() for t in todo), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(40):
        ys = [att.attend(q, batch, None, torch.empty_like(q), ws) for att, q, batch, _ in todo]
        for y, t in zip(ys, todo):
            assert torch.equal(y, t[3])


def test_captured_logit_rules_follow_the_history(bq):
    V, S, cap = 5000, 2, 16
    ids, length = torch.zeros((S, cap), dtype=torch.int32, device="cuda"), i32([0, 0])
    rules = bq.LogitRules(V, ids, length, frequency=torch.ones(S, device="cuda"))
    x, out = torch.zeros((S, V), device="cuda"), torch.empty((S, V), device="cuda")
    rules(x, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rules(x, out)
    made = [[], []]
    for step in range(cap):
        for s in range(S):
            t = (step * (s + 3)) % 5
            ids[s, step] = t
            made[s].append(t)
        length += 1
        graph.replay()
        want = torch.zeros((S, V))
        for s in range(S):
            for t in made[s]:
                want[s, t] -= 1
        assert torch.equal(out.cpu(), want)


def test_an_int8_cache_as_numbers(bq):
    for D in (64, 128, 256):
        lay = ref.Paged(1, [3], [40], 32)
        t, k64, v64 = make_cache(lay, 3, D, I8, D)
        cache = bq.KVCache(*[x.cuda() for x in t])
        assert torch.equal(cache.values("k").cpu(), t[0].float() * t[2][..., None])
        assert torch.equal(cache.values("v", torch.empty(t[1].shape, device="cuda")).cpu(), t[1].float() * t[3][..., None])
    c = bq.KVCache.empty(2, 16, 1, 64, F16)
    assert c.values("k") is c.k and c.values("v") is c.v


# ------------------------------------------------------------- logits, more
def test_more_different_tokens_than_a_table_holds(bq):
    """Every id of a vocabulary of 150000 in one history, three times: the tokens are taken in parts."""
    V = 150000
    g = torch.Generator().manual_seed(1)
    ids = torch.cat([torch.randperm(V, generator=g) for _ in range(3)]).int()[None].contiguous()
    x = torch.randn((1, V), generator=g)
    rules = bq.LogitRules(V, ids.cuda(), i32([3 * V]), i32([V]), frequency=torch.full((1,), 0.25, device="cuda"))
    assert torch.equal(rules(x.cuda()).cpu(), x - 0.25 * 2)
    # and ids that all share their hash's lower bits
    some = torch.arange(0, 1 << 24, 1 << 9, dtype=torch.int32)[None]
    x = torch.zeros((1, 1 << 24))
    rules = bq.LogitRules(1 << 24, some.cuda(), i32([some.numel()]), presence=torch.ones(1, device="cuda"))
    y = rules(x.cuda()).cpu()
    assert float(y.sum()) == -some.numel() and bool((y[0, some[0].long()] == -1).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V,wide,shift", [(1000, 0, 1), (1001, 0, 0), (1001, 2, 3), (37, 0, 5), (3, 0, 1), (8195, 5, 2)])
def test_rows_at_every_alignment(bq, V, wide, shift, dtype):
    """Rows that begin anywhere in a 16-byte word, outputs that begin elsewhere."""
    S = 5
    for oshift in (shift, shift + 1):
        store = torch.randn(S * (V + wide) + 16).to(dtype)
        x = store[shift: shift + S * (V + wide)].view(S, V + wide)[:, :V]
        gx = store.cuda()[shift: shift + S * (V + wide)].view(S, V + wide)[:, :V]
        go = torch.zeros(S * (V + wide) + 16, dtype=dtype, device="cuda")
        out = go[oshift: oshift + S * (V + wide)].view(S, V + wide)[:, :V]
        ok = torch.rand((S, V), generator=torch.Generator().manual_seed(V)) < 0.6
        bits = torch.zeros((S, (V + 31) // 32 * 32), dtype=torch.int64)
        bits[:, :V] = ok
        words = (bits.view(S, -1, 32) << torch.arange(32)).sum(-1)
        words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
        bq.LogitRules(V, sequences=S)(gx, out, allowed=words.cuda())
        assert torch.equal(out.cpu(), torch.where(ok, x, torch.full_like(x, float("-inf"))))
        go[oshift: oshift + S * (V + wide)].view(S, V + wide)[:, :V] = 0
        assert not bool(go.any())                               # nothing beside the rows
