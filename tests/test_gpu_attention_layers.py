"""Layers of a step behind each other, every launch a programmatic dependent of the one before it: what one layer's launches leave
in shared buffers, the next one's must not see."""
import pytest
import torch

import attention_reference as ref
from helpers import cuda_ok
from test_gpu_attention import BF16, F32, I8

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("Hq,Hkv,D,n,B,dtype", [(28, 4, 128, 1, 1, BF16), (28, 4, 128, 16, 1, BF16), (8, 1, 256, 5, 2, I8), (8, 2, 64, 1, 40, BF16)])
def test_layers_that_share_queries_and_a_workspace(Hq, Hkv, D, n, B, dtype):
    """Twelve layers in one graph, no other kernel between them, replayed with new rows and longer contexts: each layer's output
    and cache are those of calls on buffers of their own with a wait behind each."""
    import bit_quantized_decode_gb300 as bq
    layers, page, steps = 12, 16, 25
    lay = ref.Paged(1, [n] * B, [50 + 13 * b + steps * n for b in range(B)], page)
    table, ctx, q_start = (t.cuda() for t in lay.tensors())
    ctx -= steps * n
    batch = bq.KVBatch(table, ctx, q_start, n)
    rope = bq.RopeTable.build(2048, D)
    T, g = lay.T, torch.Generator(device="cuda").manual_seed(1)
    caches = [[bq.KVCache.empty(lay.pages, page, Hkv, D, dtype) for _ in range(layers)] for _ in range(2)]
    atts = [[bq.CachedAttention(c, Hq, rope=rope) for c in cs] for cs in caches]
    qkv = torch.zeros((layers, T, (Hq + 2 * Hkv) * D), device="cuda")
    mask = ref.as_int64([(2 << i) - 1 for i in range(n)] * B).cuda()
    shared = atts[0][0].buffers(T, batch)
    ys = [torch.empty_like(shared.y) for _ in range(layers)]

    def step():
        for att, x, y in zip(atts[0], qkv, ys):
            att(x, batch, None, mask, type(shared)(shared.q, y, shared.workspace))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(steps):
        qkv.normal_(generator=g)
        graph.replay() if k % 5 else step()
        torch.cuda.synchronize()
        for i, (att, x) in enumerate(zip(atts[1], qkv)):
            own = att.buffers(T, batch)
            torch.cuda.synchronize()
            att.append(x, batch, None, own.q)
            torch.cuda.synchronize()
            att.attend(own.q, batch, mask, own.y, own.workspace)
            torch.cuda.synchronize()
            assert own.y.dtype == F32 and torch.equal(own.y, ys[i]), (k, i)
        ctx += n
    for a, b in zip(*caches):
        assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
    assert bq._lib.device_error() == 0


@pytest.mark.parametrize("Hq", [4, 32])
def test_calls_on_given_buffers_allocate_nothing(Hq):
    """Append, attention of either kernel, the joined call and logit rules: neither torch's allocator nor the device gives
    memory, and a capture, which would refuse it, takes them."""
    import bit_quantized_decode_gb300 as bq
    lay = ref.Paged(1, [3, 1], [100, 7], 16)
    batch = bq.KVBatch(*[t.cuda() for t in lay.tensors()], max_tokens=3)
    att = bq.CachedAttention(bq.KVCache.empty(lay.pages, 16, 2, 64, BF16), Hq, rope=bq.RopeTable.build(128, 64))
    qkv, b = torch.randn((4, (Hq + 4) * 64), device="cuda"), att.buffers(4, batch)
    mask = ref.as_int64([1, 3, 7, 1]).cuda()
    ids = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    rules = bq.LogitRules(3000, ids, torch.full((2,), 4, dtype=torch.int32, device="cuda"), frequency=torch.ones(2, device="cuda"))
    x, out = torch.zeros((2, 3000), device="cuda"), torch.empty((2, 3000), device="cuda")
    allowed = torch.full((2, 94), -1, dtype=torch.int32, device="cuda")

    def calls():
        att.append(qkv, batch, None, b.q)
        att.attend(b.q, batch, mask, b.y, b.workspace)
        att(qkv, batch, None, mask, b)
        rules(x, out, allowed=allowed)

    calls()                                     # (kernels are loaded)
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"], torch.cuda.mem_get_info()[0]
    for _ in range(20):
        calls()
    torch.cuda.synchronize()
    assert (torch.cuda.memory_stats()["allocation.all.allocated"], torch.cuda.mem_get_info()[0]) == before
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    b.y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert bool((b.y != 0).any()) and bool((out[:, 8:] == 0).all()) and float(out[:, :8].sum()) == -8
