"""Attention over a paged cache against 64 bits with bounds that do not grow to percents over long contexts: scales that differ
from tile to tile, probabilities far below the largest, sums of one sign."""
import pytest
import torch

import attention_reference as ref
from helpers import cuda_ok
from test_gpu_attention import BF16, F16, F32, I8, half_unit, on_gpu

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module")
def bq():
    import bit_quantized_decode_gb300 as pkg
    pkg._lib.load()
    pkg._lib.clear_device_error()
    yield pkg
    assert pkg._lib.device_error() == 0


def parts_unit(cache_dtype, y_dtype):
    """Relative rounding of a probability: the square of its type's, twice, where it has two parts or more (all but bf16
    outputs over an fp16 cache: 11 bits)."""
    u = half_unit(F16 if cache_dtype == F16 else BF16)
    return u if cache_dtype == F16 and y_dtype == BF16 else 2 * u * u


def cuts_of(half, y_dtype):
    """Steps on the tensor cores that add up in a sum: 192 (12 a tile of 64 places, 16 tiles); 1024 for fp16 over an fp16 cache,
    8192 for bf16."""
    return 192 if y_dtype == F32 else 8192 if y_dtype == BF16 else 1024 if half else 192


def attend_64(lay, q, k, v, masks, scale, y_dtype, p_unit, half, exact):
    """Outputs in 64 bits and the bound of the kernels' error, on q's device.  The score's and the exponential's part is that of
    attention_reference.attend.  The sums': a product's step on the tensor cores cuts 2^-23 of the sum at most, cuts_of of them
    add up; the sums in fp32 take a step of 2^-24 for every
    16 places at most, and some 64 to join the parts.  Numerator and sum have them both.  A probability in fp16 parts is
    2^9 times as large as it stands to the largest, or more, and off by half of fp16's least step, 2^-25.  exact: the scores'
    products and their sums are fp32 numbers."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    y, bound = torch.zeros_like(q), torch.zeros_like(q)
    for b, (n, ctx) in enumerate(zip(lay.ns, lay.ctxs)):
        page = torch.tensor(lay.table[b][: (ctx + n + lay.page - 1) // lay.page], device=q.device)
        K, V = (t[page].transpose(0, 1).reshape(Hkv, -1, D)[:, : ctx + n] for t in (k, v))
        for i in range(n):
            t = lay.q_start[b] + i
            see = torch.arange(ctx + n, device=q.device) < ctx
            for j in range(n):
                see[ctx + j] = bool(masks[t] >> j & 1)
            qq, Ks, Vs = q[t].view(Hkv, -1, D), K[:, see], V[:, see]
            s = scale * torch.einsum("hgd,hld->hgl", qq, Ks)
            p = torch.softmax(s, -1)
            y[t] = torch.einsum("hgl,hld->hgd", p, Vs).reshape(Hq, D)
            mag = scale * torch.einsum("hgd,hld->hgl", qq.abs(), Ks.abs()).amax(-1, keepdim=True)
            ds = (0.0 if exact else mag * (D + 16) * 2.0 ** -23) + 3 * s.abs().amax(-1, keepdim=True) * 2.0 ** -22
            cuts = cuts_of(half, y_dtype)
            e = 2 * ds + 2.0 ** -20 + 2 * (cuts * 2.0 ** -23 + (Ks.shape[1] / 16 + 64) * 2.0 ** -24)
            weight = torch.einsum("hgl,hld->hgd", p, Vs.abs())
            least = 2.0 ** -34 * p.amax(-1, keepdim=True) * Vs.abs().sum(1)[:, None] if half else 0.0
            bound[t] = (weight * (e + p_unit) + least).reshape(Hq, D) + y[t].abs() * (half_unit(y_dtype) + 2.0 ** -22)
            if y_dtype == F16:                  # an output below 2^-14 has fp16's least step, 2^-24: off by half of it
                bound[t] += 2.0 ** -25
    return y, bound


def check(bq, lay, tensors, k64, v64, q, masks, y_dtype, but=(), exact=False):
    """All rows but some against 64 bits; the outputs."""
    cache, batch = on_gpu(bq, lay, tensors)
    T, Hq, D = q.shape
    att = bq.CachedAttention(cache, Hq, q_dtype=q.dtype)
    y = att.attend(q.cuda(), batch, ref.as_int64(masks).cuda(), torch.empty((T, Hq, D), dtype=y_dtype, device="cuda"))
    want, bound = attend_64(lay, q.cuda().double(), k64.cuda(), v64.cuda(), masks, att.scale, y_dtype,
                            parts_unit(tensors[0].dtype, y_dtype), tensors[0].dtype == F16, exact)
    err = (y.double() - want).abs()
    err[list(but)] = 0.0
    assert bool((err <= bound + 1e-30).all()), f"error {float(err.max())}, {float((err / (bound + 1e-30)).max())} of the bound"
    return y.cpu()


@pytest.mark.parametrize("y_dtype", [F32, F16])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (40, 2, 64), (2, 1, 128), (28, 4, 128), (64, 2, 128), (2, 1, 256), (8, 1, 256), (32, 2, 256)])
def test_int8_scales_that_differ_from_tile_to_tile(bq, Hq, Hkv, D, y_dtype):
    """Every tile of 16 places has scales of its own, up to 32 times another's: the scales of another tile give percents."""
    for ns, ctxs, page in (([5], [2900], 16), ([5, 2], [700, 61], 64), ([5] * 40, [130 + 16 * b for b in range(40)], 32)):
        lay = ref.Paged(D + Hq, ns, ctxs, page)
        g = torch.Generator().manual_seed(D + Hq)
        shape = (lay.pages, Hkv, page, D)
        k, v = (torch.randint(-127, 128, shape, generator=g, dtype=torch.int8) for _ in range(2))
        power = torch.randint(0, 6, (2, lay.pages, Hkv, page // 16, 1), generator=g).expand(-1, -1, -1, -1, 16).reshape(2, *shape[:3])
        ks, vs = 2.0 ** power * 0.002 * (0.5 + torch.rand((2, *shape[:3]), generator=g))
        masks = [m for n in ns for m in [1, 3, 5, 13, 17][:n]]
        q = (0.2 * torch.randn((lay.T, Hq, D), generator=g)).to(BF16)
        check(bq, lay, (k, v, ks, vs), k.double() * ks.double()[..., None], v.double() * vs.double()[..., None], q, masks, y_dtype)


@pytest.mark.parametrize("y_dtype", [F32, F16])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,ctx", [(1, 100), (3, 700), (160, 1030)])
def test_hidden_infinities_in_a_tile_that_raises_the_maximum(bq, B, ctx, dtype, y_dtype):
    """The tile of the drafts holds a key that all rows like 2^20 and more better than those before: the output so far is
    rescaled (with 160 sequences, it is also taken out before, 16 tiles into a block), and an infinite draft that one row of
    three sees is added by both halves of a row's threads."""
    D, Hq, n, page = 64, 8, 3, 32
    lay = ref.Paged(B, [n] * B, [ctx] * B, page)
    g = torch.Generator().manual_seed(B)
    like = torch.randn(D, generator=g)
    like *= D ** 0.5 / like.norm()
    q = (like + 0.1 * torch.randn((lay.T, Hq, D), generator=g)).to(dtype)
    k, v = (torch.randn((lay.pages, 1, page, D), generator=g) for _ in range(2))
    k *= 0.3
    for b in range(B):
        liked, hidden = ctx // 64 * 64, ctx + 1
        k[lay.table[b][liked // page], 0, liked % page] = 2.5 * like
        v[lay.table[b][hidden // page], 0, hidden % page] = float("inf")
    k, v = k.to(dtype), v.to(dtype)
    seeing = [lay.q_start[b] + 1 for b in range(B)]
    y = check(bq, lay, (k, v, None, None), k.double(), v.double(), q, [1, 3, 5] * B, y_dtype, but=seeing)
    assert not bool(torch.isfinite(y[seeing]).any())


@pytest.mark.parametrize("gap", [6, 10, 14, 18, 22])
@pytest.mark.parametrize("y_dtype", [F32, F16])
@pytest.mark.parametrize("Hq,D,n", [(4, 64, 1), (28, 128, 1), (28, 128, 5), (8, 256, 4)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_one_place_far_ahead_of_all_others(bq, dtype, Hq, D, n, y_dtype, gap):
    """A place that is `gap` nats ahead and adds next to nothing (an attention sink), first, in the middle and last: what the
    others add, each e^-gap of it, must not be lost in a probability's 16 bits.  Queries of ones, keys of one magnitude or
    zero: exact scores."""
    ctx, page, Hkv = 8190, 64, 1
    for ahead in (0, 4000, ctx - 1):
        lay = ref.Paged(gap, [n], [ctx], page)
        g = torch.Generator().manual_seed(gap)
        like = torch.ones(D)
        like[torch.randperm(D, generator=g)[: D // 2]] = -1.0
        k = torch.zeros((lay.pages, Hkv, page, D))
        v = 1.0 + torch.rand((lay.pages, Hkv, page, D), generator=g)
        at = lay.table[0][ahead // page], 0, ahead % page
        k[at], v[at] = gap / D ** 0.5 * like, 0.0
        q = like.expand(lay.T, Hq, D).to(dtype)
        k, v = k.to(dtype), v.to(dtype)
        check(bq, lay, (k, v, None, None), k.double(), v.double(), q, [(2 << i) - 1 for i in range(n)], y_dtype, exact=True)


# ------------------------------- long sums for 16-bit outputs (probabilities of one part)
def on_gpu_only(bq, B, n, ctx, Hkv, D, dtype, seed, grow=False, sign=False):
    """A cache made on the GPU: its parts, their numbers in 64 bits are the caller's."""
    page = 64
    lay = ref.Paged(seed, [n] * B, [ctx] * B, page)
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (lay.pages, Hkv, page, D)
    kind = F16 if dtype == F16 else BF16
    if dtype == I8:
        k, v = (torch.randint(-127, 128, shape, generator=g, dtype=torch.int8, device="cuda") for _ in range(2))
        scales = [0.004 * (0.5 + torch.rand(shape[:3], generator=g, device="cuda")) for _ in range(2)]
    else:
        k, v = (torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g) for _ in range(2))
        k *= 0.3
        scales = [None, None]
    if sign:
        v.abs_()
    if grow:                                    # keys (their scales) that grow with the place
        table = torch.tensor(lay.table, device="cuda").clamp(min=0).flatten()
        by = torch.zeros(lay.pages, device="cuda")
        by[table] = 0.02 + 3.0 * torch.arange(len(lay.table[0]), device="cuda").repeat(B) / len(lay.table[0])
        if dtype == I8:
            scales[0] *= by[:, None, None]
        else:
            k *= by[:, None, None, None].to(dtype)
    batch = bq.KVBatch(*[t.cuda() for t in lay.tensors()], max_tokens=n)
    q = lambda Hq: torch.randn((lay.T, Hq, D), generator=g, device="cuda").to(kind)          # noqa: E731
    return lay, bq.KVCache(k, v, *scales), batch, q


@pytest.mark.parametrize("G,n", [(16, 2), (8, 1)])
def test_long_sums_of_one_sign_stay_centred(bq, G, n):
    """131071 places to a block, values that are all positive, fp16 outputs: what the tensor cores cut from the sums is 1024
    steps of 2^-23 at most, however long the context.  The mean over many outputs, which their rounding leaves alone: it is
    2^-12 / sqrt(3) / sqrt(count) off, taken six times."""
    B, ctx, Hkv, D = 19, 131071, 8, 64
    lay, cache, batch, make_q = on_gpu_only(bq, B, n, ctx, Hkv, D, F16, 3, sign=True)
    q = make_q(G * Hkv)
    y = bq.CachedAttention(cache, G * Hkv).attend(q, batch)
    off = []
    for b in (0, 7, 18):
        table = torch.tensor(lay.table[b], device="cuda")
        for h in range(0, Hkv, 2):
            K, V = (t[table, h].reshape(-1, D).double()[: ctx + n] for t in (cache.k, cache.v))
            for i in range(n):
                t, rows = lay.q_start[b] + i, slice(G * h, G * h + G)
                s = (q[t, rows].double() @ K[: ctx + i + 1].T) * D ** -0.5
                off.append((y[t, rows].double() / (torch.softmax(s, -1) @ V[: ctx + i + 1]) - 1).flatten())
    off = torch.cat(off)
    assert abs(float(off.mean())) <= 1024 * 2.0 ** -23 + 2.0 ** -19 + 6 * 2.0 ** -12 / 3 ** 0.5 / off.numel() ** 0.5, float(off.mean())


@pytest.mark.parametrize("D,dtype,y_dtype", [(64, F16, F16), (64, BF16, BF16), (128, F16, F16), (128, I8, BF16), (256, F16, F16), (256, I8, BF16)])
def test_sums_taken_out_late(bq, D, dtype, y_dtype):
    """313 tiles to a block, one part: the sum is taken out once, at another maximum than in the end."""
    B, ctx, Hkv, n, Hq = 38, 20000, 4, 2, 64
    lay, cache, batch, make_q = on_gpu_only(bq, B, n, ctx, Hkv, D, dtype, D, grow=True)
    q = make_q(Hq)
    att = bq.CachedAttention(cache, Hq)
    y = att.attend(q, batch, y=torch.empty(q.shape, dtype=y_dtype, device="cuda"))
    for b in (0, 20, 37):
        one = ref.Paged(0, [n], [ctx], 64)
        one.table = [list(range(len(lay.table[b])))]
        table = torch.tensor(lay.table[b], device="cuda")
        k, v = (t[table].double() * (1.0 if s is None else s[table].double()[..., None])
                for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        rows = slice(lay.q_start[b], lay.q_start[b] + n)
        want, bound = attend_64(one, q[rows].double(), k, v, [1, 3], att.scale, y_dtype, parts_unit(dtype, y_dtype), dtype == F16, False)
        err = (y[rows].double() - want).abs()
        assert bool((err <= bound).all()), float((err / bound).max())


# -------------------------------------------------------- infinities that are seen
@pytest.mark.parametrize("y_dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hq,D,n,B,ctx", [(4, 64, 1, 1, 300), (28, 128, 1, 2, 1000), (28, 128, 2, 1, 300), (8, 256, 4, 1, 700), (32, 64, 2, 160, 1500)])
def test_infinite_values_give_infinities(bq, Hq, D, n, B, ctx, dtype, y_dtype):
    """A cached place has infinities in ten columns and those of the other sign in ten others: so have all rows, and their other
    columns are what they are without.  (160 sequences: 24 tiles to a block, so sums are taken out.)"""
    page = 32
    lay = ref.Paged(5, [n] * B, [ctx] * B, page)
    g = torch.Generator().manual_seed(D)
    k, v = (torch.randn((lay.pages, 1, page, D), generator=g).to(dtype) for _ in range(2))
    q = (0.3 * torch.randn((lay.T, Hq, D), generator=g)).to(dtype)
    for b in range(B):
        p = (7 + 64 * b) % ctx
        at = lay.table[b][p // page], 0, p % page
        v[at][:10], v[at][10:20] = float("inf"), float("-inf")
    cache, batch = on_gpu(bq, lay, (k, v, None, None))
    y = bq.CachedAttention(cache, Hq).attend(q.cuda(), batch, y=torch.empty((lay.T, Hq, D), dtype=y_dtype, device="cuda"))
    assert bool((y[..., :10] == float("inf")).all()) and bool((y[..., 10:20] == float("-inf")).all())
    masks = [(2 << i) - 1 for i in range(n)] * B
    want, bound = attend_64(lay, q.cuda().double(), k.cuda().double(), v.cuda().double().nan_to_num(0, 0, 0), masks, D ** -0.5, y_dtype,
                            parts_unit(dtype, y_dtype), dtype == F16, False)
    err = (y.double() - want).abs()[..., 20:]
    assert bool((err <= bound[..., 20:]).all()), float((err / bound[..., 20:]).max())


@pytest.mark.parametrize("y_dtype", [F32, F16, BF16])
@pytest.mark.parametrize("Hq,D,n", [(4, 64, 1), (28, 128, 2), (8, 256, 1), (8, 256, 4)])
def test_an_infinite_scale_gives_infinities(bq, Hq, D, n, y_dtype):
    """An INT8 cache's value scale: the codes' signs decide, and a code of 0 times infinity is not a number."""
    lay = ref.Paged(5, [n], [300], 32)
    g = torch.Generator().manual_seed(D)
    shape = (lay.pages, 1, 32, D)
    k, v = (torch.randint(-127, 128, shape, generator=g, dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.full(shape[:3], 0.01) for _ in range(2))
    at = lay.table[0][3], 0, 7
    vs[at], v[at][0] = float("inf"), 0
    cache, batch = on_gpu(bq, lay, (k, v, ks, vs))
    q = (0.3 * torch.randn((n, Hq, D), generator=g)).to(BF16)
    y = bq.CachedAttention(cache, Hq).attend(q.cuda(), batch, y=torch.empty((n, Hq, D), dtype=y_dtype, device="cuda")).cpu()
    want = v[at].float() * float("inf")
    assert bool(torch.isnan(y[..., 0]).all())
    assert torch.equal(torch.isnan(y), torch.isnan(want).expand_as(y))
    good = ~torch.isnan(want)
    assert bool((y[..., good].float() == want[good]).all())


# ------------------------------------------------------------- 16-bit outputs
@pytest.mark.parametrize("dtype,y_dtype", [(BF16, BF16), (I8, BF16), (F16, F16), (BF16, F16), (I8, F16), (F16, BF16)])
@pytest.mark.parametrize("Hq,Hkv,D,n,B", [(4, 2, 64, 1, 40), (28, 4, 128, 1, 20), (28, 4, 128, 16, 3), (8, 1, 256, 1, 30), (8, 1, 256, 5, 8)])
def test_16_bit_outputs_are_as_good_as_rounded_ones(bq, Hq, Hkv, D, n, B, dtype, y_dtype):
    """One place of 300 has values; its probability, below 1 by a place's five before it, is some number that 8 bits do not hold: all
    values of a row would be off by its rounding, the same way.  In two parts they are off by 2^-15 (fp16 2^-20, or 2^-11 in the one
    part that a bf16 output has) and what exponentials and scores (2^-19) and 40 steps of the sums (2^-17) take, and rounded: a value
    that rounding takes to the same side differs as the definition's rounded value does, another one by twice that more.  Exact
    scores: rows and keys of one magnitude."""
    ctx, page = 300, 32
    lay = ref.Paged(D, [n] * B, [ctx] * B, page)
    g = torch.Generator().manual_seed(D + n)
    shape = (lay.pages, Hkv, page, D)
    like = torch.where(torch.rand(D, generator=g) < 0.5, -1.0, 1.0)
    q = (like * (0.5 + torch.rand((lay.T, Hq, 1), generator=g))).to(F16 if dtype == F16 else BF16)
    k, v = torch.zeros(shape), torch.zeros(shape)
    ks, vs = (0.5 + torch.rand(shape[:3], generator=g) for _ in range(2))
    for b in range(B):
        for place, size in ((195, 127.0), (200, 64.0)):
            k[lay.table[b][place // page], :, place % page] = like * size
        at = lay.table[b][200 // page], slice(None), 200 % page
        v[at] = (60 * torch.randn((Hkv, D), generator=g)).clamp(-127, 127).round()
        ks[lay.table[b][195 // page], :, 195 % page] = ks[at] = 2.0 ** -8 / D ** 0.5
    if dtype == I8:
        tensors = (k.to(torch.int8), v.to(torch.int8), ks, vs)
        k64, v64 = k.double() * ks.double()[..., None], v.double() * vs.double()[..., None]
    else:
        k, v = (k * 2.0 ** -8 / D ** 0.5).to(dtype), v.to(dtype)
        tensors, k64, v64 = (k, v, None, None), k.double(), v.double()
    masks = [(2 << i) - 1 for i in range(n)] * B
    y = check(bq, lay, tensors, k64, v64, q, masks, y_dtype, exact=True).double()
    want, _ = attend_64(lay, q.double(), k64, v64, masks, D ** -0.5, y_dtype, 0.0, dtype == F16, True)
    rounded = want.to(y_dtype).double()
    most = (rounded - want).norm() + 2 * (parts_unit(dtype, y_dtype) + 2.0 ** -17 + 2.0 ** -19) * want.norm()
    assert float((y - want).norm()) <= float(most), float((y - want).norm() / (rounded - want).norm())
