"""The cache append and the tree attention on the GPU against 64-bit implementations: types, layouts, pages, lengths from
one place on, masks that leave rows empty, values that nothing may see."""
import random

import pytest
import torch

import attention_reference as ref
from helpers import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]
F16, BF16, I8, F32 = torch.float16, torch.bfloat16, torch.int8, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def bq():
    import bit_quantized_decode_gb300 as pkg
    pkg._lib.load()
    pkg._lib.clear_device_error()
    yield pkg
    assert pkg._lib.device_error() == 0


def half_unit(t):
    return torch.finfo(t).eps / 2


def make_cache(lay, Hkv, D, dtype, seed):
    """Host tensors k, v (and scales) and their numbers in 64 bits."""
    g = torch.Generator().manual_seed(seed)
    shape = (lay.pages, Hkv, lay.page, D)
    if dtype == I8:
        k, v = (torch.randint(-128, 128, shape, generator=g, dtype=torch.int8) for _ in range(2))
        ks, vs = (0.02 * (0.5 + torch.rand(shape[:3], generator=g)) for _ in range(2))
        return (k, v, ks, vs), k.double() * ks.double()[..., None], v.double() * vs.double()[..., None]
    k, v = (torch.randn(shape, generator=g).to(dtype) for _ in range(2))
    return (k, v, None, None), k.double(), v.double()


def on_gpu(bq, lay, tensors, max_tokens=None):
    cache = bq.KVCache(*[None if t is None else t.cuda() for t in tensors])
    batch = bq.KVBatch(*[t.cuda() for t in lay.tensors()], max_tokens=max_tokens or max(lay.ns + [1]))
    return cache, batch


def units(cache_dtype, y_dtype):
    """Relative rounding of a probability (two parts and more where the output has more bits), of an output (a 32-bit one is
    divided and rounded too)."""
    pt = F16 if cache_dtype == F16 else BF16
    p = half_unit(pt) ** 2 * 2 if y_dtype == F32 or (y_dtype, pt) == (F16, BF16) else half_unit(pt)
    return p, half_unit(y_dtype) + 2.0 ** -22


def check_attention(bq, seed, ns, ctxs, page, Hq, Hkv, D, dtype, y_dtype, masks=None, q_dtype=None, scale=None, pad=0, q_gain=1.0):
    lay = ref.Paged(seed, ns, ctxs, page)
    tensors, k64, v64 = make_cache(lay, Hkv, D, dtype, seed)
    q_dtype = q_dtype or (BF16 if dtype == I8 else dtype)
    q = (q_gain * torch.randn((lay.T + pad, Hq, D), generator=torch.Generator().manual_seed(seed + 1))).to(q_dtype)
    cache, batch = on_gpu(bq, lay, tensors)
    att = bq.CachedAttention(cache, Hq, scale=scale, q_dtype=q_dtype)
    y = torch.full((lay.T + pad, Hq, D), 7.0, dtype=y_dtype, device="cuda")
    m = None if masks is None else ref.as_int64(masks + [0] * pad).cuda()
    ws = torch.full((att.workspace(lay.T + pad, batch).numel(),), 255, dtype=torch.uint8, device="cuda")   # nothing to keep
    att.attend(q.cuda(), batch, m, y, ws)
    rows = masks if masks is not None else [(2 << i) - 1 for n in ns for i in range(n)]
    want, bound = ref.attend(lay, q[: lay.T].double(), k64, v64, rows, att.scale, *units(dtype, y_dtype), rounded_scales=dtype == I8)
    got = y.cpu()
    err = (got[: lay.T].double() - want).abs()
    assert bool((err <= bound + 1e-30).all()), f"error {float(err.max())}, {float((err / (bound + 1e-30)).max())} of the bound"
    assert bool((got[lay.T:] == 7.0).all()), "rows behind the last sequence"
    return got


SHAPES = [(28, 4, 128), (8, 1, 256), (4, 4, 64), (6, 2, 64), (3, 1, 128), (16, 2, 256)]


@pytest.mark.parametrize("y_dtype", [F32, F16, BF16])
@pytest.mark.parametrize("dtype", [BF16, F16, I8])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
def test_attention_of_trees_of_ragged_sequences(bq, Hq, Hkv, D, dtype, y_dtype):
    rng = random.Random(Hq * D)
    ns, ctxs = [5, 1, 16, 2], [37, 300, 0, 130]
    masks = [m for n in ns for m in ref.tree(rng, n)[0]]
    check_attention(bq, 3, ns, ctxs, 32, Hq, Hkv, D, dtype, y_dtype, masks, pad=3)


@pytest.mark.parametrize("dtype", [BF16, F16, I8])
@pytest.mark.parametrize("ctx", [0, 1, 14, 15, 16, 17, 63, 64, 127, 128, 1000, 2047])
def test_attention_of_one_token_at_every_length(bq, ctx, dtype):
    check_attention(bq, ctx, [1], [ctx], 16, 28, 4, 128, dtype, F32)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D,dtype", [(64, I8), (64, BF16), (128, F16), (256, I8), (256, BF16)])
def test_attention_over_pages_of_every_size(bq, page, D, dtype):
    check_attention(bq, page, [3, 7], [page * 3 - 5, page + 1], page, 14, 2, D, dtype, BF16 if dtype != F16 else F16)


@pytest.mark.parametrize("n", [2, 17, 33, 63, 64])
@pytest.mark.parametrize("dtype,y_dtype", [(BF16, BF16), (F16, F32), (I8, F32)])
def test_attention_of_wide_trees(bq, n, dtype, y_dtype):
    masks = ref.tree(random.Random(n), n)[0]
    check_attention(bq, n, [n], [91], 16, 14, 2, 128, dtype, y_dtype, masks)


@pytest.mark.parametrize("dtype", [BF16, I8])
def test_causal_rows_without_a_mask(bq, dtype):
    check_attention(bq, 9, [64, 1, 30], [5, 900, 0], 64, 8, 2, 128, dtype, F32)


def test_fp16_queries_over_an_int8_cache_and_another_scale(bq):
    check_attention(bq, 4, [4], [500], 32, 8, 1, 256, I8, F16, q_dtype=F16, scale=0.2)


@pytest.mark.parametrize("dtype", [BF16, F16, I8])
def test_large_scores(bq, dtype):
    """Scores in the hundreds: most probabilities vanish, maxima move late."""
    check_attention(bq, 6, [3], [700], 64, 7, 1, 128, dtype, F32, q_gain=12.0)


@pytest.mark.parametrize("dtype", [BF16, F16, I8])
def test_many_sequences_share_the_blocks(bq, dtype):
    """More segments than blocks, of lengths from nothing to some hundred, sequences without rows among them."""
    rng = random.Random(8)
    ns = [rng.choice([0, 1, 1, 2, 5]) for _ in range(150)]
    ctxs = [rng.choice([0, 1, 3, 40, 333]) for _ in ns]
    masks = [m for n in ns for m in ref.tree(rng, n)[0]]
    check_attention(bq, 8, ns, ctxs, 16, 8, 4, 64, dtype, F32, masks, pad=2)


@pytest.mark.parametrize("B", [1024])
def test_the_most_sequences(bq, B):
    check_attention(bq, 10, [1] * B, [b % 20 for b in range(B)], 16, 2, 1, 64, BF16, BF16)


@pytest.mark.parametrize("dtype", [BF16, F16, I8])
def test_rows_that_see_nothing_are_zero(bq, dtype):
    masks = [0b0000, 0b0010, 0b0000, 0b1001]
    got = check_attention(bq, 2, [4], [0], 16, 8, 2, 128, dtype, F32, masks)
    assert bool((got[0] == 0).all()) and bool((got[2] == 0).all())
    # the same with a context: only the drafts are hidden
    check_attention(bq, 2, [4], [100], 16, 8, 2, 128, dtype, F32, masks)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [BF16, F16, I8])
def test_what_a_row_does_not_see_does_not_reach_it(bq, dtype, bad):
    """Infinities and NaN in drafts of other paths, behind the last place and in pages of nobody."""
    D, Hq, Hkv, page = 128, 8, 2, 16
    for ctx in (3, 45):
        lay = ref.Paged(5, [4], [ctx], page)
        tensors, k64, v64 = make_cache(lay, Hkv, D, dtype, 5)
        clean = [None if t is None else t.clone() for t in tensors]
        used = ctx + 4
        hidden = [ctx + 1] + list(range(used, len(lay.table[0]) * page))        # draft 1, and behind the end
        for p in hidden:
            pg, off = lay.table[0][p // page], p % page
            if dtype == I8:
                tensors[2][pg, :, off], tensors[3][pg, :, off] = bad, bad
            else:
                tensors[0][pg, :, off], tensors[1][pg, :, off] = bad, bad
        masks = [0b0001, 0b0011, 0b0101, 0b1101]                                # only row 1 sees draft 1
        q = torch.randn((4, Hq, D), generator=torch.Generator().manual_seed(1)).to(F16 if dtype == F16 else BF16)
        ys = []
        for ts in (tensors, clean):
            cache, batch = on_gpu(bq, lay, ts)
            ys.append(bq.CachedAttention(cache, Hq).attend(q.cuda(), batch, ref.as_int64(masks).cuda(),
                                                           torch.empty((4, Hq, D), device="cuda")).cpu())
        want, bound = ref.attend(lay, q.double(), k64, v64, masks, D ** -0.5, *units(dtype, F32), rounded_scales=dtype == I8)
        for t in (0, 2, 3):
            for y in ys:
                assert bool(((y[t].double() - want[t]).abs() <= bound[t]).all())
        assert not bool(torch.isfinite(ys[0][1]).any())
        assert bool(((ys[1][1].double() - want[1]).abs() <= bound[1]).all())


def test_pages_that_the_cache_does_not_have_hold_nothing(bq):
    lay = ref.Paged(1, [2], [60], 16)
    tensors, k64, v64 = make_cache(lay, 2, 64, BF16, 1)
    q = torch.randn((2, 4, 64), generator=torch.Generator().manual_seed(1)).to(BF16)
    table, ctx, q_start = lay.tensors()
    short = ref.Paged(1, [2], [60], 16)
    for entry in (-1, lay.pages, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[0, 1] = entry                                                         # places 16 .. 31
        batch = bq.KVBatch(t.cuda(), ctx.cuda(), q_start.cuda(), max_tokens=2)
        cache = bq.KVCache(tensors[0].cuda(), tensors[1].cuda())
        y = bq.CachedAttention(cache, 4).attend(q.cuda(), batch, y=torch.empty((2, 4, 64), device="cuda")).cpu()
        keep = [p for p in range(62) if not 16 <= p < 32]
        K, V = (short.gather(x, 0, 62)[:, keep] for x in (k64, v64))
        for i in range(2):
            n = len(keep) - 1 + i
            s = torch.einsum("hgd,hld->hgl", q[i].double().view(2, 2, 64), K[:, :n]) / 8
            want = torch.einsum("hgl,hld->hgd", torch.softmax(s, -1), V[:, :n]).reshape(4, 64)
            assert float((y[i].double() - want).abs().max()) <= 2.0 ** -13    # (probabilities of 16 bits and a part: far less)


def test_arrays_beyond_their_ranges_touch_nothing_else(bq):
    """Starts behind the rows, negative contexts, contexts past the table: results only where there are rows and places."""
    lay = ref.Paged(3, [1, 1], [20, 20], 16)
    tensors, _, _ = make_cache(lay, 2, 64, F16, 3)
    cache = bq.KVCache(tensors[0].cuda(), tensors[1].cuda())
    table, ctx, q_start = lay.tensors()
    q = torch.randn((2, 4, 64), generator=torch.Generator().manual_seed(1)).to(F16).cuda()
    att = bq.CachedAttention(cache, 4)
    for ctxs, starts in (([-5, 1 << 30], [0, 1, 2]), ([20, 20], [0, 1, 100]), ([20, 20], [5, 6, 7]), ([2 ** 31 - 1, 3], [0, 2, 2]),
                         ([20, 20], [0, -3, 2]), ([20, 20], [-4, 1, 2]), ([20, 20], [2, 1, 0])):
        batch = bq.KVBatch(table.cuda(), torch.tensor(ctxs, dtype=torch.int32).cuda(), torch.tensor(starts, dtype=torch.int32).cuda(), 2)
        y = torch.full((4, 4, 64), 3.0, device="cuda")
        att.attend(q, batch, y=y[1:3].contiguous())
        att.append(torch.randn((2, 8 * 64), device="cuda"), batch, q=q.clone())
        assert bool((y[0] == 3.0).all()) and bool((y[3] == 3.0).all())
    torch.cuda.synchronize()


# ------------------------------------------------------------------ append
def check_append(bq, seed, ns, ctxs, page, Hq, Hkv, D, dtype, x_dtype, rot, layout, norm, positions=None, pad=0, wide=0, q_dtype=None,
                 gain=3.0):
    lay = ref.Paged(seed, ns, ctxs, page)
    tensors, _, _ = make_cache(lay, Hkv, D, dtype, seed)
    g = torch.Generator().manual_seed(seed + 2)
    width = (Hq + 2 * Hkv) * D
    store = (gain * torch.randn((lay.T + pad, width + wide), generator=g)).to(x_dtype)
    gq, gk = (1 + 0.2 * torch.randn(D, generator=g) for _ in range(2))
    pos = torch.tensor(positions if positions is not None else [x + i for n, x in zip(ns, ctxs) for i in range(n)], dtype=torch.int32)
    table_len = int(pos.max()) + 1 if len(pos) else 1
    inv, sc = bq.RopeTable.frequencies(rot, 1e4)
    ang = torch.arange(table_len, dtype=torch.float64)[:, None] * inv
    turns = torch.stack([ang.cos() * sc, ang.sin() * sc], -1).to(F32)
    cache, batch = on_gpu(bq, lay, tensors)
    rope = bq.RopeTable(turns.cuda(), layout) if rot else None
    q_dtype = q_dtype or (BF16 if dtype == I8 else dtype)
    att = bq.CachedAttention(cache, Hq, rope=rope, q_norm=gq.cuda() if norm else None, k_norm=gk.cuda() if norm else None, eps=EPS,
                             q_dtype=q_dtype)
    q = torch.full((lay.T + pad, Hq, D), 7.0, dtype=q_dtype, device="cuda")
    gpu_store = store.cuda()
    att.append(gpu_store[:, :width], batch, None if positions is None else torch.cat([pos, torch.zeros(pad, dtype=torch.int32)]).cuda(), q)
    x = store[: lay.T, :width].double().view(lay.T, Hq + 2 * Hkv, D)
    xq, xk, xv = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if norm:
        xq, xk = ref.norm_heads(xq, gq.double(), EPS), ref.norm_heads(xk, gk.double(), EPS)
    tt = turns.double()[pos.long()] if rot else torch.zeros((lay.T, 0, 2), dtype=torch.float64)
    yq, yk = (ref.rotate(t, tt, layout == "interleaved") for t in (xq, xk))
    # a rotated fp32 value: two products and a sum, each off by half a step of numbers up to |a| + |b|; then the type's step
    mag = lambda t: ref.rotate(t.abs(), torch.stack([tt[..., 0].abs(), -tt[..., 1].abs()], -1), layout == "interleaved").abs() + (  # noqa: E731
        ref.rotate(t.abs(), tt.abs(), layout == "interleaved").abs())
    tol = lambda t, y, dt: 3 * 2.0 ** -24 * mag(t) + y.abs() * half_unit(dt) * (1 + 2.0 ** -8) + 2.0 ** -25      # noqa: E731
    got = q.cpu()
    assert bool(((got[: lay.T].double() - yq).abs() <= tol(xq, yq, q_dtype)).all()), "queries"
    assert bool((got[lay.T:] == 7.0).all()), "queries behind the last sequence"
    # the cache: new places as the definition has them, all others as they were
    want_k, want_v = tensors[0].clone(), tensors[1].clone()
    new = [(lay.table[b][(x0 + i) // page], (x0 + i) % page) for b, (n, x0) in enumerate(zip(ns, ctxs)) for i in range(n)]
    pg, off = (torch.tensor([p[j] for p in new], dtype=torch.long) for j in (0, 1))
    if dtype == I8:
        ks, vs = tensors[2].clone(), tensors[3].clone()
        want_k[pg, :, off], ks[pg, :, off] = ref.codes(ref.one(yk))
        want_v[pg, :, off], vs[pg, :, off] = ref.codes(xv)
        assert torch.equal(cache.k.cpu(), want_k) and torch.equal(cache.v.cpu(), want_v)
        assert torch.equal(cache.k_scale.cpu(), ks) and torch.equal(cache.v_scale.cpu(), vs)
        assert torch.equal(cache.values("k").cpu(), want_k * ks[..., None])
        return
    got_k = cache.k.cpu()
    assert bool(((got_k[pg, :, off].double() - yk).abs() <= tol(xk, yk, dtype)).all()), "keys"
    got_k[pg, :, off] = want_k[pg, :, off]
    assert torch.equal(got_k, want_k), "other places of the keys"
    want_v[pg, :, off] = xv.to(dtype)
    assert torch.equal(cache.v.cpu(), want_v), "values"


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("x_dtype", [F32, BF16, F16])
@pytest.mark.parametrize("dtype", [BF16, F16, I8])
@pytest.mark.parametrize("Hq,Hkv,D", [(28, 4, 128), (8, 1, 256), (5, 5, 64), (3, 1, 64)])
def test_append_types_and_heads(bq, Hq, Hkv, D, dtype, x_dtype, norm):
    check_append(bq, D + Hq, [5, 1, 16, 3], [37, 300, 0, 61], 32, Hq, Hkv, D, dtype, x_dtype, D, "half", norm, pad=2)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [F16, I8])
@pytest.mark.parametrize("D,rot", [(64, 0), (64, 8), (64, 32), (128, 64), (128, 120), (128, 128), (256, 64), (256, 256)])
def test_append_rotates_part_of_the_head_in_either_layout(bq, D, rot, layout, dtype):
    check_append(bq, rot, [7], [100], 16, 6, 2, D, dtype, F32, rot, layout, True)


@pytest.mark.parametrize("dtype", [BF16, I8])
def test_append_far_positions_of_a_tree(bq, dtype):
    """Positions by depth, not by place, and far out."""
    _, depth = ref.tree(random.Random(4), 16)
    check_append(bq, 4, [16], [250], 64, 8, 2, 128, dtype, F32, 128, "half", True, positions=[131000 + d for d in depth])


@pytest.mark.parametrize("T", [1, 2, 257, 1500])
def test_append_prompts(bq, T):
    check_append(bq, T, [T], [13], 256, 4, 1, 128, I8, BF16, 128, "half", True)


def test_append_rows_that_are_apart(bq):
    check_append(bq, 7, [5], [10], 16, 4, 2, 64, BF16, F32, 64, "half", False, wide=36)
    check_append(bq, 7, [5], [10], 16, 4, 2, 64, F16, BF16, 64, "half", True, wide=8)
    check_append(bq, 7, [1], [10], 16, 4, 2, 64, F16, F32, 64, "half", True, wide=3)


def test_append_small_and_zero_values(bq):
    check_append(bq, 8, [3], [0], 16, 2, 1, 64, I8, F32, 64, "half", False, gain=0.0)
    check_append(bq, 8, [3], [0], 16, 2, 1, 64, I8, F32, 64, "half", False, gain=1e-36)
    check_append(bq, 8, [3], [0], 16, 2, 1, 64, I8, F32, 64, "interleaved", False, gain=1e30)


def test_append_positions_outside_the_table_give_nan(bq):
    for dtype in (BF16, I8):
        cache = bq.KVCache.empty(2, 16, 1, 64, dtype)
        turns = torch.ones((4, 32, 2), device="cuda")
        att = bq.CachedAttention(cache, 2, rope=bq.RopeTable(turns))
        i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()                  # noqa: E731
        batch = bq.KVBatch(i32([[0, 1]]), i32([0]), i32([0, 3]), 3)
        q = att.append(torch.ones((3, 4 * 64), device="cuda"), batch, i32([-1, 2, 4]))
        assert bool(torch.isnan(q[0]).all()) and bool(torch.isnan(q[2]).all()) and bool(torch.isfinite(q[1].float()).all())
        k = cache.values("k")[0, 0]
        assert bool(torch.isnan(k[0]).all()) and bool(torch.isnan(k[2]).all()) and bool(torch.isfinite(k[1].float()).all())
        assert bool((cache.values("v")[0, 0, :3].float() - 1).abs().max() < 0.01)


def test_append_places_without_a_page_are_not_written(bq):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()                      # noqa: E731
    for table in ([[-1, 1]], [[7, 1]], [[0, 1]]):
        cache = bq.KVCache.empty(2, 16, 1, 64, F16)
        batch = bq.KVBatch(i32(table), i32([14 if table[0][0] != 0 else 31]), i32([0, 4]), 4)
        q = bq.CachedAttention(cache, 2).append(torch.ones((4, 4 * 64), device="cuda"), batch)
        assert bool((q == 1).all())
        want = torch.zeros(2, 16)
        want[1, [15] if table[0][0] == 0 else [0, 1]] = 1
        assert torch.equal(cache.k[:, 0, :, 0].cpu().float(), want) and torch.equal(cache.v[:, 0, :, 5].cpu().float(), want)


@pytest.mark.parametrize("scaling", [None, {"kind": "linear", "factor": 4.0}, {"kind": "base", "factor": 8.0},
                                     {"kind": "by_parts", "factor": 4.0, "trained": 4096}])
def test_rope_table_against_64_bits(bq, scaling):
    rot, positions = 128, 140000
    t = bq.RopeTable.build(positions, rot, 1e6, scaling=scaling).turns.cpu()
    inv, scale = bq.RopeTable.frequencies(rot, 1e6, scaling)
    ang = torch.arange(positions, dtype=torch.float64)[:, None] * inv
    # angles up to 140000 in 64 bits: 2^-36 off at most, with the device's sincos; rounded to 32 bits
    for j, f in enumerate((torch.cos, torch.sin)):
        want = f(ang) * scale
        assert float((t[..., j].double() - want).abs().max()) <= 2.0 ** -25 * 2 + 2.0 ** -33


# ------------------------------------------------------------- together
@pytest.mark.parametrize("dtype,x_dtype", [(BF16, F32), (I8, F32), (F16, BF16)])
def test_steps_of_a_decode_append_then_attend(bq, dtype, x_dtype):
    """Steps of drafts of three sequences on one cache, the contexts updated on the device: each step's attention against
    the 64-bit attention over the cache as it is then."""
    D, Hq, Hkv, page, B = 128, 14, 2, 16, 3
    rng = random.Random(1)
    g = torch.Generator().manual_seed(1)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()                      # noqa: E731
    cache = bq.KVCache.empty(40, page, Hkv, D, dtype)
    pages = list(range(40))
    rng.shuffle(pages)
    table = [pages[12 * b:12 * b + 12] for b in range(B)]
    att = bq.CachedAttention(cache, Hq, rope=bq.RopeTable.build(512, D))
    ctx = i32([0, 0, 0])
    batch = bq.KVBatch(i32(table), ctx, i32([0, 4, 8, 12]), max_tokens=4)
    buffers = att.buffers(12, batch, F32)
    for step in range(9):
        trees = [ref.tree(rng, 4) for _ in range(B)]
        masks = [m for t in trees for m in t[0]]
        ctxs = ctx.tolist()
        pos = i32([x + d for x, t in zip(ctxs, trees) for d in t[1]])
        qkv = torch.randn((12, (Hq + 2 * Hkv) * D), generator=g).to(x_dtype).cuda()
        y = att(qkv, batch, pos, ref.as_int64(masks).cuda(), buffers)
        lay = ref.Paged(0, [4] * B, ctxs, page)
        lay.table = table
        want, bound = ref.attend(lay, buffers.q.cpu().double(), cache.values("k").cpu().double(), cache.values("v").cpu().double(),
                                 masks, D ** -0.5, *units(dtype, F32), rounded_scales=dtype == I8)
        # (codes times scales are rounded in values(): half a step of each number)
        slack = 0 if dtype != I8 else float(want.abs().max()) * 2.0 ** -20
        assert bool(((y.cpu().double() - want).abs() <= bound + slack).all()), step
        ctx += i32([rng.randint(0, 4) for _ in range(B)])
