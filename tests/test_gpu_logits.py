"""Logit penalties, biases and grammar masks on the GPU against a 64-bit implementation."""
import random

import pytest
import torch

import attention_reference as ref
from helpers import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def bq():
    import bit_quantized_decode_gb300 as pkg
    pkg._lib.load()
    pkg._lib.clear_device_error()
    yield pkg
    assert pkg._lib.device_error() == 0


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


def pack_bits(ok):
    R, V = ok.shape
    bits = torch.zeros((R, (V + 31) // 32 * 32), dtype=torch.int64)
    bits[:, :V] = ok
    words = (bits.view(R, -1, 32) << torch.arange(32)).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


def make_rules(rng, S, V, cap, nb):
    rules = []
    for s in range(S):
        n = rng.choice([0, 1, cap, rng.randint(0, cap)]) if cap else 0
        # repeats, neighbours, ids that no vocabulary has
        ids = [rng.choice([rng.randint(0, V - 1), rng.randint(0, min(V, 9) - 1), -1, V, V + 40000, 2 ** 31 - 1, -2 ** 31]) for _ in range(n)]
        p = rng.randint(0, n)
        bias = [(rng.choice([rng.randint(0, V - 1), V - 1, 0, -1, V + 5]), rng.choice([rng.uniform(-5, 5), float("-inf"), 100.0]))
                for _ in range(nb)]
        rules.append({"prompt": ids[:p], "made": ids[p:], "rep": float(torch.tensor(rng.uniform(0.8, 1.6))),
                      "freq": float(torch.tensor(rng.uniform(0, 1))), "pres": float(torch.tensor(rng.uniform(-0.5, 1))),
                      "bias": [(t, float(torch.tensor(a))) for t, a in bias]})
    return rules


def on_gpu(bq, rules, V, cap, nb):
    S = len(rules)
    ids = torch.full((S, cap), 5, dtype=torch.int32)                  # what is behind the length does not count
    for s, u in enumerate(rules):
        both = u["prompt"] + u["made"]
        ids[s, : len(both)] = torch.tensor(both, dtype=torch.int32)
    vec = lambda k: torch.tensor([u[k] for u in rules], dtype=F32).cuda()          # noqa: E731
    return bq.LogitRules(V, ids.cuda() if cap else None, i32([len(u["prompt"]) + len(u["made"]) for u in rules]).cuda() if cap else None,
                         i32([len(u["prompt"]) for u in rules]).cuda() if cap else None, vec("rep"), vec("freq"), vec("pres"),
                         i32([[t for t, _ in u["bias"]] for u in rules]).cuda() if nb else None,
                         torch.tensor([[a for _, a in u["bias"]] for u in rules], dtype=F32).cuda() if nb else None)


def check(got, want, x, rules_most, dtype):
    """Each of up to four fp32 steps is off by half a step of numbers no larger than `rules_most` beside the logit."""
    fin = torch.isfinite(want)
    assert torch.equal(fin, torch.isfinite(got)), "infinities"
    assert torch.equal(want[~fin & ~torch.isnan(want)], got[~fin & ~torch.isnan(want)].double())
    assert torch.equal(torch.isnan(want), torch.isnan(got))
    mag = x.double().abs().nan_to_num(0, 0, 0)[fin] * 2 + rules_most
    bound = mag * 6 * 2.0 ** -24 + want[fin].abs() * torch.finfo(dtype).eps / 2 + 2.0 ** -25
    assert bool(((got.double()[fin] - want[fin]).abs() <= bound).all())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V", [1, 31, 1000, 8191, 8192, 8200, 20001, 152064])
def test_rows_of_a_batch(bq, V, dtype):
    rng = random.Random(V)
    S, cap, nb, pad = 4, 77, 9, 2
    rules = make_rules(rng, S, V, cap, nb)
    x = (3 * torch.randn((S + pad, V), generator=torch.Generator().manual_seed(V))).to(dtype)
    ok = torch.rand((S + pad, V), generator=torch.Generator().manual_seed(V + 1)) < 0.7
    ok[1] = False                                                     # a grammar that allows nothing
    out = torch.full_like(x, 7.0).cuda()
    y = on_gpu(bq, rules, V, cap, nb)(x.cuda(), out, allowed=pack_bits(ok).cuda())
    assert y is out
    want = ref.logits(x.double(), rules, [(s, []) for s in range(S)], V, ok)
    check(out.cpu()[:S], want[:S], x[:S], 300.0, dtype)
    assert bool((out.cpu()[S:] == 7.0).all()), "rows behind the last sequence"


@pytest.mark.parametrize("with_mask", [True, False])
def test_rows_of_drafted_trees(bq, with_mask):
    rng = random.Random(3)
    V, ns, cap = 9000, [5, 0, 1, 64, 16], 40
    S, R = len(ns), sum(ns) + 3
    rules = make_rules(rng, S, V, cap, 3)
    drafts = [rng.randint(0, 30) for _ in range(R)]
    drafts[2] = -1
    trees = [ref.tree(rng, n, chain=not with_mask)[0] for n in ns]
    starts, rows, masks = [0], [], []
    for s, (n, t) in enumerate(zip(ns, trees)):
        f = starts[-1]
        starts.append(f + n)
        rows += [(s, [drafts[f + j] for j in range(n) if m >> j & 1]) for m in t]
        masks += t
    x = torch.randn((R, V), generator=torch.Generator().manual_seed(1))
    out = torch.full_like(x, 7.0).cuda()
    on_gpu(bq, rules, V, cap, 3)(x.cuda(), out, i32(starts).cuda(), i32(drafts).cuda(),
                                 ref.as_int64(masks + [-1] * 3).cuda() if with_mask else None)
    want = ref.logits(x.double(), rules, rows + [None] * 3, V)
    check(out.cpu()[:R - 3], want[:R - 3], x[:R - 3], 300.0, F32)
    assert bool((out.cpu()[R - 3:] == 7.0).all())


def test_in_place_and_rows_that_are_apart(bq):
    rng = random.Random(5)
    for V, wide in ((5000, 8), (5000, 3), (5003, 0), (5003, 1)):
        rules = make_rules(rng, 3, V, 20, 2)
        store = torch.randn((3, V + wide), generator=torch.Generator().manual_seed(V))
        x = store[:, :V].clone()
        gpu = store.cuda()
        on_gpu(bq, rules, V, 20, 2)(gpu[:, :V], gpu[:, :V])
        check(gpu.cpu()[:, :V], ref.logits(x.double(), rules, [(s, []) for s in range(3)], V), x, 300.0, F32)
        assert torch.equal(gpu.cpu()[:, V:], store[:, V:])


def test_infinite_and_nan_logits(bq):
    V = 100
    x = torch.zeros((1, V))
    x[0, :6] = torch.tensor([float("inf"), float("-inf"), float("nan"), float("inf"), float("-inf"), float("nan")])
    rules = [{"prompt": [0, 1, 2], "made": [0, 1, 2, 9], "rep": 2.0, "freq": 0.5, "pres": 0.25, "bias": []}]
    ok = torch.ones((1, V), dtype=torch.bool)
    ok[0, 3:6] = False
    y = on_gpu(bq, rules, V, 8, 0)(x.cuda(), allowed=pack_bits(ok).cuda()).cpu()
    assert y[0, 0] == float("inf") and y[0, 1] == float("-inf") and bool(torch.isnan(y[0, 2]))
    assert bool((y[0, 3:6] == float("-inf")).all()) and float(y[0, 9]) == -0.75


def test_rules_that_say_little(bq):
    V = 3000
    x = torch.randn((2, V), generator=torch.Generator().manual_seed(2))
    assert torch.equal(bq.LogitRules(V, sequences=2)(x.cuda()).cpu(), x)
    ids = i32([[1, 2, 3], [4, 4, 4]]).cuda()
    y = bq.LogitRules(V, ids, i32([3, 3]).cuda(), frequency=torch.tensor([0.5, 0.5]).cuda())(x.cuda()).cpu()
    want = x.clone()
    want[0, [1, 2, 3]] -= 0.5
    want[1, 4] -= 1.5
    assert torch.equal(y, want)
    assert bq.LogitRules(V, sequences=2)(torch.empty((0, V), device="cuda")).shape == (0, V)


@pytest.mark.parametrize("cap", [1, 4096, 4097, 40000])
def test_long_histories(bq, cap):
    """One token again and again, and many tokens."""
    rng = random.Random(cap)
    V = 20000
    made = [123] * (cap // 2) + [rng.randint(0, V - 1) for _ in range(cap - cap // 2)]
    rules = [{"prompt": made[: cap // 4], "made": made[cap // 4:], "rep": 1.25, "freq": 0.0009765625, "pres": 0.5, "bias": []}]
    x = torch.randn((1, V), generator=torch.Generator().manual_seed(2))
    y = on_gpu(bq, rules, V, cap, 0)(x.cuda()).cpu()
    check(y, ref.logits(x.double(), rules, [(0, [])], V), x, 60.0, F32)


def test_biases_of_one_token_add_up_in_their_order(bq):
    """1e8, 1 and -1e8 in fp32: the order decides."""
    V, nb = 10000, 1024
    for order, want in (([1e8, 1.0, -1e8], 0.0), ([1e8, -1e8, 1.0], 1.0)):
        ids, vals = torch.full((1, nb), -1, dtype=torch.int32), torch.zeros((1, nb))
        for j, v in zip((5, 500, 1020), order):
            ids[0, j], vals[0, j] = 8500, v
        y = bq.LogitRules(V, bias_ids=ids.cuda(), bias_values=vals.cuda())(torch.zeros((1, V), device="cuda")).cpu()
        assert float(y[0, 8500]) == want and float(y.abs().sum()) == want
