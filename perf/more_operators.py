"""Cases, plain forms and 64-bit values of three operators of a step that decodes, or verifies a tree of drafted tokens:

  * append: RMSNorm of each query and key head, their rotation by position, and the keys' and values' way into a paged
    cache of 16-bit or INT8 values;
  * attend: attention of a few drafted tokens of each sequence over its cached tokens and over the drafts on their path;
  * logits: penalties for repeated tokens, biases and grammar masks on the rows of the vocabulary projection.

Definitions ("fp32" marks a value rounded once to 32 bits because an integer code hangs on it):

  tokens       sequence b has rows q_start[b] .. q_start[b + 1] - 1; its i-th row is cached at place ctx[b] + i, which is
               place % page_size of the page table[b][place / page_size]; rows behind the last sequence are left alone
  norm         S = fp32(sum x^2), r = 1 / sqrt(S / D + eps), x' = (x r) g, each step one fp32 operation
  rotation     of the first `rot` values of a head by (cos, sin) of its position, fp32 numbers of a table: pairs (i, i + rot / 2)
               or, interleaved, (2 i, 2 i + 1); a' = fp32(a c - b s), b' = fp32(b c + a s)
  INT8 cache   for each token and head s = fp32(max|x| / 127), q = clip(rint(fp32(x / s)), -127, 127); zeros have s = 0, q = 0
  attention    o = sum p v, p = softmax(scale q k) over places below ctx[b] and the drafts j whose bit the row's mask has
  logits       n: how often the row's sequence has generated v, the drafts on the row's path among it; seen: n > 0 or v in the
               prompt; l = l > 0 ? l / rep : l rep if seen; l - freq n - (n > 0 ? pres : 0) + bias; -inf unless v is allowed
"""
import random

import torch

own = False

EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "i8": torch.int8}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "i8": 1}


# ------------------------------------------------------------------ cases
def listed():
    base = {"Hq": 28, "Hkv": 4, "D": 128, "page": 64, "pad": 0}
    return [
        # the token of a decode step: latency
        {"name": "append 1 token", "op": "append", **base, "B": 1, "n": 1, "ctx": 4000, "spread": 0.0, "x": "f32", "cache": "bf16",
         "norm": False, "rot": 128, "layout": "half", "tree": False},
        # sixteen drafted tokens with normalized heads, into an INT8 cache
        {"name": "append 16 drafts int8", "op": "append", **base, "B": 1, "n": 16, "ctx": 2000, "spread": 0.0, "x": "f32",
         "cache": "i8", "norm": True, "rot": 128, "layout": "half", "tree": True},
        # prompts of eight sequences, heads of 256 of which a quarter rotates, as an INT8 linear gives them: bandwidth
        {"name": "append prompts", "op": "append", "Hq": 8, "Hkv": 1, "D": 256, "page": 32, "pad": 0, "B": 8, "n": 2047, "ctx": 1,
         "spread": 0.5, "x": "bf16", "cache": "f16", "norm": True, "rot": 64, "layout": "interleaved", "tree": False},
        # the token of a decode step over a short context: latency
        {"name": "attend 1 token", "op": "attend", **base, "B": 1, "n": 1, "ctx": 1000, "spread": 0.0, "cache": "bf16", "y": "f32",
         "tree": False},
        # sixteen drafted tokens of one sequence
        {"name": "attend 16 drafts", "op": "attend", **base, "B": 1, "n": 16, "ctx": 4096, "spread": 0.0, "cache": "bf16",
         "y": "f32", "tree": True},
        # five drafted tokens over a long INT8 cache, heads of 256
        {"name": "attend 5 drafts int8 long", "op": "attend", "Hq": 8, "Hkv": 1, "D": 256, "page": 16, "pad": 3, "B": 1, "n": 5,
         "ctx": 120001, "spread": 0.0, "cache": "i8", "y": "bf16", "tree": True},
        # one token over the longest context: the cache's bandwidth on one sequence
        {"name": "attend 1 token long", "op": "attend", **base, "B": 1, "n": 1, "ctx": 131071, "spread": 0.0, "cache": "bf16",
         "y": "f32", "tree": False},
        # a batch of decode streams of very different lengths
        {"name": "attend 64 streams", "op": "attend", **base, "B": 64, "n": 1, "ctx": 8190, "spread": 0.95, "cache": "f16",
         "y": "f16", "tree": False},
        # wide trees of eight sequences: arithmetic
        {"name": "attend 8 x 64 drafts", "op": "attend", **base, "B": 8, "n": 64, "ctx": 4000, "spread": 0.3, "cache": "bf16",
         "y": "bf16", "tree": True},
        # the logits of a decode step
        {"name": "logits 1 row", "op": "logits", "V": 152064, "S": 1, "n": 1, "history": 4096, "x": "f32", "bias": 40,
         "grammar": False, "tree": False, "pad": 0},
        # sixteen drafted tokens under a grammar
        {"name": "logits 16 drafts grammar", "op": "logits", "V": 152064, "S": 1, "n": 16, "history": 2000, "x": "f32", "bias": 0,
         "grammar": True, "tree": True, "pad": 0},
        # a large batch over the largest vocabulary: bandwidth
        {"name": "logits 200 streams", "op": "logits", "V": 262144, "S": 200, "n": 1, "history": 1500, "x": "f32", "bias": 17,
         "grammar": True, "tree": False, "pad": 1},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "logits"])
    if op == "logits":
        while True:
            c = {"op": op, "V": _log(rng, 1000, 262144), "S": _log(rng, 1, 200), "n": rng.choice([1, 1, rng.randint(2, 16)]),
                 "history": _log(rng, 1, 32768), "x": rng.choice(["f32", "f32", "bf16", "f16"]), "bias": rng.choice([0, rng.randint(1, 300)]),
                 "grammar": rng.random() < 0.5, "tree": False, "pad": rng.choice([0, 0, 2])}
            if c["S"] * c["n"] * c["V"] <= 200 * 262144 and c["S"] * c["n"] * c["history"] <= 400000:
                break
        c["tree"] = c["n"] > 1
        return c
    while True:
        D = rng.choice([64, 128, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        c = {"op": op, "Hq": Hkv * rng.randint(1, 8), "Hkv": Hkv, "D": D, "page": rng.choice([16, 32, 64, 128, 256]),
             "pad": rng.choice([0, 0, rng.randint(1, 5)]), "B": _log(rng, 1, 64), "cache": rng.choice(["bf16", "f16", "i8"])}
        if op == "append":
            c |= {"n": _log(rng, 1, 4096), "ctx": _log(rng, 1, 20000), "spread": round(rng.random(), 3),
                  "x": rng.choice(["f32", "bf16", "f16"]), "norm": rng.random() < 0.5,
                  "rot": rng.choice([D, D, D // 2, D // 4]), "layout": rng.choice(["half", "half", "interleaved"])}
            c["tree"] = 1 < c["n"] <= 64 and rng.random() < 0.7
            if c["B"] * c["n"] * (c["Hq"] + 2 * Hkv) * D <= 8 * 2047 * 2560 and c["B"] * (c["ctx"] + c["n"]) * Hkv * D <= 6e7:
                return c
            continue
        c |= {"n": rng.choice([1, 1, rng.randint(2, 16), rng.randint(2, 64)]), "ctx": _log(rng, 1, 131071),
              "spread": round(rng.random(), 3), "y": rng.choice(["f32", "bf16", "f16"])}
        c["tree"] = c["n"] > 1 and rng.random() < 0.8
        tokens = c["B"] * c["ctx"]
        if tokens * Hkv * D <= 64 * 4300 * 512 and tokens * c["n"] * c["Hq"] * D <= 8 * 64 * 28 * 128 * 3400:
            return c


def _lengths(c):
    """Rows and cached tokens of each sequence: the first has the case's numbers, the others up to `spread` less."""
    less = [(0.618034 * b) % 1.0 for b in range(c["B"])]
    ns = [max(1, c["n"] - int(c["spread"] * f * c["n"])) for f in less]
    return ns, [max(0, c["ctx"] - int(c["spread"] * f * c["ctx"])) for f in less]


def work(c):
    if c["op"] == "logits":
        R, V = c["S"] * c["n"], c["V"]
        b = R * V * 2 * BYTES[c["x"]] + (R * ((V + 31) // 32) * 4 if c["grammar"] else 0) + c["S"] * (4 * c["history"] + 8 * c["bias"] + 20)
        return {"bytes": b, "flops": 3 * R * V}
    ns, ctx = _lengths(c)
    T, Hq, Hkv, D = sum(ns), c["Hq"], c["Hkv"], c["D"]
    kv = 2 * Hkv * (D * BYTES[c["cache"]] + 4 * (c["cache"] == "i8"))       # a cached token
    if c["op"] == "append":
        b = T * ((Hq + 2 * Hkv) * D * BYTES[c["x"]] + 4 * c["rot"] + 2 * Hq * D + kv)
        return {"bytes": b + 8 * D * c["norm"], "flops": T * (Hq + Hkv) * (3 * c["rot"] + 5 * D * c["norm"])}
    b = sum(n + x for n, x in zip(ns, ctx)) * kv + T * Hq * D * (2 + BYTES[c["y"]])
    return {"bytes": b, "flops": sum(4 * D * Hq * n * (x + n / 2) for n, x in zip(ns, ctx))}


# ----------------------------------------------------------------- inputs
def _tree(rng, n, tree):
    """Masks (bit j: row j is on the row's path, the row's own bit set) and depths of a drafted tree, or of a chain."""
    masks, depth = [], []
    for i in range(n):
        p = i - 1 if not tree else (rng.randint(max(-1, i - 4), i - 1) if i else -1)
        masks.append((masks[p] if p >= 0 else 0) | 1 << i)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return [m - (1 << 64) if m >> 63 else m for m in masks], depth


def _device(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype).cuda()


def _starts(ns):
    s = [0]
    for n in ns:
        s.append(s[-1] + n)
    return s


def _inputs(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = random.Random(int(seed))
    randn = lambda *s, dtype=torch.float32: torch.randn(*s, generator=gen, device="cuda", dtype=dtype)  # noqa: E731
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda")                                      # noqa: E731
    d = {}
    if c["op"] == "logits":
        S, n, V = c["S"], c["n"], c["V"]
        R = S * n + c["pad"]
        d["logits"] = (2.5 * randn(R, V)).to(TYPES[c["x"]])
        d["ids"] = (rand(S, c["history"]) ** 3 * V).int()                   # frequent tokens have low numbers
        less = [(0.618034 * s) % 1.0 for s in range(S)]
        length = [c["history"] - int(0.5 * f * c["history"]) for f in less]
        d["length"], d["prompt"] = _device(length), _device([int(v * 0.6) for v in length])
        d["rep"], d["freq"], d["pres"] = 1.0 + 0.3 * rand(S), 0.5 * rand(S), 0.5 * rand(S)
        if c["bias"]:
            d["bias_ids"] = (rand(S, c["bias"]) * V).int()
            d["bias_values"] = 2.0 * randn(S, c["bias"])
        if c["grammar"]:                                                    # a digit, an identifier, nearly everything
            share = 0.001 ** rand(R, 1)
            bits = torch.zeros(R, (V + 31) // 32 * 32, dtype=torch.bool, device="cuda")
            bits[:, :V] = rand(R, V) < share
            weight = torch.ones(32, dtype=torch.int64, device="cuda") << torch.arange(32, device="cuda")
            d["allowed"] = (bits.view(R, -1, 32) * weight).sum(-1).to(torch.int32)
        if c["tree"]:
            d["drafts"] = (rand(R) ** 3 * V).int()
            d["row_start"] = _device(_starts([n] * S))
            d["mask"] = _device([m for _ in range(S) for m in _tree(rng, n, True)[0]] + [0] * c["pad"], torch.int64)
        return d
    ns, ctx = _lengths(c)
    B, T, Hq, Hkv, D, page = c["B"], sum(ns), c["Hq"], c["Hkv"], c["D"], c["page"]
    R = T + c["pad"]
    d["ctx"], d["q_start"] = _device(ctx), _device(_starts(ns))
    need = [(x + n + page - 1) // page for x, n in zip(ctx, ns)]
    pages = sum(need) + max(2, sum(need) // 16)
    free = torch.randperm(pages, generator=gen, device="cuda").int()
    d["table"] = torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        d["table"][b, :k] = free[at : at + k]
        at += k
    shape = (pages, Hkv, page, D)
    if c["cache"] == "i8":
        for t in "kv":
            d[t] = torch.randint(-127, 128, shape, generator=gen, device="cuda", dtype=torch.int8)
            d[t + "_scale"] = 0.03 * (0.5 + rand(*shape[:3]))
    else:
        d["k"], d["v"] = randn(*shape, dtype=TYPES[c["cache"]]), randn(*shape, dtype=TYPES[c["cache"]])
    trees = [_tree(rng, n, c["tree"]) for n in ns] if c["tree"] or c["op"] == "append" else []
    d["mask"] = _device([m for t in trees for m in t[0]] + [0] * c["pad"], torch.int64) if c["tree"] else None
    if c["op"] == "attend":
        qtype = "bf16" if c["cache"] == "i8" else c["cache"]
        d["q"] = (1.5 * randn(R, Hq, D)).to(TYPES[qtype])
        d["out"] = torch.zeros(R, Hq, D, dtype=TYPES[c["y"]], device="cuda")
        return d
    d["qkv"] = (3.0 * randn(R, (Hq + 2 * Hkv) * D)).to(TYPES[c["x"]])
    d["pos"] = _device([x + k for x, t in zip(ctx, trees) for k in t[1]] + [0] * c["pad"])
    angle = torch.arange(max(ctx) + max(ns), dtype=torch.float64, device="cuda")[:, None] * (
        1e6 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"]))
    d["turns"] = torch.stack([angle.cos(), angle.sin()], -1).float()        # [positions, rot / 2, 2]
    if c["norm"]:
        d["q_norm"], d["k_norm"] = 1 + 0.2 * randn(D), 1 + 0.2 * randn(D)
    d["out"] = torch.zeros(R, Hq, D, dtype=TYPES["bf16" if c["cache"] == "i8" else c["cache"]], device="cuda")
    return d


def prepare(case, seed):
    st = {"case": case, **_inputs(case, seed)}
    if case["op"] == "logits":
        st["out"] = torch.zeros_like(st["logits"])
    if own:
        import bit_quantized_decode_gb300 as bq
        if case["op"] == "logits":
            st["rules"] = bq.LogitRules(case["V"], st["ids"], st["length"], st["prompt"], repetition=st["rep"],
                                        frequency=st["freq"], presence=st["pres"], bias_ids=st.get("bias_ids"),
                                        bias_values=st.get("bias_values"))
            return st
        ns, _ = _lengths(case)
        cache = bq.KVCache(st["k"], st["v"], st.get("k_scale"), st.get("v_scale"))
        rope = bq.RopeTable(st["turns"], case["layout"]) if case["op"] == "append" else None
        st["cache"] = cache
        st["op"] = bq.CachedAttention(cache, case["Hq"], rope=rope, q_norm=st.get("q_norm"), k_norm=st.get("k_norm"), eps=EPS)
        st["batch"] = bq.KVBatch(st["table"], st["ctx"], st["q_start"], max_tokens=max(ns))
        if case["op"] == "attend":
            st["workspace"] = st["op"].workspace(sum(ns) + case["pad"], st["batch"])
    return st


# ------------------------------------------------------------ plain forms
def _places(st):
    """Sequence, row within it, page and place in the page of every row of a sequence."""
    c = st["case"]
    T = sum(_lengths(c)[0])
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(st["q_start"], t, right=True) - 1
    i = t - st["q_start"][b]
    place = st["ctx"][b] + i
    return T, b, i, st["table"][b, (place // c["page"]).long()].long(), (place % c["page"]).long()


def _norm(x, g):
    one = lambda t: t.float().double()                                       # noqa: E731
    S = one(x.double().square().sum(-1, keepdim=True))
    r = one(1.0 / one(torch.sqrt(one(one(S / x.shape[-1]) + torch.tensor(EPS, device=x.device).double()))))
    return (x * r.float()) * g


def _turn(x, turns, layout):
    """x [T, heads, D] rotated by turns [T, rot / 2, 2]: the products in 64 bits, rounded once."""
    half = turns.shape[1]
    cos, sin = turns[:, None, :, 0].double(), turns[:, None, :, 1].double()
    head, rest = x[..., : 2 * half].double(), x[..., 2 * half :]
    if layout == "half":
        a, b = head[..., :half], head[..., half:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = head[..., 0::2], head[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([y.float(), rest], -1)


def _codes(x):
    s = (x.abs().amax(-1, keepdim=True).double() / 127.0).float()
    q = (x.double() / s.double()).float().round().clamp(-127, 127)
    return torch.where(s > 0, q, torch.zeros_like(q)).to(torch.int8), s[..., 0]


def _append(st):
    c = st["case"]
    T, b, i, page, off = _places(st)
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    x = st["qkv"][:T].float().view(T, Hq + 2 * Hkv, D)
    q, k, v = x[:, :Hq], x[:, Hq : Hq + Hkv], x[:, Hq + Hkv :]
    if c["norm"]:
        q, k = _norm(q, st["q_norm"]), _norm(k, st["k_norm"])
    turns = st["turns"][st["pos"][:T].long()]
    q, k = _turn(q, turns, c["layout"]), _turn(k, turns, c["layout"])
    st["out"][:T] = q.to(st["out"].dtype)
    if c["cache"] == "i8":
        st["k"][page, :, off], st["k_scale"][page, :, off] = _codes(k)
        st["v"][page, :, off], st["v_scale"][page, :, off] = _codes(v)
        return {"q": st["out"], "k": st["k"].float() * st["k_scale"][..., None], "v": st["v"].float() * st["v_scale"][..., None]}
    st["k"][page, :, off], st["v"][page, :, off] = k.to(st["k"].dtype), v.to(st["v"].dtype)
    return {"q": st["out"], "k": st["k"], "v": st["v"]}


def _attend(st):
    c = st["case"]
    ns, ctx = _lengths(c)
    B, n, Hq, Hkv, D = c["B"], max(ns), c["Hq"], c["Hkv"], c["D"]
    T, b, i, _, _ = _places(st)
    table = st["table"].clamp(min=0).long()

    def cached(t):                                           # [B, Hkv, places, D]
        x = st[t][table].float()                             # [B, pages, Hkv, page, D]
        if c["cache"] == "i8":
            x = x * st[t + "_scale"][table][..., None]
        return x.transpose(1, 2).reshape(B, Hkv, -1, D)

    k, v = cached("k"), cached("v")
    L = k.shape[2]
    place = torch.arange(L, device="cuda")
    late = place[None, :] - st["ctx"][:, None]               # [B, L]: which draft a place holds
    v = torch.where((late < (st["q_start"][1:] - st["q_start"][:-1])[:, None])[:, None, :, None], v, torch.zeros_like(v))
    mask = st["mask"][:T] if c["tree"] else (torch.full_like(i, 2, dtype=torch.int64) << i) - 1
    sees = torch.zeros(B, n, L, dtype=torch.bool, device="cuda")
    j = late[b]
    sees[b, i] = (j < 0) | ((j >= 0) & (j < 64) & ((mask[:, None] >> j.clamp(0, 63)) & 1).bool())
    q = torch.zeros(B, n, Hq, D, device="cuda")
    q[b, i] = st["q"][:T].float()
    q = q.view(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    s = (q @ k.transpose(2, 3)).mul_(D ** -0.5).view(B, Hkv, Hq // Hkv, n, L)
    s.masked_fill_(~sees[:, None, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top > float("-inf"), top, torch.zeros_like(top))).exp_()
    p /= p.sum(-1, keepdim=True).clamp(min=1e-30)
    y = (p.view(B, Hkv, -1, L) @ v).view(B, Hkv, Hq // Hkv, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    st["out"][:T] = y[b, i].to(st["out"].dtype)
    return st["out"]


def _logits(st):
    c = st["case"]
    S, n, V = c["S"], c["n"], c["V"]
    R = S * n
    x = st["logits"][:R].float()
    place = torch.arange(c["history"], device="cuda")[None, :]
    inside = place < st["length"][:, None]
    made = inside & (place >= st["prompt"][:, None])
    count = torch.zeros(S, V, device="cuda").scatter_add_(1, st["ids"].long(), made.float())
    seen = torch.zeros(S, V, device="cuda").scatter_add_(1, st["ids"].long(), inside.float())
    if c["tree"]:
        path = ((st["mask"][:R, None] >> torch.arange(n, device="cuda")) & 1).float()            # [R, n]
        ids = st["drafts"][:R].long().view(S, 1, n).expand(S, n, n).reshape(R, n)
        count, seen = (t.repeat_interleave(n, 0).scatter_add_(1, ids, path) for t in (count, seen))
    of = lambda t: t.repeat_interleave(n, 0)[:, None]                        # noqa: E731
    x = torch.where(seen > 0, torch.where(x > 0, x / of(st["rep"]), x * of(st["rep"])), x)
    x = x - of(st["freq"]) * count - of(st["pres"]) * (count > 0)
    if c["bias"]:
        x = x + torch.zeros(S, V, device="cuda").scatter_add_(1, st["bias_ids"].long(), st["bias_values"]).repeat_interleave(n, 0)
    if c["grammar"]:
        bits = (st["allowed"][:R, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        x = x.masked_fill(bits.view(R, -1)[:, :V] == 0, float("-inf"))
    st["out"][:R] = x.to(st["out"].dtype)
    return st["out"]


def run(st):
    c = st["case"]
    if own:
        if c["op"] == "logits":
            tree = {"drafts": st["drafts"], "row_start": st["row_start"], "mask": st["mask"]} if c["tree"] else {}
            return st["rules"](st["logits"], st["out"], allowed=st.get("allowed"), **tree)
        if c["op"] == "attend":
            return st["op"].attend(st["q"], st["batch"], st["mask"], st["out"], st["workspace"])
        q = st["op"].append(st["qkv"], st["batch"], st["pos"], st["out"])
        if c["cache"] == "i8":
            return {"q": q, "k": st["cache"].values("k"), "v": st["cache"].values("v")}
        return {"q": q, "k": st["k"], "v": st["v"]}
    return {"append": _append, "attend": _attend, "logits": _logits}[c["op"]](st)


# -------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    """The definition, one sequence after the other, in 64 bits but for what it rounds to 32."""
    d = _inputs(case, seed)
    one = lambda t: t.to(torch.float32).to(torch.float64)                    # noqa: E731
    if case["op"] == "logits":
        Y = torch.zeros_like(d["logits"], dtype=torch.float64)
        S, n, V = case["S"], case["n"], case["V"]
        for s in range(S):
            length, prompt = int(d["length"][s]), int(d["prompt"][s])
            count = torch.bincount(d["ids"][s, prompt:length], minlength=V)
            asked = torch.bincount(d["ids"][s, :prompt], minlength=V)
            add = torch.zeros(V, dtype=torch.float64, device="cuda")
            if case["bias"]:
                add.index_put_((d["bias_ids"][s].long(),), d["bias_values"][s].double(), accumulate=True)
            rep, freq, pres = (float(d[k][s]) for k in ("rep", "freq", "pres"))
            for r in range(s * n, s * n + n):
                made = count
                if case["tree"]:
                    m = int(d["mask"][r])
                    path = [int(d["drafts"][s * n + j]) for j in range(n) if m >> j & 1]
                    made = count + torch.bincount(torch.tensor(path, device="cuda"), minlength=V)
                x = d["logits"][r].double()
                known = (made + asked) > 0
                x[known] = torch.where(x[known] > 0, x[known] / rep, x[known] * rep)
                x = x - freq * made.double() - pres * (made > 0).double() + add
                if case["grammar"]:
                    v = torch.arange(V, device="cuda")
                    ok = (d["allowed"][r][v // 32].long() >> (v % 32)) & 1
                    x[ok == 0] = -torch.inf
                Y[r] = x
        return Y
    ns, ctx = _lengths(case)
    starts = _starts(ns)
    Hq, Hkv, D, page = case["Hq"], case["Hkv"], case["D"], case["page"]
    table = d["table"].tolist()
    if case["op"] == "attend":
        if sum(n * x for n, x in zip(ns, ctx)) * Hq * D > 8e9:
            return None
        Y = torch.zeros(d["out"].shape, dtype=torch.float64, device="cuda")
        for b, (n, x) in enumerate(zip(ns, ctx)):
            used = torch.tensor(table[b][: (x + n + page - 1) // page], device="cuda")
            K, W = (d[t][used].double() * (d[t + "_scale"][used].double()[..., None] if case["cache"] == "i8" else 1.0) for t in "kv")
            K, W = (t.permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, : x + n] for t in (K, W))
            for i in range(n):
                m = int(d["mask"][starts[b] + i]) if case["tree"] else (2 << i) - 1
                keep = list(range(x)) + [x + j for j in range(n) if m >> j & 1]
                keep = slice(0, x + i + 1) if len(keep) == x + i + 1 else torch.tensor(keep, device="cuda")
                q = d["q"][starts[b] + i].double().view(Hkv, -1, D)
                s = torch.einsum("hgd,hld->hgl", q, K[:, keep]) / D ** 0.5
                w = torch.exp(s - torch.logsumexp(s, -1, keepdim=True))
                Y[starts[b] + i] = torch.einsum("hgl,hld->hgd", w, W[:, keep]).reshape(Hq, D)
        return Y
    T = sum(ns)
    X = d["qkv"][:T].double().view(T, Hq + 2 * Hkv, D)
    part = {"q": X[:, :Hq], "k": X[:, Hq : Hq + Hkv], "v": X[:, Hq + Hkv :]}
    turns = d["turns"][d["pos"][:T].long()].double()
    for t in "qk":
        Z = part[t].clone()
        if case["norm"]:
            mean = one(one((Z * Z).sum(-1, keepdim=True)) / D)
            r = one(one(mean + one(torch.tensor(EPS, dtype=torch.float64, device="cuda"))).sqrt()).reciprocal()
            Z = one(one(Z * one(r)) * d[t + "_norm"].double())
        half = case["rot"] // 2
        lo = slice(0, half) if case["layout"] == "half" else slice(0, 2 * half, 2)
        hi = slice(half, 2 * half) if case["layout"] == "half" else slice(1, 2 * half, 2)
        a, b = Z[..., lo].clone(), Z[..., hi].clone()
        z = torch.complex(a, b) * torch.complex(turns[..., 0], turns[..., 1])[:, None]
        Z[..., lo], Z[..., hi] = z.real, z.imag
        part[t] = Z
    Q = torch.zeros(d["out"].shape, dtype=torch.float64, device="cuda")
    Q[:T] = part["q"]
    at = [(table[b][p // page], p % page) for b, (n, x) in enumerate(zip(ns, ctx)) for p in range(x, x + n)]
    pg, off = (torch.tensor(v, device="cuda") for v in zip(*at))
    got = {"q": Q}
    for t in "kv":
        C = d[t].double()
        Z = one(part[t])
        if case["cache"] == "i8":
            C = C * d[t + "_scale"].double()[..., None]
            s = one(Z.abs().amax(-1, keepdim=True) / 127)
            Z = torch.where(s > 0, torch.clip(torch.round(one(Z / s)), -127, 127), torch.zeros_like(Z)) * s
        else:
            Z = part[t]
        C[pg, :, off] = Z
        got[t] = C
    return got
