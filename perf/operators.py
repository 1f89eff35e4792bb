"""Cases, plain forms and 64-bit values of three operators of a decoder with integer weights:

  * the INT8 x INT8 linear with a scale for each token and each output channel, from one token to a long prompt;
  * the router of a mixture-of-experts layer (RMSNorm, scores, the top experts and their weights) for a few tokens;
  * the whole mixture-of-experts layer for a few tokens: the router, the experts' gated MLP on INT4 or INT8 weights
    and INT8 activations, and the weighted sum.

Definitions (q rounds half to even; "fp32" marks a value rounded once to 32 bits because an integer code or a choice
of experts hangs on it):

  RMSNorm      S = fp32(sum x^2), r = 1 / sqrt(S / K + eps), x' = (x r) g, each step one fp32 operation
  codes        s = fp32(max|x| / 127), q = clip(rint(fp32(x / s)), -127, 127); a zero token has s = 0, q = 0
  linear       y = fma(fp32(s_w s_x), sum q_w q_x, b) (+ residual), the integer sum exact
  router       l = fp32(sum x' w); softmax: the top experts by l, p = softmax(l) over all experts;
               sigmoid: the top experts by fp32(p + selection bias), p = fp32(1 / (1 + exp(-l)));
               ties to the lowest index; weights p, divided by their sum if asked, times the scale
  experts      h = fp32(act(g) u) from the linear's fp32 g and u; codes of h; d = the linear of h;
               y = sum over the chosen experts of weight * d, plus the shared experts' d (+ residual)
"""
import torch

own = False

EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode token through the fused q/k/v projection, the norm in front: latency
        {"name": "linear 1 token qkv", "op": "linear", "M": 1, "N": 4608, "K": 3584, "x": "f32", "y": "f32", "bias": True,
         "norm": True, "residual": False},
        # sixteen drafted tokens verified by the vocabulary projection: weight bandwidth
        {"name": "linear 16 tokens lm_head", "op": "linear", "M": 16, "N": 152064, "K": 3584, "x": "f32", "y": "f32",
         "bias": False, "norm": False, "residual": False},
        # a batch of 64 decode streams through the down projection: few rows, a long K
        {"name": "linear 64 tokens down", "op": "linear", "M": 64, "N": 3584, "K": 18944, "x": "bf16", "y": "bf16",
         "bias": False, "norm": False, "residual": False},
        # a short prompt of odd length through the output projection, added to the residual stream
        {"name": "linear 333 tokens o", "op": "linear", "M": 333, "N": 3584, "K": 3584, "x": "f16", "y": "f32",
         "bias": True, "norm": False, "residual": True},
        # a prompt of a small model through its q/k/v projection
        {"name": "linear 1000 tokens small qkv", "op": "linear", "M": 1000, "N": 2560, "K": 1536, "x": "f32", "y": "f16",
         "bias": False, "norm": True, "residual": False},
        # a long prompt through the fused gate/up projection: arithmetic
        {"name": "linear 4096 tokens gate/up", "op": "linear", "M": 4096, "N": 37888, "K": 3584, "x": "bf16",
         "y": "bf16", "bias": False, "norm": False, "residual": False},
        # the choice of 8 of 64 experts for one token
        {"name": "route 1 token", "op": "route", "M": 1, "K": 3584, "E": 64, "top_k": 8, "score": "softmax",
         "renormalize": True, "x": "f32"},
        # the choice of 6 of 256 experts by sigmoid scores with a selection bias for a verified draft
        {"name": "route 16 tokens sigmoid", "op": "route", "M": 16, "K": 1536, "E": 256, "top_k": 6, "score": "sigmoid",
         "renormalize": True, "x": "bf16"},
        # one token of a small layer: latency
        {"name": "moe 1 token small", "op": "moe", "fmt": "w4", "M": 1, "H": 1536, "I": 768, "E": 32, "shared": 0,
         "top_k": 4, "act": "gelu_tanh", "score": "softmax", "renormalize": True, "x": "f32", "y": "f32", "residual": True},
        # one token of a large layer: the chosen experts' weights
        {"name": "moe 1 token", "op": "moe", "fmt": "w4", "M": 1, "H": 3584, "I": 2368, "E": 64, "shared": 0,
         "top_k": 8, "act": "silu", "score": "softmax", "renormalize": True, "x": "f32", "y": "f32", "residual": True},
        # sixteen tokens of it: nearly every expert is read
        {"name": "moe 16 tokens", "op": "moe", "fmt": "w4", "M": 16, "H": 3584, "I": 2368, "E": 64, "shared": 0,
         "top_k": 8, "act": "silu", "score": "softmax", "renormalize": True, "x": "f32", "y": "f32", "residual": True},
        # five tokens, INT8 experts, one expert shared by all tokens, sigmoid scores
        {"name": "moe 5 tokens int8 shared", "op": "moe", "fmt": "w8", "M": 5, "H": 1536, "I": 768, "E": 128, "shared": 1,
         "top_k": 6, "act": "silu", "score": "sigmoid", "renormalize": True, "x": "bf16", "y": "bf16", "residual": False},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _log32(rng, lo, hi):
    return max(lo, min(hi, 32 * ((_log(rng, lo, hi) + 16) // 32)))


def draw(rng):
    op = rng.choice(["linear", "linear", "route", "moe", "moe"])
    if op == "linear":
        while True:
            M, N, K = _log(rng, 1, 4096), _log(rng, 500, 152064), _log32(rng, 512, 18944)
            if M * N * K <= 4096 * 37888 * 3584 and M * N <= 4096 * 37888 and N * K <= 152064 * 3584:
                break
        y = rng.choice(["f32", "bf16", "f16"])
        return {"op": "linear", "M": M, "N": N, "K": K, "x": rng.choice(["f32", "bf16", "f16"]), "y": y,
                "bias": rng.random() < 0.5, "norm": rng.random() < 0.4, "residual": y == "f32" and rng.random() < 0.5}
    score = rng.choice(["softmax", "softmax", "sigmoid"])
    if op == "route":
        E = _log(rng, 8, 256)
        return {"op": "route", "M": rng.randint(1, 16), "K": _log32(rng, 512, 7168), "E": E, "top_k": rng.randint(1, 8),
                "score": score, "renormalize": rng.random() < 0.7, "x": rng.choice(["f32", "bf16", "f16"])}
    E = _log(rng, 8, 64)
    t = rng.choice(["f32", "bf16", "f16"])
    y = rng.choice([t, "f32"])
    return {"op": "moe", "fmt": rng.choice(["w4", "w4", "w8"]), "M": rng.randint(1, 16), "H": _log32(rng, 512, 3584),
            "I": _log32(rng, 256, 2368), "E": E, "shared": rng.choice([0, 0, 1, 2]), "top_k": rng.randint(1, 8),
            "act": rng.choice(["silu", "silu", "gelu_tanh"]), "score": score, "renormalize": rng.random() < 0.7, "x": t,
            "y": y, "residual": y == "f32" and rng.random() < 0.5}


def work(c):
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        b = N * K + 4 * N * (1 + c["bias"]) + M * K * BYTES[c["x"]] + M * N * (BYTES[c["y"]] + 4 * c["residual"])
        return {"bytes": b + 4 * K * c["norm"], "flops": 2 * M * N * K}
    if c["op"] == "route":
        M, K, E = c["M"], c["K"], c["E"]
        return {"bytes": 4 * E * K + 4 * K + M * K * BYTES[c["x"]] + 8 * M * c["top_k"], "flops": 2 * M * E * K}
    M, H, I, E, k = c["M"], c["H"], c["I"], c["E"], c["top_k"]
    read = E * (1 - (1 - k / E) ** M) + c["shared"]          # distinct experts, were every choice alike
    per = 3 * H * I * (0.5 if c["fmt"] == "w4" else 1) + 4 * (2 * I + H)
    return {"bytes": read * per + 4 * E * H + 4 * H + M * H * (BYTES[c["x"]] + BYTES[c["y"]] + 4 * c["residual"]),
            "flops": 2 * M * (k + c["shared"]) * 3 * H * I + 2 * M * E * H}


# ----------------------------------------------------------------- inputs
def _rows(shape, sigma, top, gen):
    """Weights N(0, sigma) as symmetric integer codes and a scale for each row: what a loader has quantized."""
    w = torch.randn(shape, generator=gen, device="cuda").mul_(sigma)
    s = w.abs().amax(-1) / torch.full((), float(top), device="cuda")
    return (w / s[..., None]).round_().clamp_(-top, top).to(torch.int8), s


def _norm_weight(K, gen):
    g = 1 + 0.1 * torch.randn(K, generator=gen, device="cuda")
    g[torch.randint(0, K, (max(1, K // 200),), generator=gen, device="cuda")] *= 8.0
    return g


def _inputs(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    d = {}
    K = c["H"] if c["op"] == "moe" else c["K"]
    x = 4.0 * randn(c["M"], K)
    if c["op"] == "linear" and not c["norm"]:
        x[randn(c["M"], K) > 3.1] *= 5.0                     # about one value in a thousand is an outlier
    d["x"] = x.to(TYPES[c["x"]])
    if c["op"] != "linear" or c["norm"]:
        d["norm"] = _norm_weight(K, gen)
    if c["op"] == "linear":
        d["w"], d["s_w"] = _rows((c["N"], K), 0.02, 127, gen)
        d["bias"] = 0.01 * randn(c["N"]) if c["bias"] else None
        d["residual"] = 4.0 * randn(c["M"], c["N"]) if c["residual"] else None
        return d
    E = c["E"]
    d["router"] = 0.02 * randn(E, K)
    d["select"] = 0.05 * randn(E) if c["score"] == "sigmoid" else None
    d["scale"] = 2.5 if c["score"] == "sigmoid" else 1.0
    if c["op"] == "moe":
        H, I, n, top = c["H"], c["I"], E + c["shared"], 7 if c["fmt"] == "w4" else 127
        parts = [(_rows((2 * I, H), 0.02, top, gen), _rows((H, I), 0.02, top, gen)) for _ in range(n)]
        d["gu"], d["s_gu"] = (torch.stack([p[0][j] for p in parts]) for j in (0, 1))
        d["dn"], d["s_dn"] = (torch.stack([p[1][j] for p in parts]) for j in (0, 1))
        d["residual"] = 4.0 * randn(c["M"], H) if c["residual"] else None
    return d


def _words(q):
    """INT4 codes as the words that a loader stores: eight to an int32, the first in the lowest bits."""
    return ((q[..., 0::2] & 15) | (q[..., 1::2] << 4)).view(torch.int32)


def prepare(case, seed):
    st = {"case": case, **_inputs(case, seed)}
    if own:
        import bit_quantized_decode_gb300 as bq
        M = case["M"]
        if case["op"] == "linear":
            bias = None if st["bias"] is None else [st["bias"]]
            lin = bq.QuantLinear.from_canonical("w8", [st.pop("w")], case["K"], [st.pop("s_w")], bias, keep_canonical=False)
            st["linear"], st["buffers"], st["workspace"] = lin, lin.buffers(M, TYPES[case["y"]]), lin.workspace(M)
            return st
        router = bq.MoeRouter(st["router"], case["top_k"], select_bias=st["select"], score=case["score"],
                              renormalize=case["renormalize"], scale=st["scale"], norm=st["norm"], eps=EPS)
        if case["op"] == "route":
            st["op"], st["buffers"] = router, router.buffers(M)
            return st
        stored = _words if case["fmt"] == "w4" else lambda q: q  # noqa: E731
        layer = bq.MoeLayer.from_canonical(case["fmt"], router, stored(st.pop("gu")), st.pop("s_gu"), stored(st.pop("dn")),
                                           st.pop("s_dn"), act=case["act"], n_shared=case["shared"])
        st["op"], st["buffers"] = layer, layer.buffers(M, TYPES[case["y"]])
    return st


# ------------------------------------------------------------ plain forms
def _f32(v):
    return v.float().double()


def _norm(x, g, K):
    S = _f32(x.double().square().sum(-1, keepdim=True))
    r = _f32(1.0 / _f32(torch.sqrt(_f32(_f32(S / K) + torch.tensor(EPS, device=x.device).double()))))
    return (x * r.float()) * g


def _codes(x):
    """INT8 codes (as floats) and the scale of each row of an fp32 tensor."""
    s = (x.abs().amax(-1, keepdim=True).double() / 127.0).float()
    q = (x.double() / s.double()).float().round().clamp(-127, 127)
    return torch.where(s > 0, q, torch.zeros_like(q)), s


def _dequant(acc, s_w, s_x, bias):
    y = (s_w * s_x).double() * acc.double()
    return (y if bias is None else y + bias.double()).float()


def _route(st, x):
    """Experts, weights of the tokens x (already normalised)."""
    c = st["case"]
    logit = (x.double() @ st["router"].double().T).float()
    if c["score"] == "softmax":
        p = torch.exp(logit - logit.amax(-1, keepdim=True))
        p, key = p / p.sum(-1, keepdim=True), logit
    else:
        p = (1 / (1 + torch.exp(-logit.double()))).float()
        key = p + st["select"]
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, : c["top_k"]]
    w = p.gather(1, ids)
    if c["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.to(torch.int32), w * st["scale"]


def _experts(st, q, s, ids):
    """The chosen (and the shared) experts' outputs [M, slots, H] for codes q [M, H] and scales s [M, 1]."""
    c = st["case"]
    M, I, n = c["M"], c["I"], c["shared"]
    every = torch.arange(c["E"], c["E"] + n, device=q.device).expand(M, n)
    e = torch.cat([ids.long(), every], 1)                    # [M, slots]
    slots = e.shape[1]
    e = e.reshape(-1)
    a = torch.bmm(st["gu"][e].float(), q.repeat_interleave(slots, 0)[:, :, None])[:, :, 0]
    gu = _dequant(a, st["s_gu"][e], s.repeat_interleave(slots, 0), None).double()
    g, u = gu[:, :I], gu[:, I:]
    if c["act"] == "silu":
        h = (g / (1 + torch.exp(-g)) * u).float()
    else:
        z = 0.7978845608028654 * (g + 0.044715 * g * g * g)
        h = (g / (1 + torch.exp(-2 * z)) * u).float()        # g / 2 (1 + tanh z) u
    qh, sh = _codes(h)
    a = torch.bmm(st["dn"][e].float(), qh[:, :, None])[:, :, 0]
    return _dequant(a, st["s_dn"][e], sh, None).reshape(M, slots, c["H"])


def run(st):
    c = st["case"]
    if own:
        if c["op"] == "linear":
            b = st["buffers"]
            return st["linear"](st["x"], *b, norm=st.get("norm"), eps=EPS, residual=st["residual"], workspace=st["workspace"])
        if c["op"] == "route":
            ids, weights = st["op"](st["x"], st["buffers"])
            return {"ids": ids, "weights": weights}
        b = st["buffers"]
        y = st["op"](st["x"], b, residual=st["residual"])
        return {"y": y, "ids": b.ids, "weights": b.weights}
    x = st["x"].float()
    if "norm" in st:
        x = _norm(x, st["norm"], x.shape[1])
    if c["op"] == "linear":
        q, s = _codes(x)
        y = _dequant(q @ st["w"].float().T, st["s_w"][None, :], s, st["bias"])
        if st["residual"] is not None:
            y = st["residual"] + y
        return y.to(TYPES[c["y"]])
    ids, weights = _route(st, x)
    if c["op"] == "route":
        return {"ids": ids, "weights": weights}
    q, s = _codes(x)
    d = _experts(st, q, s, ids)
    w = torch.cat([weights, torch.ones(c["M"], c["shared"], device=x.device)], 1)
    y = (d * w[:, :, None]).sum(1)
    if st["residual"] is not None:
        y = st["residual"] + y
    return {"y": y.to(TYPES[c["y"]]), "ids": ids, "weights": weights}


# -------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    """The definition, one row at a time where rows choose their weights; each value in 64 bits but for those that the
    definition rounds to 32 because codes or choices are taken from them."""
    d = _inputs(case, seed)
    one = lambda t: t.to(torch.float32).to(torch.float64)  # noqa: E731
    X = d["x"].double()
    if "norm" in d:
        n = X.shape[1]
        rows = []
        for v in X:
            mean = one(one((v * v).sum()) / n)
            r = one(one(mean + one(torch.tensor(EPS, dtype=torch.float64, device="cuda"))).sqrt()).reciprocal()
            rows.append(one(one(v * one(r)) * d["norm"].double()))
        X = torch.stack(rows)

    def quantized(v):
        s = one(v.abs().max() / 127)
        if float(s) == 0.0:
            return torch.zeros_like(v), s
        return torch.clip(torch.round(one(v / s)), -127, 127), s

    def product(codes, scale, w, s_w, b=None):
        y = one(s_w.double() * scale) * (w.double() @ codes)
        return y if b is None else y + b.double()

    if case["op"] == "linear":
        pairs = [quantized(v) for v in X]
        Q, S = torch.stack([p[0] for p in pairs]), torch.stack([p[1] for p in pairs])
        Y = one(S[:, None] * d["s_w"].double()[None, :]) * (Q @ d["w"].double().T)
        for part in ("bias", "residual"):
            if d[part] is not None:
                Y = Y + d[part].double()
        return Y
    chosen, weights, out = [], [], []
    for m, v in enumerate(X):
        logit = one((d["router"].double() * v).sum(1))
        if case["score"] == "softmax":
            p, key = torch.exp(logit - torch.logsumexp(logit, 0)), logit
        else:
            p = 1 / (1 + torch.exp(-logit))
            key = one(one(p) + d["select"].double())
        order = sorted(range(case["E"]), key=lambda e, k=key.tolist(): (-k[e], e))[: case["top_k"]]
        w = p[order]
        w = (w / w.sum() if case["renormalize"] else w) * d["scale"]
        chosen.append(order)
        weights.append(w)
        if case["op"] == "route":
            continue
        q, s = quantized(v)
        y = torch.zeros(case["H"], dtype=torch.float64, device="cuda")
        for e, we in zip(order + list(range(case["E"], case["E"] + case["shared"])), w.tolist() + [1.0] * case["shared"]):
            gu = one(product(q, s, d["gu"][e], d["s_gu"][e]))
            g, u = gu[: case["I"]], gu[case["I"]:]
            if case["act"] == "silu":
                a = g * torch.sigmoid(g)
            else:
                a = 0.5 * g * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)))
            y = y + we * product(*quantized(one(a * u)), d["dn"][e], d["s_dn"][e])
        out.append(y if d["residual"] is None else y + d["residual"][m].double())
    got = {"ids": torch.tensor(chosen, dtype=torch.int32), "weights": torch.stack(weights)}
    return got if case["op"] == "route" else {"y": torch.stack(out), **got}
