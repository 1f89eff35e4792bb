"""Plain 64-bit implementations (torch, host) of the cache append, attention over a paged cache and logit rules, with the
error bounds of their arithmetic.  Shares no code with the product."""
import random

import torch

F32 = torch.float32
F64 = torch.float64


def one(t):
    """Rounded once to 32 bits, held in 64."""
    return t.to(F32).to(F64)


def tree(rng, n, chain=False):
    """Masks (bit j: row j on the path, own bit set) and depths of a random tree of n rows."""
    masks, depth = [], []
    for i in range(n):
        p = i - 1 if chain else (rng.randint(max(-1, i - 3), i - 1) if i else -1)
        masks.append((masks[p] if p >= 0 else 0) | 1 << i)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return masks, depth


def as_int64(masks):
    masks = [m & (1 << 64) - 1 for m in masks]
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64)


class Paged:
    """A random paged layout: ns rows and ctxs cached places of each sequence."""

    def __init__(self, seed, ns, ctxs, page, spare=2, slack=0):
        g = random.Random(seed)
        self.ns, self.ctxs, self.page = ns, ctxs, page
        need = [(n + x + page - 1) // page for n, x in zip(ns, ctxs)]
        self.pages = sum(need) + spare
        free = list(range(self.pages))
        g.shuffle(free)
        width = max(need + [1]) + slack
        self.table = []
        for k in need:
            self.table.append(free[:k] + [-1] * (width - k))
            free = free[k:]
        self.q_start = [0]
        for n in ns:
            self.q_start.append(self.q_start[-1] + n)
        self.T = self.q_start[-1]

    def tensors(self):
        i32 = lambda v: torch.tensor(v, dtype=torch.int32)          # noqa: E731
        return i32(self.table), i32(self.ctxs), i32(self.q_start)

    def gather(self, t, b, count):
        """The first `count` places of sequence b of a cache tensor [pages][heads][page](..): [heads][count](..)."""
        p = torch.arange(count)
        pg = torch.tensor(self.table[b], dtype=torch.long)[p // self.page]
        return t[pg, :, p % self.page].transpose(0, 1)


def norm_heads(x, g, eps):
    """RMSNorm of each head in the steps of the definition, in fp32 roundings; x, g float64 holding fp32 numbers."""
    S = one((x * x).sum(-1, keepdim=True))
    r = one(1.0 / one(torch.sqrt(one(one(S / x.shape[-1]) + one(torch.tensor(eps, dtype=F64))))))
    return one(one(x * r) * g)


def rotate(x, turns, interleaved):
    """x [T][heads][D] by turns [T][rot / 2][2], in 64 bits."""
    h = turns.shape[1]
    c, s = turns[:, None, :, 0], turns[:, None, :, 1]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        y[..., :h], y[..., h:2 * h] = a * c - b * s, b * c + a * s
    return y


def codes(x):
    """INT8 codes and scale of each last axis of float64 values that are fp32 numbers."""
    s = one(x.abs().amax(-1, keepdim=True) / 127)
    q = torch.where(s > 0, torch.round(one(x / torch.where(s > 0, s, torch.ones_like(s)))).clamp(-127, 127), torch.zeros_like(x))
    return q.to(torch.int8), s[..., 0].to(F32)


def attend(lay, q, k, v, masks, scale, p_unit, y_unit, rounded_scales=False):
    """Outputs [T][Hq][D] in 64 bits and the bound of the kernel's error.  q float64 [T][Hq][D]; k, v float64
    [pages][Hkv][page][D] (the cache's numbers); masks: per row; p_unit: relative rounding of a probability, y_unit: of an
    output."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    y, bound = torch.zeros_like(q), torch.zeros_like(q)
    for b, (n, ctx) in enumerate(zip(lay.ns, lay.ctxs)):
        if n == 0:
            continue
        K, V = lay.gather(k, b, ctx + n), lay.gather(v, b, ctx + n)
        place = torch.arange(ctx + n)
        for i in range(n):
            t = lay.q_start[b] + i
            see = (place < ctx) | torch.tensor([p >= ctx and bool(masks[t] >> (p - ctx) & 1) for p in range(ctx + n)])
            if not bool(see.any()):
                continue
            qq = q[t].view(Hkv, G, D)
            Ks, Vs = K[:, see], V[:, see]
            s = scale * torch.einsum("hgd,hld->hgl", qq, Ks)
            p = torch.softmax(s, -1)
            y[t] = torch.einsum("hgl,hld->hgd", p, Vs).reshape(Hq, D)
            # A score: D products summed in fp32 (a step of the sum rounds or truncates), its factors, its difference to the
            # maximum; the exponential; sums of as many terms as are seen; both the numerator and the sum have the errors.
            mag = scale * torch.einsum("hgd,hld->hgl", qq.abs(), Ks.abs()).amax(-1, keepdim=True)
            ds = mag * (D + 16) * 2.0 ** -23 + (3 if rounded_scales else 1) * s.abs().amax(-1, keepdim=True) * 2.0 ** -22
            e = 2 * ds + 2.0 ** -20 + int(see.sum()) * 2.0 ** -22
            weight = torch.einsum("hgl,hld->hgd", p, Vs.abs())
            bound[t] = (weight * (e + p_unit)).reshape(Hq, D) + y[t].abs() * y_unit
    return y, bound


def logits(x, rules, rows, V, allowed=None):
    """Adjusted logits in 64 bits.  rules[s]: dict with prompt, made (lists), rep, freq, pres, bias (list of pairs); rows[r]:
    (s, path tokens) or None for a row that is left alone."""
    y = x.clone()
    for r, row in enumerate(rows):
        if row is None:
            continue
        s, path = row
        u = rules[s]
        made = torch.zeros(V, dtype=F64)
        for t in list(u["made"]) + list(path):
            if 0 <= t < V:
                made[t] += 1
        seen = made > 0
        for t in u["prompt"]:
            if 0 <= t < V:
                seen[t] = True
        v = x[r].clone()
        v = torch.where(seen, torch.where(v > 0, v / u["rep"], v * u["rep"]), v)
        v = torch.where(made > 0, v - u["freq"] * made - u["pres"], v)
        for t, add in u["bias"]:
            if 0 <= t < V:
                v[t] = v[t] + add
        if allowed is not None:
            v[~allowed[r]] = -float("inf")
        y[r] = v
    return y
