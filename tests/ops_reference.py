"""Plain 64-bit forms of the operators with integer weights: the codes (fp32 where the definition decides a code in
fp32), the linear, the router and the experts.  numpy on the host, no code of the package."""
import numpy as np

F32, F64 = np.float32, np.float64


def one(v):
    """Rounded once to fp32, kept in 64 bits."""
    return np.asarray(v, F64).astype(F32).astype(F64)


def rmsnorm(x, g, eps):
    x = np.asarray(x, F64)
    S = one(np.sum(x * x, axis=1, keepdims=True))
    r = one(1.0 / one(np.sqrt(one(one(S / x.shape[1]) + one(eps)))))
    return one(one(x * r) * np.asarray(g, F64))


def codes(x):
    """x [M][K] (values of fp32) -> integer codes and fp32 scales, in 64 bits."""
    x = np.asarray(x, F64)
    s = one(np.abs(x).max(axis=1, keepdims=True) / 127.0)
    q = np.clip(np.rint(one(x / np.where(s > 0, s, 1.0))), -127, 127)
    return np.where(s > 0, q, 0.0), s[:, 0]


def linear(q, s, w, s_w, b=None):
    """y [M][N] in 64 bits, fp32(s_w s_x) times the exact sum, plus b; and the fp32 value of the library's epilogue."""
    acc = np.asarray(q, F64) @ np.asarray(w, F64).T                 # exact: below 2^53
    sc = one(np.asarray(s, F64)[:, None] * np.asarray(s_w, F64)[None, :])
    bias = 0.0 if b is None else np.asarray(b, F64)[None, :]
    return sc * acc + bias, one(sc * one(acc) + bias)


EPS = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}   # half a step, relative
TINY = {"float32": 2.0 ** -149, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -133}


def logits(x, w):
    return one(np.asarray(x, F64) @ np.asarray(w, F64).T)


def route(l, top_k, score, bias, renorm, scale):
    """ids [M][top_k] and weights in 64 bits from the logits l [M][E]."""
    l = np.asarray(l, F64)
    if score == "softmax":
        e = np.exp(l - l.max(axis=1, keepdims=True))
        p, key = e / e.sum(axis=1, keepdims=True), l
    else:
        p = 1.0 / (1.0 + np.exp(-l))
        key = one(p) if bias is None else one(one(p) + np.asarray(bias, F64))
    ids = np.argsort(-key, axis=1, kind="stable")[:, :top_k]
    w = np.take_along_axis(p, ids, axis=1)
    if renorm:
        w = w / w.sum(axis=1, keepdims=True)
    return ids, w * scale


def act(kind, g, u):
    g, u = np.asarray(g, F64), np.asarray(u, F64)
    with np.errstate(over="ignore"):
        if kind == "silu":
            return one(g / (1.0 + np.exp(-g)) * u)
        return one(g / (1.0 + np.exp(-2.0 * np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3))) * u)


def experts(q, s, ids, weights, gu, s_gu, dn, s_dn, kind, n_shared=0, b_gu=None, b_dn=None):
    """y [M][H] in 64 bits and a bound of its fp32 roundings.  gu [n][2I][H], dn [n][H][I] integer codes."""
    M, H = q.shape
    n, I = len(gu), gu[0].shape[0] // 2
    E = n - n_shared
    y, room = np.zeros((M, H)), np.zeros((M, H))
    for m in range(M):
        slots = [(int(e), float(w)) for e, w in zip(ids[m], weights[m]) if 0 <= e < E] + [(E + j, 1.0) for j in range(n_shared)]
        for e, w in slots:
            _, v = linear(q[m:m + 1], s[m:m + 1], gu[e], s_gu[e], None if b_gu is None else b_gu[e])
            h = act(kind, v[0, :I], v[0, I:])
            qh, sh = codes(h[None])
            d, _ = linear(qh, sh, dn[e], s_dn[e], None if b_dn is None else b_dn[e])
            prod, _ = linear(qh, sh, dn[e], s_dn[e])
            y[m] += w * d[0]
            room[m] += abs(w) * (np.abs(prod[0]) + np.abs(d[0])) + (len(slots) + 1) * np.abs(w * d[0])
    return y, 2.0 ** -24 * room
