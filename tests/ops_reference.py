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
