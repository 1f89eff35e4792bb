"""Attention over a paged cache for decode steps and drafted trees: the
load-time preparation and the per-step calls.

`KVCache` is one layer's cache, `KVBatch` says which rows of a step are whose,
`RopeTable` holds the rotations, and `CachedAttention` takes the rows of a
fused q/k/v projection through head norms, rotation and the cache to the
attention's output.  Buffers are torch tensors (device memory only); a caller
that runs a layer in every step makes them once with `buffers(T, batch)`.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import _lib


class KVCache:
    """k, v: fp16, bf16 or int8 [pages][heads][page_size][head_dim]; an int8 cache has a scale for each token and head,
    float32 [pages][heads][page_size]."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        self.desc = _lib.kv_cache(k, v, k_scale, v_scale)

    k, v, k_scale, v_scale = (property(lambda self, i=i: self.desc._tensors[i]) for i in range(4))

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, head_dim: int, dtype=torch.bfloat16, device="cuda") -> "KVCache":
        """A cache with memory of its own, all zeros."""
        shape = (pages, heads, page_size, head_dim)
        k, v = torch.zeros(shape, dtype=dtype, device=device), torch.zeros(shape, dtype=dtype, device=device)
        if dtype != torch.int8:
            return cls(k, v)
        return cls(k, v, torch.zeros(shape[:3], device=device), torch.zeros(shape[:3], device=device))

    def values(self, which: str, out=None, stream=None):
        """All cached keys ("k") or values ("v") as numbers: the 16-bit tensor itself, or an int8 cache's codes times scales
        in float32."""
        t = {"k": self.k, "v": self.v}[which]
        if t.dtype != torch.int8:
            return t
        if out is None:
            with _lib.allocating_on(stream):
                out = torch.empty(t.shape, dtype=torch.float32, device=t.device)
        _lib.w4_kv_values(self.desc, which, out, stream)
        return out


class KVBatch:
    """table int32 [B][max_pages], ctx int32 [B], q_start int32 [B + 1]: sequence b has rows q_start[b] .. q_start[b + 1] - 1
    behind ctx[b] cached tokens.  The tensors stay on the device and may be updated in place between calls.
    max_tokens: the most rows of a sequence.  It decides which kernel attends (up to 16 rows of max_tokens times query heads to a
    key head, or more) and the workspace's size, so a program that has steps of one token and of many drafts makes a batch
    object for each, on the same tensors."""

    def __init__(self, table, ctx, q_start, max_tokens: int):
        self.desc = _lib.kv_batch(table, ctx, q_start, max_tokens)


class RopeTable:
    """turns: float32 [positions][rot / 2][2], (cos, sin) of each position; layout "half" (pairs i, i + rot / 2) or
    "interleaved" (pairs 2 i, 2 i + 1)."""

    def __init__(self, turns, layout: str = "half"):
        self.desc = _lib.rope_desc(turns, layout)

    @property
    def turns(self):
        return self.desc._tensors[0]

    @staticmethod
    def frequencies(rot: int, base: float = 10000.0, scaling: dict = None):
        """Angles per position (float64 [rot / 2]) and the factor of the rotated values.  scaling, for contexts past the
        trained length: {"kind": "linear", "factor"} divides all angles; {"kind": "base", "factor"} raises the base so that
        the slowest pair is divided by it; {"kind": "by_parts", "factor", "trained", "slow": 1, "fast": 32} divides the pairs that turn
        less than `slow` times over the trained length, leaves those that turn more than `fast` times, goes linearly in the turns
        between them, and scales the rotated values by 0.1 ln(factor) + 1 (or "attention").  Programs that go linearly in the
        pair's number between two rounded borders get other angles in between: their tables go to RopeTable itself."""
        if rot < 0 or rot % 8:
            raise ValueError(f"rot {rot} is not a multiple of 8")
        s = dict(scaling or {"kind": "none"})
        kind, f = s.pop("kind", None), float(s.pop("factor", 1.0))
        if kind not in ("none", "linear", "base", "by_parts") or not f >= 1.0:
            raise ValueError(f"scaling {scaling!r}: kinds are linear, base and by_parts, factors at least 1")
        if kind == "base":
            base = base * f ** (rot / (rot - 2))
        inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
        scale = 1.0
        if kind == "linear":
            inv = inv / f
        elif kind == "by_parts":
            slow, fast = float(s.pop("slow", 1.0)), float(s.pop("fast", 32.0))
            if "trained" not in s or not float(s["trained"]) > 0.0 or not 0.0 <= slow < fast:
                raise ValueError(f"scaling {scaling!r}: by_parts takes a trained length and slow below fast")
            scale = float(s.pop("attention", 0.1 * math.log(f) + 1.0))
            turns = float(s.pop("trained")) * inv / (2 * math.pi)
            keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
            inv = inv * (keep + (1.0 - keep) / f)
        if s:
            raise ValueError(f"scaling {scaling!r}: {sorted(s)} are not part of {kind!r}")
        return inv, scale

    @classmethod
    def build(cls, positions: int, rot: int, base: float = 10000.0, layout: str = "half", scaling: dict = None,
              device="cuda") -> "RopeTable":
        inv, scale = cls.frequencies(rot, base, scaling)
        turns = torch.empty((positions, rot // 2, 2), dtype=torch.float32, device=device)
        with torch.cuda.device(turns.device):
            _lib.w4_rope_table(inv.to(turns.device), turns, scale=scale)
            return cls(turns, layout)


@dataclass
class AttentionBuffers:
    q: torch.Tensor          # [T][heads][head_dim], 16 bits
    y: torch.Tensor          # [T][heads][head_dim]
    workspace: torch.Tensor  # uint8


class CachedAttention:
    """heads: query heads (a multiple of the cache's); rope: RopeTable or None; q_norm, k_norm: RMSNorm weights float32
    [head_dim] of each head, or None; scale: of the scores, 1 / sqrt(head_dim) if None; q_dtype: of the rotated queries,
    the cache's own type, or bf16 (default) or fp16 with an int8 cache."""

    def __init__(self, cache: KVCache, heads: int, rope: RopeTable = None, q_norm=None, k_norm=None, eps: float = 1e-6,
                 scale: float = None, q_dtype=None):
        kind = cache.k.dtype
        self.cache, self.heads, self.rope, self.q_norm, self.k_norm, self.eps = cache, int(heads), rope, q_norm, k_norm, eps
        self.D = cache.desc.D
        if self.heads <= 0 or self.heads % cache.desc.Hkv:
            raise ValueError(f"{heads} query heads do not share {cache.desc.Hkv} key heads evenly")
        self.q_dtype = q_dtype or (torch.bfloat16 if kind == torch.int8 else kind)
        if self.q_dtype not in (torch.float16, torch.bfloat16) or (kind != torch.int8 and self.q_dtype != kind):
            raise ValueError(f"queries of {self.q_dtype} over a cache of {kind}")
        self.scale = self.D ** -0.5 if scale is None else float(scale)
        self._rope = None if rope is None else rope.desc

    def workspace(self, T: int, batch: KVBatch):
        """A workspace for the attention of T rows (W4Error for a batch that it refuses)."""
        n = _lib.w4_tree_attention_workspace_bytes(self.cache.desc, batch.desc, T, self.heads)
        if n == 0 and T != 0 and batch.desc.B != 0:
            raise _lib.W4Error("w4_tree_attention_workspace_bytes", _lib.W4_UNSUPPORTED_SHAPE)
        return torch.empty(n, dtype=torch.uint8, device=self.cache.k.device)

    def buffers(self, T: int, batch: KVBatch, dtype=torch.float32) -> AttentionBuffers:
        """What the calls on T rows write; y of `dtype`.  Calls that share buffers must not overlap on the GPU."""
        dev, shape = self.cache.k.device, (T, self.heads, self.D)
        return AttentionBuffers(torch.empty(shape, dtype=self.q_dtype, device=dev), torch.empty(shape, dtype=dtype, device=dev),
                                self.workspace(T, batch))

    def append(self, qkv, batch: KVBatch, positions=None, q=None, flags: int = 0, stream=None):
        """The rotated queries [T][heads][head_dim] of rows qkv [T][(heads + 2 key heads) head_dim]; their keys and values go
        to the cache.  positions: int32 [T], the rows' places if None."""
        if q is None:
            with _lib.allocating_on(stream):
                q = torch.empty((qkv.shape[0], self.heads, self.D), dtype=self.q_dtype, device=qkv.device)
        _lib.w4_kv_append(self.cache.desc, batch.desc, self._rope, qkv, q, positions, self.q_norm, self.k_norm, self.eps, flags,
                          stream)
        return q

    def attend(self, q, batch: KVBatch, mask=None, y=None, workspace=None, flags: int = 0, stream=None):
        """y [T][heads][head_dim] over the cache and the drafts of each row's mask (int64 [T], bit j: the sequence's row j;
        None: the rows up to itself).  Without y it has q's type.  Sequences of up to 64 rows."""
        if y is None or workspace is None:
            with _lib.allocating_on(stream):
                y = torch.empty_like(q) if y is None else y
                workspace = self.workspace(q.shape[0], batch) if workspace is None else workspace
        _lib.w4_tree_attention(self.cache.desc, batch.desc, q, y, workspace, mask, self.scale, flags, stream)
        return y

    def __call__(self, qkv, batch: KVBatch, positions=None, mask=None, buffers: AttentionBuffers = None, flags: int = 0,
                 stream=None):
        """append, then attend: three launches, the second a programmatic dependent of the first.  Without buffers y has
        qkv's type.  What either refuses is refused before the cache is written."""
        b = buffers
        if b is None:
            with _lib.allocating_on(stream):
                b = self.buffers(qkv.shape[0], batch, qkv.dtype)
        home = _lib.check_tree_attention(self.cache.desc, batch.desc, b.q, b.y, b.workspace, mask, self.scale)
        self.append(qkv, batch, positions, b.q, flags, stream)
        _lib.launch_tree_attention(home, self.cache.desc, batch.desc, b.q, b.y, b.workspace, mask, self.scale, _lib.W4_FLAG_PDL, stream)
        return b.y
