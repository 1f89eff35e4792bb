"""Mixture-of-experts layer for 1 to 16 tokens: load-time preparation and the
per-step call.

`MoeRouter` chooses the experts of a few tokens; `MoeLayer` holds the experts'
gated MLP on per-row INT4 or INT8 weights and runs router and experts in two
launches.  Buffers are torch tensors (device memory only); a caller that runs a
layer in every step makes them once with `buffers(M)`.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import _lib

ACTS = {"silu": _lib.W4_GLU_SILU, "gelu_tanh": _lib.W4_GLU_GELU_TANH}


@dataclass
class RouteBuffers:
    ids: torch.Tensor        # int32 [M][top_k]
    weights: torch.Tensor    # float32 [M][top_k]


@dataclass
class MoeBuffers:
    ids: torch.Tensor        # int32 [M][top_k]
    weights: torch.Tensor    # float32 [M][top_k]
    qx: torch.Tensor         # int8 [M][H]
    sx: torch.Tensor         # float32 [M]
    y: torch.Tensor          # [M][H]
    workspace: torch.Tensor  # uint8


class MoeRouter:
    """w: float32 [E][K]; select_bias: float32 [E], added to the sigmoid scores for the choice only; norm: RMSNorm
    weight float32 [K] applied to x first (with eps)."""

    def __init__(self, w, top_k: int, select_bias=None, score: str = "softmax", renormalize: bool = True,
                 scale: float = 1.0, norm=None, eps: float = 1e-6):
        self.E, self.K = w.shape
        self.top_k = int(top_k)
        self.desc = _lib.moe_router(w, top_k, select_bias, score, renormalize, scale, norm, eps)

    def buffers(self, M: int) -> RouteBuffers:
        dev = self.desc._tensors[0].device
        return RouteBuffers(torch.empty((M, self.top_k), dtype=torch.int32, device=dev),
                            torch.empty((M, self.top_k), dtype=torch.float32, device=dev))

    def __call__(self, x, buffers: RouteBuffers = None, qx=None, sx=None, flags: int = 0, stream=None):
        """ids and weights of x [M][K] (fp32, fp16 or bf16); qx, sx: receive the (normalized) tokens' codes."""
        b = buffers
        if b is None:
            with _lib.allocating_on(stream):
                b = self.buffers(x.shape[0])
        _lib.w4_moe_route(self.desc, x, b.ids, b.weights, qx, sx, flags, stream)
        return b.ids, b.weights


class MoeLayer:
    def __init__(self, fmt: str, router: MoeRouter, experts: _lib.Experts):
        self.fmt, self.router, self.desc = fmt, router, experts
        self.H, self.I, self.E, self.n_shared = experts.H, experts.I, experts.E, experts.n_shared

    # ------------------------------------------------------------- building
    @classmethod
    def from_float(cls, fmt: str, router: MoeRouter, gate_up, down, act: str = "silu", n_shared: int = 0, b_gu=None,
                   b_dn=None) -> "MoeLayer":
        """gate_up: float32 CUDA tensors [2 I][H] (gate rows first), down: [H][I], one per expert, the n_shared shared
        experts last (each is quantized as it is reached, so they may come from a generator); biases [experts][..]."""
        if fmt not in _lib.EXPERT_FORMATS:
            raise ValueError(f"experts are {sorted(_lib.EXPERT_FORMATS)}, not {fmt!r}")
        q = _lib.w4_quantize_rows if fmt == "w4" else _lib.w8_quantize_rows

        def quantized(W):
            W = W.contiguous()
            n, K = W.shape
            c = (torch.empty((n, K // 8), dtype=torch.int32, device=W.device) if fmt == "w4"
                 else torch.empty((n, K), dtype=torch.int8, device=W.device))
            s = torch.empty(n, dtype=torch.float32, device=W.device)
            q(W, c, s)
            return c, s

        gu, dn = [quantized(W) for W in gate_up], [quantized(W) for W in down]
        return cls.from_canonical(fmt, router, [c for c, _ in gu], torch.stack([s for _, s in gu]), [c for c, _ in dn],
                                  torch.stack([s for _, s in dn]), act, n_shared, b_gu, b_dn)

    @classmethod
    def from_canonical(cls, fmt: str, router: MoeRouter, gate_up, s_gu, down, s_dn, act: str = "silu", n_shared: int = 0,
                       b_gu=None, b_dn=None) -> "MoeLayer":
        """Repack quantized experts.  gate_up[e]: canonical rows [2 I] of H weights, gate rows first (int32 words
        [2 I][H / 8] for "w4", int8 codes [2 I][H] for "w8"); down[e]: [H] rows of I weights; s_gu [experts][2 I],
        s_dn [experts][H] and the optional biases b_gu, b_dn: float32."""
        if fmt not in _lib.EXPERT_FORMATS:
            raise ValueError(f"experts are {sorted(_lib.EXPERT_FORMATS)}, not {fmt!r}")
        if act not in ACTS:
            raise ValueError(f"act {act!r} is not one of {sorted(ACTS)}")
        n = len(gate_up)
        if n != router.E + n_shared or len(down) != n:
            raise ValueError(f"{n} gate/up and {len(down)} down matrices for {router.E} routed and {n_shared} shared experts")
        H, I = router.K, gate_up[0].shape[0] // 2
        if H % 32 or I % 32:
            raise ValueError("hidden and intermediate sizes are multiples of 32")
        rows = ((2 * I, H // 8), (H, I // 8)) if fmt == "w4" else ((2 * I, H), (H, I))
        glu_bytes = _lib.w4_glu_repacked_bytes(I, H) if fmt == "w4" else _lib.w8_glu_repacked_bytes(I, H)
        dn_bytes = _lib.w4_repacked_bytes(H, I) if fmt == "w4" else _lib.w8_repacked_bytes(H, I)
        dev = gate_up[0].device
        w_gu = torch.empty(n * glu_bytes, dtype=torch.uint8, device=dev)
        w_dn = torch.empty(n * dn_bytes, dtype=torch.uint8, device=dev)
        glu, plain = (_lib.w4_repack_glu, _lib.w4_repack) if fmt == "w4" else (_lib.w8_repack_glu, _lib.w8_repack)
        for e in range(n):
            if tuple(gate_up[e].shape) != rows[0] or tuple(down[e].shape) != rows[1]:
                raise ValueError(f"expert {e}: {tuple(gate_up[e].shape)} and {tuple(down[e].shape)}, not {rows}")
            glu(gate_up[e][:I], gate_up[e][I:], H, w_gu[e * glu_bytes:(e + 1) * glu_bytes])
            plain([down[e]], I, w_dn[e * dn_bytes:(e + 1) * dn_bytes])
        return cls(fmt, router, _lib.moe_experts(fmt, w_gu, s_gu.contiguous(), w_dn, s_dn.contiguous(), router.E, n_shared,
                                                 H, I, ACTS[act], b_gu, b_dn))

    # ------------------------------------------------------------- per step
    def buffers(self, M: int, dtype=torch.float32) -> MoeBuffers:
        """What M tokens' calls write; y of `dtype`.  Calls that share buffers must not overlap on the GPU."""
        dev = self.desc._tensors[0].device
        k = self.router.top_k
        return MoeBuffers(torch.empty((M, k), dtype=torch.int32, device=dev), torch.empty((M, k), device=dev),
                          torch.empty((M, self.H), dtype=torch.int8, device=dev), torch.empty(M, device=dev),
                          torch.empty((M, self.H), dtype=dtype, device=dev),
                          torch.empty(_lib.w4_moe_workspace_bytes(self.desc, M, k), dtype=torch.uint8, device=dev))

    def __call__(self, x, buffers: MoeBuffers = None, residual=None, flags: int = 0, stream=None):
        """y [M][H] for x [M][H] (fp32, fp16 or bf16): the router's norm, its choice, the experts, plus residual
        (float32 [M][H]).  Without buffers y has x's type, or float32 with a residual."""
        b = buffers
        if b is None:
            with _lib.allocating_on(stream):
                b = self.buffers(x.shape[0], x.dtype if residual is None else torch.float32)
        _lib.w4_moe_layer(self.router.desc, self.desc, x, b.ids, b.weights, b.qx, b.sx, b.y, b.workspace, residual, flags,
                          stream)
        return b.y

    def experts(self, qx, sx, ids, weights, y, workspace=None, residual=None, flags: int = 0, stream=None):
        """The experts alone on int8 codes and a choice made elsewhere (an id outside 0 .. E - 1 is an empty slot)."""
        if workspace is None:
            with _lib.allocating_on(stream):
                workspace = torch.empty(_lib.w4_moe_workspace_bytes(self.desc, ids.shape[0], ids.shape[1]),
                                        dtype=torch.uint8, device=y.device)
        _lib.w4_moe_experts(self.desc, qx, sx, ids, weights, y, workspace, residual, flags, stream)
        return y
