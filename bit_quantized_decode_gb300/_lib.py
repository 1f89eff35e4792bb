"""ctypes binding of ``libw4a8.so`` (C ABI declared in include/w4a8.h).

Argument marshalling only: every function takes torch tensors that already
live on the current CUDA device, checks dtypes and shapes, and passes raw
pointers and the current stream to the C entry point of the same name.  All
arithmetic runs in the library's CUDA kernels; there is no CPU path.  If the
library has not been built, loading fails with an error saying how to build
it.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4a8.so")

W4_OK, W4_INVALID_ARG, W4_UNSUPPORTED_SHAPE, W4_MISALIGNED = range(4)
STATUS = {
    0: "W4_OK",
    1: "W4_ERR_INVALID_ARG",
    2: "W4_ERR_UNSUPPORTED_SHAPE",
    3: "W4_ERR_MISALIGNED",
    4: "W4_ERR_CUDA",
    5: "W4_ERR_DEVICE_TIMEOUT",
}
W4_FLAG_PDL = 1
TUNE_KEYS = {"blocks_per_sm": 0, "max_stages": 1, "grid_blocks": 2, "tc_min_m": 3, "chain_prefetch_kb": 4, "k_splits": 5,
             "group_launch_tokens": 6}
W4_MAX_M = 16
W4_MAX_K = 131072
W4_MAX_SHARDS = 8

# exported symbol -> (argtypes, restype)
_P = ctypes.c_void_p
_I = ctypes.c_int
_U = ctypes.c_uint
_SZ = ctypes.c_size_t
_PP = ctypes.POINTER(ctypes.c_void_p)
_PI = ctypes.POINTER(ctypes.c_int)
SIGNATURES = {
    "w4_status_str": ([_I], ctypes.c_char_p),
    "w4_version": ([], _I),
    "w4_set_tuning": ([_I, _I], _I),
    "w4_get_tuning": ([_I], _I),
    "w4_quantize_rows": ([_P, _I, _I, _P, _P, _P], _I),
    "q4_0_quantize": ([_P, _I, _I, _P, _P], _I),
    "i8g32_quantize": ([_P, _I, _I, _P, _P, _P], _I),
    "w4_repacked_bytes": ([_I, _I], _SZ),
    "q4_0_repacked_bytes": ([_I, _I], _SZ),
    "i8g32_repacked_bytes": ([_I, _I], _SZ),
    "q6g32_repacked_bytes": ([_I, _I], _SZ),
    "w4_repack": ([_PP, _PI, _I, _I, _P, _SZ, _P], _I),
    "q4_0_repack": ([_PP, _PI, _I, _I, _P, _SZ, _P], _I),
    "i8g32_repack": ([_PP, _PP, _PI, _I, _I, _P, _SZ, _P], _I),
    "q6g32_repack": ([_PP, _PP, _PI, _I, _I, _P, _SZ, _P], _I),
    "w4_concat_f32": ([_PP, _PI, _I, _P, _P], _I),
    "a8_quantize": ([_P, _I, _I, _P, _P, _P], _I),
    "w4a8_gemv": ([_P, _P, _P, _P, _P, _I, _I, _I, _P, _P], _I),
    "q4_0_gemv": ([_P, _P, _P, _P, _I, _I, _I, _P, _P], _I),
    "i8g32_gemv": ([_P, _P, _P, _P, _I, _I, _I, _P, _P], _I),
    "q6g32_gemv": ([_P, _P, _P, _P, _I, _I, _I, _P, _P], _I),
    "w4a8_linear": ([_P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _U, _P], _I),
    "q4_0_linear": ([_P, _P, _P, _I, _I, _I, _P, _P, _P, _U, _P], _I),
    "i8g32_linear": ([_P, _P, _P, _I, _I, _I, _P, _P, _P, _U, _P], _I),
    "q6g32_linear": ([_P, _P, _P, _I, _I, _I, _P, _P, _P, _U, _P], _I),
    "w4_device_error": ([ctypes.POINTER(ctypes.c_uint)], _I),
    "w4_clear_device_error": ([], _I),
}


class Fusion(ctypes.Structure):
    """w4_fusion of include/w4a8.h."""
    _fields_ = [("norm_weight", _P), ("norm_eps", ctypes.c_float), ("glu", _I), ("residual", _P)]


W4_GLU_NONE = 0
W4_GLU_SILU = 1
W4_GLU_GELU_TANH = 2
_F = ctypes.c_float
_LL = ctypes.c_longlong
_PF = ctypes.POINTER(Fusion)
SIGNATURES.update({
    "w4_glu_repacked_bytes": ([_I, _I], _SZ),
    "q4_0_glu_repacked_bytes": ([_I, _I], _SZ),
    "w4_repack_glu": ([_P, _P, _I, _I, _P, _SZ, _P], _I),
    "q4_0_repack_glu": ([_P, _P, _I, _I, _P, _SZ, _P], _I),
    "w4a8_linear_fused": ([_P, _P, _P, _P, _I, _I, _I, _P, _P, _P, _PF, _U, _P], _I),
    "q4_0_linear_fused": ([_P, _P, _P, _I, _I, _I, _P, _P, _P, _PF, _U, _P], _I),
    "i8g32_linear_fused": ([_P, _P, _P, _I, _I, _I, _P, _P, _P, _PF, _U, _P], _I),
    "q6g32_linear_fused": ([_P, _P, _P, _I, _I, _I, _P, _P, _P, _PF, _U, _P], _I),
    "rms_a8_quantize": ([_P, _P, _F, _I, _I, _P, _P, _U, _P], _I),
    "w4_rmsnorm": ([_P, _P, _F, _I, _I, _P, _U, _P], _I),
    "w4_glu": ([_P, _I, _I, _I, _P, _U, _P], _I),
    "w4_add": ([_P, _P, _LL, _P, _U, _P], _I),
    "w8_quantize_rows": ([_P, _I, _I, _P, _P, _P], _I),
    "w8_repacked_bytes": ([_I, _I], _SZ),
    "w8_repack": ([_PP, _PI, _I, _I, _P, _SZ, _P], _I),
    "w4a32_gemv": ([_P, _P, _P, _P, _I, _I, _I, _P, _U, _P], _I),
    "w8a32_gemv": ([_P, _P, _P, _P, _I, _I, _I, _P, _U, _P], _I),
})


class LinearDesc(ctypes.Structure):
    """w4_linear_desc of include/w4a8.h."""
    _fields_ = [("w", _P), ("s_w", _P), ("bias", _P), ("x", _P), ("y", _P), ("qx", _P), ("sx", _P),
                ("N", _I), ("K", _I)]


class DeviceDesc(ctypes.Structure):
    """w4_device_desc of include/w4a8.h."""
    _fields_ = [("sms", _I), ("smem_per_sm", _I), ("smem_reserved", _I), ("smem_optin", _I)]


class LaunchPlan(ctypes.Structure):
    """w4_launch_plan of include/w4a8.h."""
    _fields_ = [("path", _I), ("quantize_launches", _I), ("grid", _I), ("threads", _I), ("smem_bytes", _I),
                ("stages", _I), ("k_splits", _I), ("gemv_launches", _I)]


FORMATS = {"w4": 0, "q4_0": 1, "i8g32": 2, "q6g32": 3}
W4_PLAN_LINEAR = 1
W4_PLAN_NORM = 2
W4_PLAN_GLU = 4
PATHS = {0: "none", 1: "fused", 2: "codes_smem", 3: "codes_global", 4: "tensor_cores"}
SIGNATURES["w4_plan"] = ([_I, _I, _I, _I, _U, ctypes.POINTER(DeviceDesc), ctypes.POINTER(LaunchPlan)], _I)
SIGNATURES["w4_describe_device"] = ([ctypes.POINTER(DeviceDesc)], _I)
SIGNATURES["w4_chain_workspace_bytes"] = ([], _SZ)
SIGNATURES["w4_chain_noalloc_scratch_bytes"] = ([], _SZ)
SIGNATURES["w4a8_linear_chain_noalloc"] = ([ctypes.POINTER(LinearDesc), _I, _I, _P], _I)
SIGNATURES["w4a8_linear_chain"] = ([ctypes.POINTER(LinearDesc), _I, _I, _P, _SZ, _P], _I)
SIGNATURES["w4_workspace_bytes"] = ([_I, _I, _I], _SZ)
SIGNATURES["w4_quantize_rows_host"] = ([_P, _I, _I, _P, _P], _I)
SIGNATURES["q4_0_quantize_host"] = ([_P, _I, _I, _P], _I)
SIGNATURES["i8g32_quantize_host"] = ([_P, _I, _I, _P, _P], _I)
SIGNATURES["w4_last_device_error"] = ([ctypes.POINTER(ctypes.c_uint)], _I)
SIGNATURES["w4_hbm_read"] = ([_P, _SZ, _P, _P], _I)
SIGNATURES["w4_selftest_wait_timeout"] = ([_I, ctypes.c_uint, _P], _I)
SIGNATURES["w8a8_workspace_bytes"] = ([_I, _I, _I], _SZ)
SIGNATURES["w8a8_matmul"] = ([_P, _P, _P, _P, _P, _I, _I, _I, _P, _I, _P, _SZ, _P], _I)
SIGNATURES["w8a8_linear"] = ([_P, _P, _P, _P, _I, _I, _I, _I, _P, _I, _P, _P, _PF, _U, _P, _SZ, _P], _I)
class Router(ctypes.Structure):
    """w4_router of include/w4a8.h."""
    _fields_ = [("norm_weight", _P), ("norm_eps", _F), ("w", _P), ("select_bias", _P), ("E", _I), ("top_k", _I),
                ("score", _I), ("renormalize", _I), ("scale", _F)]


class Experts(ctypes.Structure):
    """w4_experts of include/w4a8.h."""
    _fields_ = [("fmt", _I), ("E", _I), ("n_shared", _I), ("H", _I), ("I", _I), ("glu", _I), ("w_gu", _P),
                ("s_gu", _P), ("b_gu", _P), ("w_dn", _P), ("s_dn", _P), ("b_dn", _P)]


_PR = ctypes.POINTER(Router)
_PE = ctypes.POINTER(Experts)
SIGNATURES["w8_glu_repacked_bytes"] = ([_I, _I], _SZ)
SIGNATURES["w8_repack_glu"] = ([_P, _P, _I, _I, _P, _SZ, _P], _I)
SIGNATURES["w4_moe_route"] = ([_PR, _P, _I, _I, _I, _P, _P, _P, _P, _U, _P], _I)
SIGNATURES["w4_moe_workspace_bytes"] = ([_PE, _I, _I], _SZ)
SIGNATURES["w4_moe_experts"] = ([_PE, _P, _P, _P, _P, _I, _I, _P, _P, _I, _P, _SZ, _U, _P], _I)
SIGNATURES["w4_moe_layer"] = ([_PR, _PE, _P, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P, _SZ, _U, _P], _I)
EXPERT_FORMATS = {"w4": 0, "w8": 5}                    # W4_FMT_W4, W4_FMT_W8
ROUTE_SCORES = {"softmax": 0, "sigmoid": 1}
W4_MAX_TOP_K = 16
W4_MAX_EXPERTS = 1024
W4_MAX_SHARED = 4
ELEM_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}   # W4_F32, W4_F16, W4_BF16
W4_MAX_TOKENS = 1 << 20
W4_MAX_CHAIN = 128


class KVCacheDesc(ctypes.Structure):
    """w4_kv_cache of include/w4a8.h."""
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("type", _I), ("pages", _I), ("page_size", _I),
                ("Hkv", _I), ("D", _I)]


class KVBatchDesc(ctypes.Structure):
    """w4_kv_batch of include/w4a8.h."""
    _fields_ = [("table", _P), ("ctx", _P), ("q_start", _P), ("B", _I), ("max_pages", _I), ("max_tokens", _I)]


class RopeDesc(ctypes.Structure):
    """w4_rope of include/w4a8.h."""
    _fields_ = [("turns", _P), ("positions", _I), ("rot", _I), ("layout", _I)]


class LogitRulesDesc(ctypes.Structure):
    """w4_logit_rules of include/w4a8.h."""
    _fields_ = [("V", _I), ("S", _I), ("ids", _P), ("cap", _I), ("length", _P), ("prompt", _P), ("repetition", _P),
                ("frequency", _P), ("presence", _P), ("bias_ids", _P), ("bias", _P), ("n_bias", _I)]


_PC = ctypes.POINTER(KVCacheDesc)
_PB = ctypes.POINTER(KVBatchDesc)
SIGNATURES["w4_rope_table"] = ([_P, ctypes.c_double, ctypes.c_double, _I, _I, _P, _P], _I)
SIGNATURES["w4_kv_values"] = ([_PC, _I, _P, _P], _I)
SIGNATURES["w4_kv_append"] = ([_PC, _PB, ctypes.POINTER(RopeDesc), _P, _I, _LL, _I, _I, _P, _P, _P, _F, _P, _I, _U, _P], _I)
SIGNATURES["w4_tree_attention_workspace_bytes"] = ([_PC, _PB, _I, _I], _SZ)
SIGNATURES["w4_tree_attention"] = ([_PC, _PB, _P, _I, _I, _I, _P, _F, _P, _I, _P, _SZ, _U, _P], _I)
SIGNATURES["w4_logits_adjust"] = ([ctypes.POINTER(LogitRulesDesc), _P, _I, _LL, _I, _P, _P, _P, _P, _P, _LL, _U, _P], _I)
CACHE_TYPES = {torch.float16: 1, torch.bfloat16: 2, torch.int8: 3}     # W4_F16, W4_BF16, W4_I8
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
W4_MAX_SEQUENCES = 1024
W4_MAX_DRAFTS = 64
W4_MAX_BIASES = 1024

_lib = None


class W4Error(RuntimeError):
    def __init__(self, name: str, status: int):
        super().__init__(f"{name}: {STATUS.get(status, status)}")
        self.status = status


def load(path: str = LIB_PATH):
    """Load the library (once).  Raises if it is missing: there is no fallback."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m bit_quantized_decode_gb300.build` "
                "(needs nvcc); the decode GEMV has no CPU implementation")
        lib = ctypes.CDLL(path)
        for name, (args, res) in SIGNATURES.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = res
        _lib = lib
    return _lib


def _check(name: str, st: int):
    if st != W4_OK:
        raise W4Error(name, st)


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev(*ts):
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("tensor must live on a CUDA device")
            if not t.is_contiguous():
                raise ValueError("tensor must be contiguous")


def _ptr_array(ts):
    arr = (ctypes.c_void_p * len(ts))(*[t.data_ptr() if t is not None else None for t in ts])
    return ctypes.cast(arr, _PP), arr


def _int_array(vals):
    arr = (ctypes.c_int * len(vals))(*vals)
    return ctypes.cast(arr, _PI), arr


# ---------------------------------------------------------------- queries
def status_str(st: int) -> str:
    return load().w4_status_str(st).decode()


def version() -> int:
    return load().w4_version()


def w4_describe_device() -> dict:
    """The current device's description (w4_device_desc) as a dict."""
    d = DeviceDesc()
    _check("w4_describe_device", load().w4_describe_device(ctypes.byref(d)))
    return {f: getattr(d, f) for f, _ in DeviceDesc._fields_}


def w4_plan(fmt: str, M: int, N: int, K: int, device: dict, linear: bool = True, norm: bool = False,
            glu: bool = False) -> dict:
    """The launch plan of a call (w4_plan): host computation only, no GPU
    needed.  device: a dict with the w4_device_desc fields."""
    d = DeviceDesc(**{f: int(device[f]) for f, _ in DeviceDesc._fields_})
    what = (W4_PLAN_LINEAR if linear else 0) | (W4_PLAN_NORM if norm else 0) | (W4_PLAN_GLU if glu else 0)
    p = LaunchPlan()
    _check("w4_plan", load().w4_plan(FORMATS[fmt], M, N, K, what, ctypes.byref(d), ctypes.byref(p)))
    out = {f: getattr(p, f) for f, _ in LaunchPlan._fields_}
    out["path"] = PATHS[out["path"]]
    return out


def set_tuning(key: str, value: int):
    """Launch tuning (see include/w4a8.h): blocks_per_sm, max_stages, grid_blocks; 0 = automatic."""
    _check("w4_set_tuning", load().w4_set_tuning(TUNE_KEYS[key], int(value)))


def get_tuning(key: str) -> int:
    return int(load().w4_get_tuning(TUNE_KEYS[key]))


def w4_repacked_bytes(N: int, K: int) -> int:
    return int(load().w4_repacked_bytes(N, K))


def q4_0_repacked_bytes(N: int, K: int) -> int:
    return int(load().q4_0_repacked_bytes(N, K))


def q6g32_repacked_bytes(N: int, K: int) -> int:
    return int(load().q6g32_repacked_bytes(N, K))


def i8g32_repacked_bytes(N: int, K: int) -> int:
    return int(load().i8g32_repacked_bytes(N, K))


# ------------------------------------------------------------- quantizers
def w4_quantize_rows(W, packed, s_w, stream=None):
    """W float32 [N][K] -> packed int32 [N][K/8] (canonical words), s_w float32 [N]."""
    _dev(W, packed, s_w)
    N, K = W.shape
    _check("w4_quantize_rows", load().w4_quantize_rows(_ptr(W), N, K, _ptr(packed), _ptr(s_w), _stream(stream)))


def q4_0_quantize(W, blocks, stream=None):
    """W float32 [N][K] -> blocks uint8 [N][K/32][18]."""
    _dev(W, blocks)
    N, K = W.shape
    _check("q4_0_quantize", load().q4_0_quantize(_ptr(W), N, K, _ptr(blocks), _stream(stream)))


def i8g32_quantize(W, q, d, stream=None):
    """W float32 [N][K] -> q int8 [N][K], d fp16 bits int16 [N][K/32]."""
    _dev(W, q, d)
    N, K = W.shape
    _check("i8g32_quantize", load().i8g32_quantize(_ptr(W), N, K, _ptr(q), _ptr(d), _stream(stream)))


# ------------------------------------------------- quantizers on the host
def _host_arr(a, dtype):
    """A C-contiguous numpy array of `dtype` (the host entry points take host memory)."""
    import numpy as np
    if not isinstance(a, np.ndarray) or a.dtype != dtype or not a.flags.c_contiguous:
        raise ValueError(f"expected a C-contiguous numpy array of {np.dtype(dtype)}")
    return ctypes.c_void_p(a.ctypes.data)


def w4_quantize_rows_host(W):
    """Host numpy float32 [N][K] -> (packed uint32 [N][K/8], s_w float32 [N]), by the library's host code."""
    import numpy as np
    N, K = W.shape
    packed = np.zeros((N, K // 8), np.uint32)
    sw = np.zeros(N, np.float32)
    _check("w4_quantize_rows_host", load().w4_quantize_rows_host(_host_arr(W, np.float32), N, K,
                                                                 _host_arr(packed, np.uint32), _host_arr(sw, np.float32)))
    return packed, sw


def q4_0_quantize_host(W):
    """Host numpy float32 [N][K] -> Q4_0 blocks uint8 [N][K/32][18], by the library's host code."""
    import numpy as np
    N, K = W.shape
    blocks = np.zeros((N, K // 32, 18), np.uint8)
    _check("q4_0_quantize_host", load().q4_0_quantize_host(_host_arr(W, np.float32), N, K,
                                                           _host_arr(blocks, np.uint8)))
    return blocks


def i8g32_quantize_host(W):
    """Host numpy float32 [N][K] -> (q int8 [N][K], d fp16 bits uint16 [N][K/32]), by the library's host code."""
    import numpy as np
    N, K = W.shape
    q = np.zeros((N, K), np.int8)
    d = np.zeros((N, K // 32), np.uint16)
    _check("i8g32_quantize_host", load().i8g32_quantize_host(_host_arr(W, np.float32), N, K, _host_arr(q, np.int8),
                                                             _host_arr(d, np.uint16)))
    return q, d


def workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load().w4_workspace_bytes(M, N, K))


# ---------------------------------------------------------------- repack
def w4_repack(shards, K, out, stream=None):
    """shards: list of canonical packed tensors [rows_s][K/8]; out: uint8 buffer."""
    _dev(out, *shards)
    pp, keep = _ptr_array(shards)
    rows, keep2 = _int_array([s.shape[0] for s in shards])
    _check("w4_repack", load().w4_repack(pp, rows, len(shards), K, _ptr(out), out.numel() * out.element_size(),
                                         _stream(stream)))


def q4_0_repack(shards, K, out, stream=None):
    _dev(out, *shards)
    pp, keep = _ptr_array(shards)
    rows, keep2 = _int_array([s.shape[0] for s in shards])
    _check("q4_0_repack", load().q4_0_repack(pp, rows, len(shards), K, _ptr(out), out.numel() * out.element_size(),
                                             _stream(stream)))


def i8g32_repack(q_shards, d_shards, K, out, stream=None):
    _dev(out, *q_shards, *d_shards)
    qp, keep = _ptr_array(q_shards)
    dp, keep2 = _ptr_array(d_shards)
    rows, keep3 = _int_array([s.shape[0] for s in q_shards])
    _check("i8g32_repack", load().i8g32_repack(qp, dp, rows, len(q_shards), K, _ptr(out),
                                               out.numel() * out.element_size(), _stream(stream)))


def q6g32_repack(q_shards, d_shards, K, out, stream=None):
    """Pack I8G32 canonical shards (codes in [-32, 31]) into the 6-bit device layout."""
    _dev(out, *q_shards, *d_shards)
    qp, keep = _ptr_array(q_shards)
    dp, keep2 = _ptr_array(d_shards)
    rows, keep3 = _int_array([s.shape[0] for s in q_shards])
    _check("q6g32_repack", load().q6g32_repack(qp, dp, rows, len(q_shards), K, _ptr(out),
                                               out.numel() * out.element_size(), _stream(stream)))


def w4_concat_f32(parts, out, stream=None):
    _dev(out, *parts)
    pp, keep = _ptr_array(parts)
    lens, keep2 = _int_array([p.numel() for p in parts])
    _check("w4_concat_f32", load().w4_concat_f32(pp, lens, len(parts), _ptr(out), _stream(stream)))


# ------------------------------------------------------------- per token
def a8_quantize(x, qx, sx, stream=None):
    """x float32 [M][K] -> qx int8 [M][K], sx float32 [M]."""
    _dev(x, qx, sx)
    M, K = x.shape
    _check("a8_quantize", load().a8_quantize(_ptr(x), M, K, _ptr(qx), _ptr(sx), _stream(stream)))


def w4a8_gemv(w, s_w, bias, qx, sx, y, stream=None):
    """y[M][N] from repacked per-row INT4 weights and int8 activations."""
    _dev(w, s_w, bias, qx, sx, y)
    M, K = qx.shape
    N = y.shape[1]
    _check("w4a8_gemv", load().w4a8_gemv(_ptr(w), _ptr(s_w), _ptr(bias), _ptr(qx), _ptr(sx), M, N, K, _ptr(y),
                                         _stream(stream)))


def q4_0_gemv(w, bias, qx, sx, y, stream=None):
    _dev(w, bias, qx, sx, y)
    M, K = qx.shape
    N = y.shape[1]
    _check("q4_0_gemv", load().q4_0_gemv(_ptr(w), _ptr(bias), _ptr(qx), _ptr(sx), M, N, K, _ptr(y),
                                         _stream(stream)))


def i8g32_gemv(w, bias, qx, sx, y, stream=None):
    _dev(w, bias, qx, sx, y)
    M, K = qx.shape
    N = y.shape[1]
    _check("i8g32_gemv", load().i8g32_gemv(_ptr(w), _ptr(bias), _ptr(qx), _ptr(sx), M, N, K, _ptr(y),
                                           _stream(stream)))


def q6g32_gemv(w, bias, qx, sx, y, stream=None):
    _dev(w, bias, qx, sx, y)
    M, K = qx.shape
    N = y.shape[1]
    _check("q6g32_gemv", load().q6g32_gemv(_ptr(w), _ptr(bias), _ptr(qx), _ptr(sx), M, N, K, _ptr(y),
                                           _stream(stream)))


def w4a8_linear(w, s_w, bias, x, y, qx, sx, flags: int = 0, stream=None):
    """Quantize x and run the per-row INT4 GEMV in one launch; y[M][N]."""
    _dev(w, s_w, bias, x, y, qx, sx)
    M, K = x.shape
    N = y.shape[1]
    _check("w4a8_linear", load().w4a8_linear(_ptr(w), _ptr(s_w), _ptr(bias), _ptr(x), M, N, K, _ptr(y), _ptr(qx),
                                             _ptr(sx), flags, _stream(stream)))


def q4_0_linear(w, bias, x, y, qx, sx, flags: int = 0, stream=None):
    _dev(w, bias, x, y, qx, sx)
    M, K = x.shape
    N = y.shape[1]
    _check("q4_0_linear", load().q4_0_linear(_ptr(w), _ptr(bias), _ptr(x), M, N, K, _ptr(y), _ptr(qx), _ptr(sx),
                                             flags, _stream(stream)))


def i8g32_linear(w, bias, x, y, qx, sx, flags: int = 0, stream=None):
    _dev(w, bias, x, y, qx, sx)
    M, K = x.shape
    N = y.shape[1]
    _check("i8g32_linear", load().i8g32_linear(_ptr(w), _ptr(bias), _ptr(x), M, N, K, _ptr(y), _ptr(qx), _ptr(sx),
                                               flags, _stream(stream)))


def q6g32_linear(w, bias, x, y, qx, sx, flags: int = 0, stream=None):
    _dev(w, bias, x, y, qx, sx)
    M, K = x.shape
    N = y.shape[1]
    _check("q6g32_linear", load().q6g32_linear(_ptr(w), _ptr(bias), _ptr(x), M, N, K, _ptr(y), _ptr(qx), _ptr(sx),
                                               flags, _stream(stream)))


# ------------------------------------------------ fusions around the linear
def w4_glu_repacked_bytes(I: int, K: int) -> int:
    return int(load().w4_glu_repacked_bytes(I, K))


def q4_0_glu_repacked_bytes(I: int, K: int) -> int:
    return int(load().q4_0_glu_repacked_bytes(I, K))


def w4_repack_glu(gate, up, K, out, stream=None):
    """Canonical packed gate and up [I][K/8] -> the paired device layout."""
    _dev(gate, up, out)
    assert gate.shape == up.shape
    _check("w4_repack_glu", load().w4_repack_glu(_ptr(gate), _ptr(up), gate.shape[0], K, _ptr(out),
                                                 out.numel() * out.element_size(), _stream(stream)))


def q4_0_repack_glu(gate, up, K, out, stream=None):
    """Q4_0 blocks of gate and up [I][K/32][18] -> the paired device layout."""
    _dev(gate, up, out)
    assert gate.shape == up.shape
    _check("q4_0_repack_glu", load().q4_0_repack_glu(_ptr(gate), _ptr(up), gate.shape[0], K, _ptr(out),
                                                     out.numel() * out.element_size(), _stream(stream)))


def fusion(norm_weight=None, eps: float = 0.0, glu: int = W4_GLU_NONE, residual=None):
    """A w4_fusion descriptor.  It holds references to its tensors, so their
    memory stays allocated while the descriptor is alive."""
    _dev(norm_weight, residual)
    fz = Fusion(None if norm_weight is None else norm_weight.data_ptr(), float(eps), int(glu),
                None if residual is None else residual.data_ptr())
    fz._tensors = (norm_weight, residual)
    return fz


def _fused_args(fz):
    return None if fz is None else ctypes.byref(fz)


def w4a8_linear_fused(w, s_w, bias, x, y, qx, sx, fz=None, flags: int = 0, stream=None):
    """w4a8_linear with RMSNorm / GLU / residual fused (fz from fusion()); y[M][N]."""
    _dev(w, s_w, bias, x, y, qx, sx)
    M, K = x.shape
    N = y.shape[1]
    _check("w4a8_linear_fused", load().w4a8_linear_fused(_ptr(w), _ptr(s_w), _ptr(bias), _ptr(x), M, N, K, _ptr(y),
                                                         _ptr(qx), _ptr(sx), _fused_args(fz), flags,
                                                         _stream(stream)))


def _grouped_fused(name, w, bias, x, y, qx, sx, fz, flags, stream):
    _dev(w, bias, x, y, qx, sx)
    M, K = x.shape
    N = y.shape[1]
    _check(name, getattr(load(), name)(_ptr(w), _ptr(bias), _ptr(x), M, N, K, _ptr(y), _ptr(qx), _ptr(sx),
                                       _fused_args(fz), flags, _stream(stream)))


def q4_0_linear_fused(w, bias, x, y, qx, sx, fz=None, flags: int = 0, stream=None):
    _grouped_fused("q4_0_linear_fused", w, bias, x, y, qx, sx, fz, flags, stream)


def i8g32_linear_fused(w, bias, x, y, qx, sx, fz=None, flags: int = 0, stream=None):
    _grouped_fused("i8g32_linear_fused", w, bias, x, y, qx, sx, fz, flags, stream)


def q6g32_linear_fused(w, bias, x, y, qx, sx, fz=None, flags: int = 0, stream=None):
    _grouped_fused("q6g32_linear_fused", w, bias, x, y, qx, sx, fz, flags, stream)


def rms_a8_quantize(x, norm_weight, eps, qx, sx, flags: int = 0, stream=None):
    """RMSNorm(x) then the activation quantizer: qx int8 [M][K], sx float32 [M]."""
    _dev(x, norm_weight, qx, sx)
    M, K = x.shape
    _check("rms_a8_quantize", load().rms_a8_quantize(_ptr(x), _ptr(norm_weight), float(eps), M, K, _ptr(qx),
                                                     _ptr(sx), flags, _stream(stream)))


def w4_rmsnorm(x, norm_weight, eps, out, flags: int = 0, stream=None):
    _dev(x, norm_weight, out)
    M, K = x.shape
    _check("w4_rmsnorm", load().w4_rmsnorm(_ptr(x), _ptr(norm_weight), float(eps), M, K, _ptr(out), flags,
                                           _stream(stream)))


def w4_glu(gu, kind, out, flags: int = 0, stream=None):
    """out[M][I] = act(gu[:, :I]) * gu[:, I:] for a gate|up output gu [M][2I]."""
    _dev(gu, out)
    M, I = out.shape
    assert gu.shape == (M, 2 * I)
    _check("w4_glu", load().w4_glu(_ptr(gu), int(kind), M, I, _ptr(out), flags, _stream(stream)))


def w4_add(a, b, out, flags: int = 0, stream=None):
    _dev(a, b, out)
    assert a.numel() == b.numel() == out.numel()
    _check("w4_add", load().w4_add(_ptr(a), _ptr(b), a.numel(), _ptr(out), flags, _stream(stream)))


# ------------------------------------- weight-only paths on float activations
def w8_quantize_rows(W, q, s_w, stream=None):
    """W float32 [N][K] -> q int8 [N][K] (per-row INT8), s_w float32 [N]."""
    _dev(W, q, s_w)
    N, K = W.shape
    _check("w8_quantize_rows", load().w8_quantize_rows(_ptr(W), N, K, _ptr(q), _ptr(s_w), _stream(stream)))


def w8_repacked_bytes(N: int, K: int) -> int:
    return int(load().w8_repacked_bytes(N, K))


def w8_repack(shards, K, out, stream=None):
    """shards: int8 [rows_s][K] per-row INT8 codes; out: uint8 buffer of w8_repacked_bytes."""
    _dev(out, *shards)
    pp, keep = _ptr_array(shards)
    rows, keep2 = _int_array([s.shape[0] for s in shards])
    _check("w8_repack", load().w8_repack(pp, rows, len(shards), K, _ptr(out), out.numel() * out.element_size(),
                                         _stream(stream)))


def w4a32_gemv(w, s_w, bias, x, y, flags: int = 0, stream=None):
    """Weight-only per-row INT4 (w4_repack layout) on float x [M][K], M <= 4; y[M][N]."""
    _dev(w, s_w, bias, x, y)
    M, K = x.shape
    N = y.shape[1]
    _check("w4a32_gemv", load().w4a32_gemv(_ptr(w), _ptr(s_w), _ptr(bias), _ptr(x), M, N, K, _ptr(y), flags,
                                           _stream(stream)))


def w8a32_gemv(w, s_w, bias, x, y, flags: int = 0, stream=None):
    """Weight-only per-row INT8 (w8_repack layout) on float x [M][K], M <= 4; y[M][N]."""
    _dev(w, s_w, bias, x, y)
    M, K = x.shape
    N = y.shape[1]
    _check("w8a32_gemv", load().w8a32_gemv(_ptr(w), _ptr(s_w), _ptr(bias), _ptr(x), M, N, K, _ptr(y), flags,
                                           _stream(stream)))


# -------------------------------------------- INT8 x INT8, any number of tokens
def _check_tensors(*specs):
    """Each spec: (name, tensor or None, dtypes, shape or None).  Contiguous, of one of the dtypes, of the shape, on the
    current CUDA device."""
    cur = None
    for name, t, dtypes, shape in specs:
        if t is None:
            continue
        at = t.get_device()
        if at < 0:
            raise ValueError(f"{name}: tensor must live on a CUDA device")
        if cur is None:
            cur = torch.cuda.current_device()
        if at != cur:
            raise ValueError(f"{name}: tensor lives on {t.device}, the current device is cuda:{cur}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: tensor must be contiguous")
        if t.dtype not in dtypes:
            raise ValueError(f"{name}: dtype {t.dtype} is not one of {[str(d) for d in dtypes]}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)} is not {tuple(shape)}")
    return cur


def _addr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(stream, device):
    """The stream's handle: the given one's, or the current one's of `device`."""
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device)


def allocating_on(stream):
    """Context in which a call on `stream` (None: the current one) makes its tensors, so that the allocator orders their
    memory with that stream's work."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


_F32 = (torch.float32,)
_I8 = (torch.int8,)
_U8 = (torch.uint8,)
_FLOATS = tuple(ELEM_TYPES)


def w8a8_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(load().w8a8_workspace_bytes(M, N, K))


def _places(tensors):
    """Address and bytes of each tensor: as long as they stay, what was checked of its memory holds."""
    return [(t.data_ptr(), t.nbytes) for t in tensors]


class W8Weights:
    """Checked weights of the INT8 x INT8 linear (w8_repack), for callers that use them again and again."""
    __slots__ = ("w", "s_w", "bias", "N", "K", "device", "addr", "held", "places")

    def __init__(self, w, s_w, bias, N: int, K: int):
        self.w, self.s_w, self.bias, self.N, self.K = w, s_w, bias, N, K
        self._settle()

    def _settle(self):
        N = self.N
        self.device = _check_tensors(("w", self.w, _U8, None), ("s_w", self.s_w, _F32, (N,)), ("bias", self.bias, _F32, (N,)))
        need = w8_repacked_bytes(N, self.K)
        if self.w.numel() < need:
            raise ValueError(f"w: {self.w.numel()} bytes, {need} are needed")
        self.addr = (_addr(self.w), _addr(self.s_w), _addr(self.bias))
        self.held = tuple(t for t in (self.w, self.s_w, self.bias) if t is not None)
        self.places = _places(self.held)

    def addresses(self):
        """Where the weights are now: a tensor may have got other memory since the last call, which is checked then."""
        if _places(self.held) != self.places:
            self._settle()
        return self.addr


def w8a8_matmul(w, s_w, bias, qx, sx, y, workspace, stream=None):
    """y [M][N] (fp32, fp16 or bf16) from per-row INT8 weights (w8_repack) and int8 codes qx [M][K], sx [M]."""
    M, K = qx.shape
    N = y.shape[1]
    weights = W8Weights(w, s_w, bias, N, K)
    dev = _check_tensors(("qx", qx, _I8, None), ("sx", sx, _F32, (M,)), ("y", y, _FLOATS, (M, N)),
                         ("workspace", workspace, _U8, None))
    _check("w8a8_matmul", load().w8a8_matmul(*weights.addr, _addr(qx), _addr(sx), M, N, K, _addr(y),
                                             ELEM_TYPES[y.dtype], _addr(workspace), workspace.numel(), _raw_stream(stream, dev)))


def w8a8_linear(w, s_w, bias, x, y, qx, sx, workspace, norm=None, eps: float = 0.0, residual=None, flags: int = 0,
                stream=None):
    """Quantize x [M][K] (fp32, fp16 or bf16; RMSNorm first with norm) and form y [M][N] (any of the three types)
    from per-row INT8 weights, for any number of tokens; residual float32 [M][N] is added before the rounding.
    qx: int8 [M][K] to receive the codes, or None."""
    w8a8_linear_on(W8Weights(w, s_w, bias, y.shape[1], x.shape[1]), x, y, qx, sx, workspace, norm, eps, residual, flags, stream)


def w8a8_linear_on(weights: W8Weights, x, y, qx, sx, workspace, norm=None, eps: float = 0.0, residual=None, flags: int = 0,
                   stream=None):
    """w8a8_linear on weights that were checked before."""
    M, K = x.shape
    N = weights.N
    if K != weights.K:
        raise ValueError(f"x has {K} columns, the linear takes {weights.K}")
    dev = _check_tensors(("x", x, _FLOATS, None), ("y", y, _FLOATS, (M, N)), ("qx", qx, _I8, (M, K)), ("sx", sx, _F32, (M,)),
                         ("workspace", workspace, _U8, None), ("norm", norm, _F32, (K,)), ("residual", residual, _F32, (M, N)))
    addr = weights.addresses()
    if weights.device != dev:
        raise ValueError(f"the weights live on cuda:{weights.device}, the current device is cuda:{dev}")
    fz = None
    if norm is not None or residual is not None:
        fz = ctypes.byref(Fusion(None if norm is None else norm.data_ptr(), float(eps), W4_GLU_NONE,
                                 None if residual is None else residual.data_ptr()))
    _check("w8a8_linear", load().w8a8_linear(*addr, x.data_ptr(), ELEM_TYPES[x.dtype], M, N, K,
                                             y.data_ptr(), ELEM_TYPES[y.dtype], _addr(qx), _addr(sx), fz, flags,
                                             workspace.data_ptr(), workspace.numel(), _raw_stream(stream, dev)))


# ------------------------------------------------- mixture of experts, few tokens
def w8_glu_repacked_bytes(I: int, K: int) -> int:
    return int(load().w8_glu_repacked_bytes(I, K))


def w8_repack_glu(gate, up, K, out, stream=None):
    """int8 codes of gate and up [I][K] -> the paired device layout (the experts of w4_moe_experts)."""
    dev = _check_tensors(("gate", gate, _I8, None), ("up", up, _I8, gate.shape), ("out", out, _U8, None))
    _check("w8_repack_glu", load().w8_repack_glu(_addr(gate), _addr(up), gate.shape[0], K, _addr(out), out.numel(),
                                                 _raw_stream(stream, dev)))


_I32 = (torch.int32,)


def _settle(desc):
    """Checks a descriptor's tensors and takes their addresses."""
    desc._device = _check_tensors(*((name, t, dtypes, shape) for (_, name, dtypes, shape), t in zip(desc._specs, desc._tensors)))
    for (field, *_), t in zip(desc._specs, desc._tensors):
        setattr(desc, field, _addr(t))
    desc._held = tuple(t for t in desc._tensors if t is not None)
    desc._places = _places(desc._held)
    return desc


def moe_router(w, top_k: int, select_bias=None, score: str = "softmax", renormalize: bool = True, scale: float = 1.0,
               norm=None, eps: float = 1e-6):
    """A w4_router descriptor: w float32 [E][K].  It holds references to its tensors."""
    E, K = w.shape
    if score not in ROUTE_SCORES:
        raise ValueError(f"score {score!r} is not one of {sorted(ROUTE_SCORES)}")
    r = Router(norm_eps=float(eps), E=E, top_k=int(top_k), score=ROUTE_SCORES[score], renormalize=int(bool(renormalize)),
               scale=float(scale))
    r._tensors, r._K = (w, select_bias, norm), K
    r._specs = (("w", "w", _F32, (E, K)), ("select_bias", "select_bias", _F32, (E,)), ("norm_weight", "norm", _F32, (K,)))
    return _settle(r)


def moe_experts(fmt: str, w_gu, s_gu, w_dn, s_dn, E: int, n_shared: int, H: int, I: int, glu: int, b_gu=None, b_dn=None):
    """A w4_experts descriptor over the repacked weights of E + n_shared experts.  It holds references to its tensors."""
    if fmt not in EXPERT_FORMATS:
        raise ValueError(f"experts are {sorted(EXPERT_FORMATS)}, not {fmt!r}")
    n = E + n_shared
    gu_bytes, dn_bytes = ((w4_glu_repacked_bytes(I, H), w4_repacked_bytes(H, I)) if fmt == "w4"
                          else (w8_glu_repacked_bytes(I, H), w8_repacked_bytes(H, I)))
    e = Experts(fmt=EXPERT_FORMATS[fmt], E=E, n_shared=n_shared, H=H, I=I, glu=glu)
    e._tensors = (w_gu, s_gu, b_gu, w_dn, s_dn, b_dn)
    e._specs = (("w_gu", "w_gu", _U8, (n * gu_bytes,)), ("s_gu", "s_gu", _F32, (n, 2 * I)), ("b_gu", "b_gu", _F32, (n, 2 * I)),
                ("w_dn", "w_dn", _U8, (n * dn_bytes,)), ("s_dn", "s_dn", _F32, (n, H)), ("b_dn", "b_dn", _F32, (n, H)))
    return _settle(e)


def _check_home(dev, *descs):
    """The descriptors' tensors, wherever their memory is now, are on the current device."""
    for d in descs:
        if _places(d._held) != d._places:
            _settle(d)
        if d._device != dev:
            raise ValueError(f"the descriptor's tensors live on cuda:{d._device}, the current device is cuda:{dev}")


def w4_moe_route(router, x, ids, weights, qx=None, sx=None, flags: int = 0, stream=None):
    """ids int32 [M][top_k] and weights float32 [M][top_k] of x [M][K]; qx int8 [M][K] and sx float32 [M] receive the
    (normalized) tokens' codes and scales, or are both None."""
    M, K = x.shape
    if K != router._K:
        raise ValueError(f"x has {K} columns, the router takes {router._K}")
    dev = _check_tensors(("x", x, _FLOATS, None), ("ids", ids, _I32, (M, router.top_k)),
                         ("weights", weights, _F32, (M, router.top_k)), ("qx", qx, _I8, (M, K)),
                         ("sx", sx, _F32, (M,)))
    _check_home(dev, router)
    _check("w4_moe_route", load().w4_moe_route(ctypes.byref(router), _addr(x), ELEM_TYPES[x.dtype], M, K, _addr(ids),
                                               _addr(weights), _addr(qx), _addr(sx), flags, _raw_stream(stream, dev)))


def w4_moe_workspace_bytes(experts, M: int, top_k: int) -> int:
    return int(load().w4_moe_workspace_bytes(ctypes.byref(experts), M, top_k))


def w4_moe_experts(experts, qx, sx, ids, weights, y, workspace, residual=None, flags: int = 0, stream=None):
    """y [M][H] of the experts ids [M][top_k] with weights, on codes qx [M][H], sx [M]."""
    M, top_k = ids.shape
    H = experts.H
    dev = _check_tensors(("qx", qx, _I8, (M, H)), ("sx", sx, _F32, (M,)), ("ids", ids, _I32, None),
                         ("weights", weights, _F32, (M, top_k)), ("y", y, _FLOATS, (M, H)),
                         ("workspace", workspace, _U8, None), ("residual", residual, _F32, (M, H)))
    _check_home(dev, experts)
    _check("w4_moe_experts", load().w4_moe_experts(ctypes.byref(experts), _addr(qx), _addr(sx), _addr(ids), _addr(weights), M,
                                                   top_k, _addr(residual), _addr(y), ELEM_TYPES[y.dtype], _addr(workspace),
                                                   workspace.numel(), flags, _raw_stream(stream, dev)))


def w4_moe_layer(router, experts, x, ids, weights, qx, sx, y, workspace, residual=None, flags: int = 0, stream=None):
    """w4_moe_route on x [M][H], then w4_moe_experts on its choice, in two launches."""
    M, H = x.shape
    if H != router._K or H != experts.H:
        raise ValueError(f"x has {H} columns, the router takes {router._K}, the experts {experts.H}")
    dev = _check_tensors(("x", x, _FLOATS, None), ("ids", ids, _I32, (M, router.top_k)),
                         ("weights", weights, _F32, (M, router.top_k)), ("qx", qx, _I8, (M, H)),
                         ("sx", sx, _F32, (M,)), ("y", y, _FLOATS, (M, H)), ("workspace", workspace, _U8, None),
                         ("residual", residual, _F32, (M, H)))
    _check_home(dev, router, experts)
    _check("w4_moe_layer", load().w4_moe_layer(ctypes.byref(router), ctypes.byref(experts), _addr(x), ELEM_TYPES[x.dtype], M,
                                               _addr(ids), _addr(weights), _addr(qx), _addr(sx), _addr(residual), _addr(y),
                                               ELEM_TYPES[y.dtype], _addr(workspace), workspace.numel(), flags,
                                               _raw_stream(stream, dev)))


# --------------------------------------- attention over a paged cache, and logits
_CACHES = tuple(CACHE_TYPES)
_HALVES = (torch.float16, torch.bfloat16)
_I64 = (torch.int64,)
_F64 = (torch.float64,)


def _check_rows(name, t, dtypes, width=None):
    """A 2-D tensor whose rows are contiguous (they may be apart): the current CUDA device and the rows' distance."""
    at = t.get_device()
    if at < 0:
        raise ValueError(f"{name}: tensor must live on a CUDA device")
    if at != torch.cuda.current_device():
        raise ValueError(f"{name}: tensor lives on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} is not one of {[str(d) for d in dtypes]}")
    if t.dim() != 2 or (width is not None and t.shape[1] != width):
        raise ValueError(f"{name}: shape {tuple(t.shape)} is not rows of {width}")
    n, w = t.shape
    if w > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the values of a row must be contiguous")
    if n > 1 and t.stride(0) < w:
        raise ValueError(f"{name}: rows overlap")
    return at, t.stride(0) if n > 1 else w


def _fits(dev, t, dtypes, shape):
    """What _check_tensors asks of one tensor, as one truth value: a call takes 0.4 us for each where it takes 0.6."""
    return t.get_device() == dev and t.dtype in dtypes and t.shape == shape and t.is_contiguous()


def _row_distance(dev, name, t, dtypes, width):
    """_check_rows for the rows' distance, short where the tensor is contiguous."""
    if t.is_contiguous() and t.dim() == 2 and t.shape[1] == width and t.dtype in dtypes and t.get_device() == dev:
        return width
    return _check_rows(name, t, dtypes, width)[1]


def _with_ref(desc):
    """A settled descriptor that keeps its own reference for the calls."""
    desc._ref = ctypes.byref(desc)
    return _settle(desc)


def kv_cache(k, v, k_scale=None, v_scale=None):
    """A w4_kv_cache descriptor: k and v [pages][Hkv][page_size][D] of fp16, bf16 or int8 codes with scales float32
    [pages][Hkv][page_size].  It holds references to its tensors."""
    if k.dim() != 4:
        raise ValueError(f"k: shape {tuple(k.shape)} is not [pages][heads][page_size][head_dim]")
    if (k.dtype == torch.int8) != (k_scale is not None) or (k.dtype == torch.int8) != (v_scale is not None):
        raise ValueError("an int8 cache has scales for keys and values, a 16-bit cache has none")
    pages, heads, page_size, D = k.shape
    c = KVCacheDesc(type=CACHE_TYPES.get(k.dtype, -1), pages=pages, page_size=page_size, Hkv=heads, D=D)
    c._tensors = (k, v, k_scale, v_scale)
    c._specs = (("k", "k", _CACHES, k.shape), ("v", "v", (k.dtype,), k.shape), ("k_scale", "k_scale", _F32, k.shape[:3]),
                ("v_scale", "v_scale", _F32, k.shape[:3]))
    return _with_ref(c)


def kv_batch(table, ctx, q_start, max_tokens: int):
    """A w4_kv_batch descriptor: table int32 [B][max_pages], ctx int32 [B], q_start int32 [B + 1], all on the device.  It
    holds references to its tensors."""
    if table.dim() != 2:
        raise ValueError(f"table: shape {tuple(table.shape)} is not [sequences][pages]")
    B, max_pages = table.shape
    b = KVBatchDesc(B=B, max_pages=max_pages, max_tokens=int(max_tokens))
    b._tensors = (table, ctx, q_start)
    b._specs = (("table", "table", _I32, (B, max_pages)), ("ctx", "ctx", _I32, (B,)), ("q_start", "q_start", _I32, (B + 1,)))
    return _with_ref(b)


def rope_desc(turns, layout: str = "half"):
    """A w4_rope descriptor over turns float32 [positions][rot / 2][2].  It holds a reference to its tensor."""
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout {layout!r} is not one of {sorted(ROPE_LAYOUTS)}")
    if turns.dim() != 3 or turns.shape[2] != 2:
        raise ValueError(f"turns: shape {tuple(turns.shape)} is not [positions][rot / 2][2]")
    r = RopeDesc(positions=turns.shape[0], rot=2 * turns.shape[1], layout=ROPE_LAYOUTS[layout])
    r._tensors, r._specs = (turns,), (("turns", "turns", _F32, tuple(turns.shape)),)
    return _with_ref(r)


def w4_rope_table(inv_freq, turns, factor: float = 1.0, scale: float = 1.0, stream=None):
    """turns float32 [positions][rot / 2][2]: (cos, sin) of position * factor * inv_freq (float64 [rot / 2]), times scale."""
    positions, half, _ = turns.shape
    dev = _check_tensors(("inv_freq", inv_freq, _F64, (half,)), ("turns", turns, _F32, (positions, half, 2)))
    _check("w4_rope_table", load().w4_rope_table(_addr(inv_freq), float(factor), float(scale), positions, 2 * half, _addr(turns),
                                                 _raw_stream(stream, dev)))


def w4_kv_append(cache, batch, rope, qkv, q, positions=None, q_norm=None, k_norm=None, eps: float = 1e-6, flags: int = 0,
                 stream=None):
    """Rows qkv [T][(Hq + 2 Hkv) D] (fp32, fp16 or bf16; rows may be apart): norms and rotation of q [T][Hq][D] (fp16 or
    bf16) and of the keys, which go to the cache with the values.  positions: int32 [T] or None."""
    dev, D, s = torch.cuda.current_device(), cache.D, q.shape
    if len(s) != 3 or s[2] != D:
        raise ValueError(f"q: shape {tuple(s)} is not [rows][heads][{D}]")
    T, Hq, _ = s
    ld = _row_distance(dev, "qkv", qkv, _FLOATS, (Hq + 2 * cache.Hkv) * D)
    if not (qkv.shape[0] == T and _fits(dev, q, _HALVES, s) and (positions is None or _fits(dev, positions, _I32, (T,)))
            and (q_norm is None or _fits(dev, q_norm, _F32, (D,))) and (k_norm is None or _fits(dev, k_norm, _F32, (D,)))):
        _check_tensors(("q", q, _HALVES, (qkv.shape[0], Hq, D)), ("positions", positions, _I32, (T,)), ("q_norm", q_norm, _F32, (D,)),
                       ("k_norm", k_norm, _F32, (D,)))
    if rope is None:
        _check_home(dev, cache, batch)
    else:
        _check_home(dev, cache, batch, rope)
    st = load().w4_kv_append(cache._ref, batch._ref, None if rope is None else rope._ref, qkv.data_ptr(), ELEM_TYPES[qkv.dtype], ld, T, Hq,
                             _addr(positions), _addr(q_norm), _addr(k_norm), eps, q.data_ptr(), ELEM_TYPES[q.dtype], flags,
                             _raw_stream(stream, dev))
    if st != W4_OK:
        raise W4Error("w4_kv_append", st)


def w4_kv_values(cache, which: str, out, stream=None):
    """out float32 [pages][Hkv][page_size][D]: an int8 cache's keys ("k") or values ("v"), codes times scales."""
    dev = _check_tensors(("out", out, _F32, (cache.pages, cache.Hkv, cache.page_size, cache.D)))
    _check_home(dev, cache)
    _check("w4_kv_values", load().w4_kv_values(ctypes.byref(cache), {"k": 0, "v": 1}[which], out.data_ptr(), _raw_stream(stream, dev)))


def w4_tree_attention_workspace_bytes(cache, batch, T: int, Hq: int) -> int:
    return int(load().w4_tree_attention_workspace_bytes(ctypes.byref(cache), ctypes.byref(batch), T, Hq))


def _attention_tensors(cache, batch, q, y, workspace, mask):
    """Checks the tensors of a tree attention: their device, T and Hq."""
    dev, D, s = torch.cuda.current_device(), cache.D, q.shape
    if len(s) != 3 or s[2] != D:
        raise ValueError(f"q: shape {tuple(s)} is not [rows][heads][{D}]")
    T, Hq, _ = s
    if not (_fits(dev, q, _HALVES, s) and _fits(dev, y, _FLOATS, s) and (mask is None or _fits(dev, mask, _I64, (T,)))
            and _fits(dev, workspace, _U8, workspace.shape)):
        _check_tensors(("q", q, _HALVES, None), ("y", y, _FLOATS, s), ("mask", mask, _I64, (T,)), ("workspace", workspace, _U8, None))
    _check_home(dev, cache, batch)
    return dev, T, Hq


def check_tree_attention(cache, batch, q, y, workspace, mask=None, scale: float = None):
    """Raises what w4_tree_attention would, and launches nothing: for a caller that writes the cache first.  The tensors'
    device, rows and heads, for launch_tree_attention."""
    home = _attention_tensors(cache, batch, q, y, workspace, mask)
    _, T, Hq = home
    if T == 0 or batch.B == 0:
        return home
    need = w4_tree_attention_workspace_bytes(cache, batch, T, Hq)
    if need == 0 or workspace.numel() < need:
        raise W4Error("w4_tree_attention", W4_UNSUPPORTED_SHAPE)
    if (cache.type != CACHE_TYPES[torch.int8] and ELEM_TYPES[q.dtype] != cache.type) or not (scale is None or 0.0 < scale < 2e38):
        raise W4Error("w4_tree_attention", W4_INVALID_ARG)
    if (q.data_ptr() | y.data_ptr() | workspace.data_ptr()) % 16 or (mask is not None and mask.data_ptr() % 8):
        raise W4Error("w4_tree_attention", W4_MISALIGNED)
    return home


def launch_tree_attention(home, cache, batch, q, y, workspace, mask, scale, flags, stream):
    """w4_tree_attention of tensors that are checked."""
    dev, T, Hq = home
    st = load().w4_tree_attention(cache._ref, batch._ref, q.data_ptr(), ELEM_TYPES[q.dtype], T, Hq, _addr(mask),
                                  cache.D ** -0.5 if scale is None else scale, y.data_ptr(), ELEM_TYPES[y.dtype], workspace.data_ptr(),
                                  workspace.numel(), flags, _raw_stream(stream, dev))
    if st != W4_OK:
        raise W4Error("w4_tree_attention", st)


def w4_tree_attention(cache, batch, q, y, workspace, mask=None, scale: float = None, flags: int = 0, stream=None):
    """y [T][Hq][D] (fp32, fp16 or bf16) of q [T][Hq][D] over the cache; mask int64 [T]: bit j is the sequence's row j
    (None: a row sees the rows up to itself); scale: 1 / sqrt(D) if None."""
    launch_tree_attention(_attention_tensors(cache, batch, q, y, workspace, mask), cache, batch, q, y, workspace, mask, scale, flags,
                          stream)


def logit_rules(vocab: int, ids=None, length=None, prompt=None, repetition=None, frequency=None, presence=None, bias_ids=None,
                bias=None, sequences: int = None):
    """A w4_logit_rules descriptor: ids int32 [S][cap], length and prompt int32 [S], factors float32 [S], bias_ids int32 and
    bias float32 [S][n_bias].  It holds references to its tensors."""
    if (ids is None) != (length is None) or (ids is None and prompt is not None):
        raise ValueError("ids and length come together, prompt with them")
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias_ids and bias come together")
    S, cap, nb = sequences, 0, 0
    for t in (ids, repetition, frequency, presence, bias_ids):
        if t is not None and S is None:
            S = t.shape[0]
    if S is None:
        raise ValueError("the number of sequences is not known: give sequences")
    if ids is not None:
        cap = ids.shape[1] if ids.dim() == 2 else -1
    if bias_ids is not None:
        nb = bias_ids.shape[1] if bias_ids.dim() == 2 else -1
    if cap < 0 or nb < 0:
        raise ValueError("ids and bias_ids are [sequences][entries]")
    u = LogitRulesDesc(V=int(vocab), S=S, cap=cap, n_bias=nb)
    u._tensors = (ids, length, prompt, repetition, frequency, presence, bias_ids, bias)
    u._specs = (("ids", "ids", _I32, (S, cap)), ("length", "length", _I32, (S,)), ("prompt", "prompt", _I32, (S,)),
                ("repetition", "repetition", _F32, (S,)), ("frequency", "frequency", _F32, (S,)),
                ("presence", "presence", _F32, (S,)), ("bias_ids", "bias_ids", _I32, (S, nb)), ("bias", "bias", _F32, (S, nb)))
    return _with_ref(u)


def w4_logits_adjust(rules, logits, out, row_start=None, drafts=None, mask=None, allowed=None, flags: int = 0, stream=None):
    """out [R][V] = logits [R][V] (fp32, fp16 or bf16; rows may be apart) after penalties, biases and the grammar's mask:
    allowed int32 [R][ceil(V / 32)]; row_start int32 [S + 1], drafts int32 [R] and mask int64 [R] for drafted trees."""
    dev, V, R, kind = torch.cuda.current_device(), rules.V, logits.shape[0], logits.dtype
    ld = _row_distance(dev, "logits", logits, _FLOATS, V)
    ld_out = _row_distance(dev, "out", out, (kind,), V)
    if out.shape[0] != R:
        raise ValueError(f"out: {out.shape[0]} rows, logits have {R}")
    if not ((row_start is None or _fits(dev, row_start, _I32, (rules.S + 1,))) and (drafts is None or _fits(dev, drafts, _I32, (R,)))
            and (mask is None or _fits(dev, mask, _I64, (R,))) and (allowed is None or _fits(dev, allowed, _I32, (R, (V + 31) // 32)))):
        _check_tensors(("row_start", row_start, _I32, (rules.S + 1,)), ("drafts", drafts, _I32, (R,)), ("mask", mask, _I64, (R,)),
                       ("allowed", allowed, _I32, (R, (V + 31) // 32)))
    if rules._held:
        _check_home(dev, rules)
    st = load().w4_logits_adjust(rules._ref, logits.data_ptr(), ELEM_TYPES[kind], ld, R, _addr(row_start), _addr(drafts), _addr(mask),
                                 _addr(allowed), out.data_ptr(), ld_out, flags, _raw_stream(stream, dev))
    if st != W4_OK:
        raise W4Error("w4_logits_adjust", st)


# ---------------------------------------------------------------- chains
def chain_workspace_bytes() -> int:
    return int(load().w4_chain_workspace_bytes())


def make_chain_descs(items):
    """items: sequence of (w, s_w, bias, x, y, qx, sx) tensors (bias, qx, sx may be None)."""
    arr = (LinearDesc * len(items))()
    for i, (w, s_w, bias, x, y, qx, sx) in enumerate(items):
        _dev(w, s_w, bias, x, y, qx, sx)
        arr[i] = LinearDesc(w.data_ptr(), s_w.data_ptr(), None if bias is None else bias.data_ptr(), x.data_ptr(),
                            y.data_ptr(), None if qx is None else qx.data_ptr(),
                            None if sx is None else sx.data_ptr(), y.shape[1], x.shape[1])
    return arr


def w4a8_linear_chain(descs, M: int, workspace, stream=None):
    """Run a chain of per-row INT4 linears (descs from make_chain_descs) in one launch."""
    _dev(workspace)
    _check("w4a8_linear_chain", load().w4a8_linear_chain(descs, len(descs), M, _ptr(workspace),
                                                         workspace.numel() * workspace.element_size(),
                                                         _stream(stream)))


def w4a8_linear_chain_noalloc(descs, M: int, stream=None):
    """w4a8_linear_chain with the library's own fixed barrier scratch: for
    callers that cannot allocate device memory.  Calls sharing the scratch
    must not overlap on the GPU."""
    _check("w4a8_linear_chain_noalloc", load().w4a8_linear_chain_noalloc(descs, len(descs), M, _stream(stream)))


# ---------------------------------------------------------- device errors
def device_error() -> int:
    code = ctypes.c_uint(0)
    st = load().w4_device_error(ctypes.byref(code))
    if st not in (W4_OK, 5):
        raise W4Error("w4_device_error", st)
    return int(code.value)


def last_device_error() -> int:
    """w4_last_device_error: the same word as device_error()."""
    code = ctypes.c_uint(0)
    st = load().w4_last_device_error(ctypes.byref(code))
    if st not in (W4_OK, 5):
        raise W4Error("w4_last_device_error", st)
    return int(code.value)


def hbm_read(buf, sink, stream=None):
    """Stream every byte of the device tensor `buf` once (w4_hbm_read); sink:
    a device int32 [1] that receives the XOR of all 32-bit words."""
    _dev(buf, sink)
    _check("w4_hbm_read", load().w4_hbm_read(_ptr(buf), buf.numel() * buf.element_size(), _ptr(sink),
                                             _stream(stream)))


def selftest_wait_timeout(cluster: bool, timeout_us: int, stream=None):
    """A kernel whose bounded wait nothing completes: it gives up after
    timeout_us and sets the device error word to the wait-timeout code."""
    _check("w4_selftest_wait_timeout", load().w4_selftest_wait_timeout(1 if cluster else 0, int(timeout_us),
                                                                        _stream(stream)))


WAIT_TIMEOUT_CODE = 0x57414954


def clear_device_error():
    _check("w4_clear_device_error", load().w4_clear_device_error())
