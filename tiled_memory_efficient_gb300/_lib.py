"""ctypes binding of the C ABI in include/attn.h, ffn.h, kvcache.h and rope.h (argument
marshalling only).

Every step of the computation runs in libattn.so's CUDA kernels; torch is used
only to own device memory and to name the current stream.  There is no CPU
fallback: if the library is missing or the device is not an sm_103 GPU, the
calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
import re
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "_build", "libattn.so")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
HEADERS = [os.path.join(INCLUDE, "attn.h"), os.path.join(INCLUDE, "ffn.h"),
           os.path.join(INCLUDE, "kvcache.h"), os.path.join(INCLUDE, "rope.h")]

ATTN_OK = 0
ATTN_ERR_INVALID = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_ALIGN = 3
ATTN_ERR_CUDA = 4
ATTN_ERR_TIMEOUT = 5
ATTN_ERR_WORKSPACE = 6
ATTN_ERR_MISMATCH = 7
ATTN_ERR_PAGE = 8
ATTN_ERR_POOL = 9
FFN_ACTS = {"none": 0, "relu": 1, "gelu_tanh": 2, "silu": 3, "swiglu": 4}
ATTN_F16 = 0
ATTN_BF16 = 1
ATTN_CAUSAL_NONE = 0
ATTN_CAUSAL_TOP_LEFT = 1
ATTN_CAUSAL_BOTTOM_RIGHT = 2
ATTN_MASK_BOOL = 1
ATTN_MASK_ADDITIVE = 2
_CAUSAL_NAMES = {"none": ATTN_CAUSAL_NONE, "top_left": ATTN_CAUSAL_TOP_LEFT,
                 "bottom_right": ATTN_CAUSAL_BOTTOM_RIGHT}

_lock = threading.Lock()
_lib = None

_vp = ctypes.c_void_p
_i = ctypes.c_int
_SIGNATURES = {
    "attn_fwd": ([_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, ctypes.c_float, _i, _i, _vp],
                 _i),
    "attn_fwd_masked": ([_vp, _vp, _vp, _vp, _vp, _vp, _i, ctypes.c_longlong, ctypes.c_longlong,
                         ctypes.c_longlong, _i, _i, _i, _i, _i, _i, ctypes.c_float, _i, _i, _vp],
                        _i),
    "attn_fwd_window": ([_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _i, _i, _i, _i, _i, _i,
                         ctypes.c_float, _i, _i, _i, _vp], _i),
    "attn_fwd_window_workspace_size": ([_i, _i, _i, _i, _i, _i, _i, _i, _i], ctypes.c_size_t),
    "attn_bwd_window": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                         _i, _i, _i, _i, _i, _i, ctypes.c_float, _i, _i, _i, _vp], _i),
    "attn_bwd_window_workspace_size": ([_i, _i, _i, _i, _i, _i, _i, _i, _i], ctypes.c_size_t),
    "attn_fwd_splitkv": ([_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _i, _i, _i, _i, _i, _i,
                          ctypes.c_float, _i, _i, _i, _vp], _i),
    "attn_fwd_splitkv_workspace_size": ([_i, _i, _i, _i, _i, _i, _i], ctypes.c_size_t),
    "attn_fwd_ws": ([_vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _i, _i, _i, _i, _i, _i,
                     ctypes.c_float, _i, _i, _vp], _i),
    "attn_fwd_workspace_size": ([_i, _i, _i, _i, _i, _i, _i], ctypes.c_size_t),
    "attn_fwd_ws_splits": ([_i, _i, _i, _i, _i, _i, _i, _i], _i),
    "attn_fwd_half_positions": ([_i, _i, _i, _i, _i, _i, _i, _i, _i], _i),
    "attn_bwd_splits": ([_i, _i, _i, _i, _i, _i, _i, _i], _i),
    "attn_fwd_num_splits": ([_i, _i, _i, _i, _i, _i, _i], _i),
    "attn_bwd_workspace_size": ([_i, _i, _i, _i, _i, _i, _i], ctypes.c_size_t),
    "attn_bwd": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                  _i, _i, _i, _i, _i, _i, ctypes.c_float, _i, _i, _vp], _i),
    "attn_bwd_masked": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp,
                         _i, ctypes.c_longlong, ctypes.c_longlong, ctypes.c_longlong,
                         _i, _i, _i, _i, _i, _i, ctypes.c_float, _i, _i, _vp], _i),
    "attn_bwd_noalloc": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                          _i, _i, _i, _i, _i, _i, ctypes.c_float, _i, _i, _vp], _i),
    "attn_sync_status": ([_vp], _i),
    "ffn_workspace_size": ([_i, _i, _i], ctypes.c_size_t),
    "ffn_forward": ([_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, ctypes.c_size_t, _i,
                     _vp], _i),
    "ffn_check_chunking": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp,
                            ctypes.c_size_t, _i, _vp], _i),
    "kv8_append": ([_vp] * 9 + [_i] * 7 + [ctypes.c_longlong] * 3 + [_i, _vp], _i),
    "kv8_append_step": ([_vp] * 10 + [_i] * 7 + [ctypes.c_longlong] * 3 + [_i, _vp], _i),
    "kv8_attn": ([_vp] * 10 + [ctypes.c_size_t] + [_i] * 8 + [ctypes.c_float, _i, _i, _i, _vp], _i),
    "kv8_attn_step": ([_vp] * 12 + [ctypes.c_size_t] + [_i] * 8 + [ctypes.c_float, _i, _i, _i, _vp], _i),
    "kv8_attn_workspace_size": ([_i] * 5, ctypes.c_size_t),
    "kv8_copy_pages": ([_vp] * 7 + [_i] * 6 + [_vp], _i),
    "kvp_reserve": ([_vp] * 4 + [_i] * 6 + [_vp, _vp, ctypes.c_size_t, _vp], _i),
    "kvp_reserve_step": ([_vp] * 4 + [_i] * 6 + [_vp] * 3 + [ctypes.c_size_t, _vp], _i),
    "kvp_reassign": ([_vp] * 4 + [_i] * 4 + [_vp] * 4 + [ctypes.c_size_t, _vp], _i),
    "kvp_compact": ([_vp] * 4 + [_i] * 3 + [_vp] * 4 + [ctypes.c_size_t, _vp], _i),
    "kvp_workspace_size": ([_i] * 3, ctypes.c_size_t),
    "rope_apply": ([_vp] * 6 + [_i] * 8 + [ctypes.c_float, _i, _vp, _i, _vp], _i),
    "kv8_append_rope": ([_vp] * 13 + [_i, _i, ctypes.c_float] + [_i] * 8 + [_vp, _i, _vp], _i),
    "kv8_attn_shared": ([_vp] * 13 + [ctypes.c_size_t] + [_i] * 8 + [ctypes.c_float, _i, _vp], _i),
    "kv8_attn_shared_workspace_size": ([_i] * 5, ctypes.c_size_t),
    "kvp_find_shared": ([_vp] * 2 + [_i] * 4 + [_vp, _vp], _i),
    "kvp_plan_words": ([_i], ctypes.c_size_t),
    "attn_selftest_timeout": ([ctypes.c_ulonglong, _vp], _i),
    "attn_strerror": ([_i], ctypes.c_char_p),
    "attn_version": ([], _i),
}


class AttnError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed: {code} ({strerror(code)})")


def declared_functions() -> list:
    """Names of the functions include/attn.h, ffn.h, kvcache.h and rope.h declare."""
    names = set()
    for h in HEADERS:
        text = re.sub(r"/\*.*?\*/", "", open(h).read(), flags=re.S)
        names.update(re.findall(r"\b((?:attn|ffn|kv8|kvp|rope)_[a-z0-9_]+)\s*\(", text))
    return sorted(names)


def load(path: str | None = None):
    """dlopen libattn.so (built by __graft_entry__.build()) and set signatures."""
    global _lib
    with _lock:
        if _lib is None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(f"{p} is missing: run __graft_entry__.build() first")
            lib = ctypes.CDLL(p)
            for name, (args, res) in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.argtypes = args
                fn.restype = res
            _lib = lib
    return _lib


def strerror(code: int) -> str:
    return load().attn_strerror(code).decode()


def _stream_handle(device) -> int:
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float16:
        return ATTN_F16
    if t.dtype == torch.bfloat16:
        return ATTN_BF16
    raise TypeError(f"unsupported dtype {t.dtype}: use float16 or bfloat16")


def causal_code(causal) -> int:
    """Mask code of the C ABI: False/None -> none, True -> top-left (the SDPA
    is_causal convention), or one of "none", "top_left", "bottom_right", or
    the integer code itself."""
    if causal is None or causal is False:
        return ATTN_CAUSAL_NONE
    if causal is True:
        return ATTN_CAUSAL_TOP_LEFT
    if isinstance(causal, str):
        if causal not in _CAUSAL_NAMES:
            raise ValueError(f"causal must be one of {sorted(_CAUSAL_NAMES)}, got {causal!r}")
        return _CAUSAL_NAMES[causal]
    return int(causal)


def _check(q, k, v):
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous [B, H, N, D]")
        if t.dim() != 4:
            raise ValueError(f"{name} must be 4-D [B, H, N, D]")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k, v must share one dtype")
    if k.shape != v.shape or k.shape[0] != q.shape[0] or k.shape[3] != q.shape[3]:
        raise ValueError(f"shapes q{tuple(q.shape)} k{tuple(k.shape)} v{tuple(v.shape)}")


def prepare_mask(mask, q, Nk: int):
    """An SDPA attn_mask as the C ABI's (tensor, kind, strides): bool stays a
    byte mask (True keeps the key); a floating mask becomes an additive bias
    in q's dtype.  It must broadcast to [B, Hq, Nq, Nk].  If its rows are not
    16-byte aligned it is copied into a padded buffer (same values),
    allocated on the current stream, the one the kernel runs on."""
    import torch
    B, Hq, Nq, _ = q.shape
    if not isinstance(mask, torch.Tensor) or mask.device != q.device:
        raise ValueError("attn_mask must be a tensor on q's device")
    if mask.dtype == torch.bool:
        kind, m = ATTN_MASK_BOOL, mask
    elif mask.is_floating_point():
        kind, m = ATTN_MASK_ADDITIVE, mask.to(q.dtype)
    else:
        raise TypeError(f"attn_mask dtype {mask.dtype} is neither bool nor floating point")
    while m.dim() < 4:
        m = m.unsqueeze(0)
    if m.dim() != 4 or m.shape[-1] != Nk or any(
            d not in (1, full) for d, full in zip(m.shape[:3], (B, Hq, Nq))):
        raise ValueError(f"attn_mask shape {tuple(mask.shape)} does not broadcast to "
                         f"{(B, Hq, Nq, Nk)}")
    if m.stride(-1) != 1:
        m = m.contiguous()
    esz = m.element_size()

    def strides(t):
        return [0 if t.shape[i] == 1 else t.stride(i) for i in range(3)]
    st = strides(m)
    if m.data_ptr() % 16 or any((x * esz) % 16 for x in st):
        per = 16 // esz
        buf = torch.zeros((*m.shape[:3], (Nk + per - 1) // per * per), dtype=m.dtype,
                          device=m.device)
        buf[..., :Nk] = m
        m = buf
        st = strides(m)
    return m, kind, st


def attn_fwd(q, k, v, causal=False, scale: float | None = None, out=None, lse=None, mask=None):
    """O, LSE = attention(q, k, v).  q [B,Hq,Nq,D]; k, v [B,Hkv,Nk,D] (CUDA).

    Returns (out [B,Hq,Nq,D] in q's dtype, lse [B,Hq,Nq] fp32 natural log).
    causal: see causal_code.  mask: optional SDPA-style attn_mask (see
    prepare_mask).  Enqueued on torch's current stream; no synchronisation.
    """
    import torch
    _check(q, k, v)
    B, Hq, Nq, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), device=q.device, dtype=torch.float32)
    if mask is not None:
        m, kind, (sb, sh, sq) = prepare_mask(mask, q, Nk)
        rc = load().attn_fwd_masked(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                    lse.data_ptr(), m.data_ptr(), kind, sb, sh, sq, B, Hq, Hkv, Nq,
                                    Nk, D, float(scale), causal_code(causal), _dtype_code(q),
                                    _stream_handle(q.device))
        if rc != ATTN_OK:
            raise AttnError("attn_fwd_masked", rc)
        # (a converted / padded copy was allocated on this stream, after which
        # the kernel is queued: the allocator reuses it only for later work
        # on the same stream, so it may be released now)
        return out, lse
    rc = load().attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                         lse.data_ptr(), B, Hq, Hkv, Nq, Nk, D, float(scale), causal_code(causal),
                         _dtype_code(q), _stream_handle(q.device))
    if rc != ATTN_OK:
        raise AttnError("attn_fwd", rc)
    return out, lse


def fwd_workspace_size(B, Hq, Hkv, Nq, Nk, D, dtype) -> int:
    """Bytes of workspace attn_fwd_ws needs on the current device (0: none)."""
    code = dtype if isinstance(dtype, int) else (ATTN_BF16 if str(dtype).endswith("bfloat16")
                                                 else ATTN_F16)
    return load().attn_fwd_workspace_size(B, Hq, Hkv, Nq, Nk, D, code)


def fwd_ws_splits(B, Hq, Hkv, Nq, Nk, D, causal=False, num_sms: int = 0) -> int:
    """Key ranges attn_fwd_ws cuts its cut units into on a device of num_sms
    SMs (0: the current device; 1: the grid is not cut, no merge kernel)."""
    return load().attn_fwd_ws_splits(B, Hq, Hkv, Nq, Nk, D, causal_code(causal), num_sms)


def fwd_half_positions(B, Hq, Hkv, Nq, Nk, D, causal=True, dtype="float16",
                       num_sms: int = 0) -> int:
    """Heaviest pair positions per head that the causal forward runs as two
    one-tile CTAs per pair (0: none; see attn_fwd_half_positions)."""
    code = dtype if isinstance(dtype, int) else (ATTN_BF16 if str(dtype).endswith("bfloat16")
                                                 else ATTN_F16)
    return load().attn_fwd_half_positions(B, Hq, Hkv, Nq, Nk, D, causal_code(causal), code,
                                          num_sms)


def bwd_splits(B, Hq, Hkv, Nq, Nk, D, causal=False, num_sms: int = 0) -> int:
    """Query ranges attn_bwd cuts the dK/dV work into with its recommended
    workspace on a device of num_sms SMs (0: the current device; 1: no
    partial-sum kernel)."""
    return load().attn_bwd_splits(B, Hq, Hkv, Nq, Nk, D, causal_code(causal), num_sms)


def attn_fwd_ws(q, k, v, causal=False, scale: float | None = None, out=None, lse=None,
                workspace=None):
    """attn_fwd through attn_fwd_ws, with a workspace (allocated here on q's
    device when not given): for bf16 inputs the value tiles are converted to
    fp16 once into it, instead of inside every CTA, and grids that fill the
    GPU unevenly cut some units' keys into ranges whose partials it holds."""
    import torch
    _check(q, k, v)
    B, Hq, Nq, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), device=q.device, dtype=torch.float32)
    lib = load()
    ws_bytes = lib.attn_fwd_workspace_size(B, Hq, Hkv, Nq, Nk, D, _dtype_code(q))
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, device=q.device, dtype=torch.uint8)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib.attn_fwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                         ws_ptr, ws_len, B, Hq, Hkv, Nq, Nk, D, float(scale), causal_code(causal),
                         _dtype_code(q), _stream_handle(q.device))
    if rc != ATTN_OK:
        raise AttnError("attn_fwd_ws", rc)
    return out, lse


def num_splits(B, Hq, Hkv, Nq, Nk, D, num_sms: int = 0) -> int:
    """The library's key-range count for attn_fwd_splitkv (num_sms 0: ask the
    current device)."""
    return load().attn_fwd_num_splits(B, Hq, Hkv, Nq, Nk, D, int(num_sms))


def splitkv_workspace_size(B, Hq, Hkv, Nq, Nk, D, splits: int) -> int:
    return load().attn_fwd_splitkv_workspace_size(B, Hq, Hkv, Nq, Nk, D, int(splits))


def attn_fwd_splitkv(q, k, v, causal=False, scale: float | None = None, splits: int | None = None,
                     out=None, lse=None, workspace=None):
    """attn_fwd with the keys cut into ``splits`` ranges (None: the library's
    choice for this device) and the partial results merged; for short query
    blocks against long keys, e.g. decoding against a KV cache (use
    causal="bottom_right" when the queries are the newest positions)."""
    import torch
    _check(q, k, v)
    B, Hq, Nq, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    lib = load()
    if splits is None:
        splits = lib.attn_fwd_num_splits(B, Hq, Hkv, Nq, Nk, D, 0)
    ws_bytes = lib.attn_fwd_splitkv_workspace_size(B, Hq, Hkv, Nq, Nk, D, int(splits))
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, device=q.device, dtype=torch.uint8)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, Nq), device=q.device, dtype=torch.float32)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_len = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib.attn_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                              lse.data_ptr(), ws_ptr, ws_len, B, Hq, Hkv, Nq, Nk, D, float(scale),
                              causal_code(causal), _dtype_code(q), int(splits),
                              _stream_handle(q.device))
    if rc != ATTN_OK:
        raise AttnError("attn_fwd_splitkv", rc)
    return out, lse


_BOUND = ("kv8_append_step", "kv8_attn_step", "kv8_attn_workspace_size", "kv8_copy_pages",
          "kvp_reserve_step", "kvp_reassign", "kvp_compact", "kvp_workspace_size", "attn_fwd_window",
          "attn_fwd_window_workspace_size", "attn_bwd_window", "attn_bwd_window_workspace_size",
          "rope_apply", "kv8_append_rope", "kv8_attn_shared", "kv8_attn_shared_workspace_size",
          "kvp_find_shared", "kvp_plan_words")
_bind = None


def _load_bind():
    """The compiled part of this binding (csrc/bind.cpp): the checks, outputs and
    workspaces of the calls below, which decoding steps make many of."""
    global _bind
    lib = load()
    with _lock:
        if _bind is None:
            import importlib.util
            path = os.path.join(PKG, "_build", "_bind.so")
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: run __graft_entry__.build() first")
            import torch  # noqa: F401  (its libraries, before the module that needs them)
            spec = importlib.util.spec_from_file_location("_bind", path)
            mod = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(mod)
            mod.init(*(ctypes.cast(getattr(lib, n), _vp).value for n in _BOUND))
            _bind = mod
    return _bind


def _need(name, t, shape, dtype, dev):
    """Raises unless t is a contiguous tensor of that shape and dtype on CUDA device dev."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"CUDA device {dev}, not {t.dtype} {tuple(t.shape)} on {t.device}")


def _need_workspace(t, dev):
    if t is not None and (t.get_device() != dev or not t.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on CUDA device {dev}")


def _refused(fn: str, rc: int, explain):
    """Raises for a call that did not run: a status of the library, or arguments that
    do not fit together, which `explain` raises for."""
    if rc > 0:
        raise AttnError(fn, rc)
    explain()
    raise ValueError(f"{fn}: arguments do not fit together")


def _explain_window(q, k, v):
    """Device of a sliding-window call's q, k, v; raises when they do not fit."""
    _check(q, k, v)
    _dtype_code(q)
    dev = q.get_device()
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError(f"tensors on {q.device}, {k.device} and {v.device}: one device is needed")
    return dev


def attn_fwd_window(q, k, v, window: int, sinks: int = 0, scale: float | None = None, out=None,
                    lse=None, workspace=None):
    """Sliding-window attention with sinks: query i stands at position
    p = i + Nk - Nq and sees keys j <= p with j > p - window or j < sinks.
    Returns (out, lse) as attn_fwd does; workspace (allocated here when not
    given) as in include/attn.h."""
    r = (_bind or _load_bind()).attn_fwd_window(q, k, v, window, sinks, scale, out, lse, workspace)
    if type(r) is tuple:
        return r

    def explain():
        import torch
        dev = _explain_window(q, k, v)
        if out is not None:
            _need("out", out, q.shape, q.dtype, dev)
        if lse is not None:
            _need("lse", lse, q.shape[:3], torch.float32, dev)
        _need_workspace(workspace, dev)
    _refused("attn_fwd_window", r, explain)


def attn_bwd_window(q, k, v, out, dout, lse, window: int, sinks: int = 0,
                    scale: float | None = None, dq=None, dk=None, dv=None, workspace=None):
    """dq, dk, dv of attn_fwd_window (dk, dv summed over each GQA group)."""
    r = (_bind or _load_bind()).attn_bwd_window(q, k, v, out, dout, lse, window, sinks, scale, dq, dk,
                                                dv, workspace)
    if type(r) is tuple:
        return r

    def explain():
        import torch
        dev = _explain_window(q, k, v)
        _need("out", out, q.shape, q.dtype, dev)
        _need("dout", dout, q.shape, q.dtype, dev)
        _need("lse", lse, q.shape[:3], torch.float32, dev)
        for name, g, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
            if g is not None:
                _need(name, g, like.shape, like.dtype, dev)
        _need_workspace(workspace, dev)
    _refused("attn_bwd_window", r, explain)


def window_attention(q, k, v, window: int, sinks: int = 0, scale: float | None = None):
    """attn_fwd_window as a differentiable function: its output alone."""
    r = (_bind or _load_bind()).window_attention(q, k, v, window, sinks, scale)
    if type(r) is not int:
        return r
    _refused("attn_fwd_window", r, lambda: _explain_window(q, k, v))


def attn_bwd(q, k, v, out, dout, lse, causal: bool = False, scale: float | None = None,
             dq=None, dk=None, dv=None, workspace=None, mask=None):
    """dq, dk, dv of attn_fwd (dk, dv summed over each GQA group); with the
    forward's mask, of attn_fwd(mask=...)."""
    import torch
    _check(q, k, v)
    B, Hq, Nq, D = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    dt = _dtype_code(q)
    lib = load()
    ws_bytes = lib.attn_bwd_workspace_size(B, Hq, Hkv, Nq, Nk, D, dt)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), device=q.device, dtype=torch.uint8)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if mask is not None:
        m, kind, (sb, sh, sq) = prepare_mask(mask, q, Nk)
        rc = lib.attn_bwd_masked(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                 dout.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                 dv.data_ptr(), workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), m.data_ptr(), kind,
                                 sb, sh, sq, B, Hq, Hkv, Nq, Nk, D, float(scale),
                                 causal_code(causal), dt, _stream_handle(q.device))
        if rc != ATTN_OK:
            raise AttnError("attn_bwd_masked", rc)
        return dq, dk, dv
    rc = lib.attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), dout.data_ptr(),
                      lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                      workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                      B, Hq, Hkv, Nq, Nk, D, float(scale), causal_code(causal), dt,
                      _stream_handle(q.device))
    if rc != ATTN_OK:
        raise AttnError("attn_bwd", rc)
    return dq, dk, dv


def sync_status(device=None) -> int:
    """Synchronise the current stream and return (and clear) the most urgent kind of
    error the device recorded: ATTN_ERR_TIMEOUT, _PAGE, _POOL, or ATTN_OK."""
    import torch
    dev = device if device is not None else torch.cuda.current_device()
    return load().attn_sync_status(_stream_handle(dev))


def _ptr(t):
    return None if t is None else t.data_ptr()


def ffn_forward(x, w1, b1, w2, b2, act: str = "gelu_tanh", chunk: int = 4096, out=None,
                workspace=None):
    """y = act(x W1^T + b1) W2^T + b2 over x [T, d_model], `chunk` tokens at a
    time (include/ffn.h).  swiglu: W1 = [Wg; Wu] of 2*d_ff rows."""
    import torch
    T, d_model = x.shape
    d_ff = w2.shape[1]
    for name, t in (("x", x), ("w1", w1), ("w2", w2)):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != x.dtype:
            raise ValueError(f"{name} must be a contiguous CUDA tensor of x's dtype")
    lib = load()
    if workspace is None:
        workspace = torch.empty(max(16, lib.ffn_workspace_size(T, d_ff, chunk)),
                                dtype=torch.uint8, device=x.device)
    y = torch.empty((T, d_model), dtype=x.dtype, device=x.device) if out is None else out
    rc = lib.ffn_forward(x.data_ptr(), w1.data_ptr(), _ptr(b1), w2.data_ptr(), _ptr(b2),
                         y.data_ptr(), T, d_model, d_ff, FFN_ACTS[act], int(chunk),
                         workspace.data_ptr(), workspace.numel(), _dtype_code(x),
                         _stream_handle(x.device))
    if rc != ATTN_OK:
        raise AttnError("ffn_forward", rc)
    return y


def ffn_check_chunking(x, w1, b1, w2, b2, act: str = "gelu_tanh", chunk: int = 4096):
    """Runs the FFN chunked and unchunked and compares bit for bit on the
    device; returns (y, ok)."""
    import torch
    T, d_model = x.shape
    d_ff = w2.shape[1]
    lib = load()
    ws = torch.empty(max(16, lib.ffn_workspace_size(T, d_ff, T)), dtype=torch.uint8,
                     device=x.device)
    y = torch.empty((T, d_model), dtype=x.dtype, device=x.device)
    y_ref = torch.empty_like(y)
    rc = lib.ffn_check_chunking(x.data_ptr(), w1.data_ptr(), _ptr(b1), w2.data_ptr(), _ptr(b2),
                                y.data_ptr(), y_ref.data_ptr(), T, d_model, d_ff, FFN_ACTS[act],
                                int(chunk), ws.data_ptr(), ws.numel(), _dtype_code(x),
                                _stream_handle(x.device))
    if rc not in (ATTN_OK, ATTN_ERR_MISMATCH):
        raise AttnError("ffn_check_chunking", rc)
    return y, rc == ATTN_OK


# ------------------------------------------------------------------ rotary positions

def _followed(t):
    """Whether a graph follows a tensor, or a forward-mode derivative does."""
    import torch
    from torch.autograd import forward_ad
    return (torch.is_grad_enabled() and t.requires_grad) or forward_ad.unpack_dual(t).tangent is not None


def _explain_result(name, out, like, **others):
    """Raises when `out` cannot take the rows of `like`, or begins where one of the others does."""
    if out is None:
        return
    if out.shape != like.shape or out.dtype is not like.dtype or out.device != like.device:
        raise ValueError(f"{name} must be a {like.dtype} tensor {tuple(like.shape)} on {like.device}")
    if _followed(out) or _followed(like):
        raise ValueError(f"{name} is written to behind autograd's back: use the differentiable call")
    steps = sorted((s, n) for s, n in zip(out.stride()[:3], out.shape) if n > 1)
    reach, apart = out.shape[3], out.stride(3) == 1 and out.data_ptr() % 16 == 0
    for s, n in steps:
        apart, reach = apart and s % 8 == 0 and s >= reach, reach + (n - 1) * s
    if not apart:
        raise ValueError(f"{name} needs dense, 16-byte aligned rows that do not overlap")
    for other, t in others.items():
        if t is not None and t.data_ptr() == out.data_ptr():
            raise ValueError(f"{name} begins where {other} does")


def _explain_rope(q, k, positions, rope):
    import torch
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or q.shape[3] != rope.head_dim:
        raise ValueError(f"rows {tuple(getattr(q, 'shape', ()))} are not [B, H, N, {rope.head_dim}]")
    for name, t in (("q", q), ("k", k)):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 4:
            raise ValueError(f"{name} must be a CUDA tensor [B, H, N, D]")
        _dtype_code(t)
    if k is not None and (k.dtype is not q.dtype or k.device != q.device or k.shape[0] != q.shape[0]
                          or k.shape[2:] != q.shape[2:]):
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} must share dtype, device, B, N and D")
    if positions is not None:
        B, _, N, _ = q.shape
        if not isinstance(positions, torch.Tensor) or positions.dtype is not torch.int32 \
                or positions.device != q.device or tuple(positions.shape) not in ((N,), (1, N), (B, N)):
            raise ValueError(f"positions must be an int32 tensor [{N}], [1, {N}] or [{B}, {N}] on {q.device}")


def rope(q, k, rope, positions=None, start: int = 0, q_out=None, k_out=None, transposed: bool = False):
    """q [B, Hq, N, D] and k [B, Hk, N, D] (k None: q alone) turned to positions (int32
    [N], [1, N] or [B, N]; None: start + n) by a rope.Rope (include/rope.h): the pair, or q
    alone.  q_out and k_out may be q and k, and overlap nothing else.  transposed turns back, times the amplitude.
    Not differentiable: see rotary."""
    r = (_bind or _load_bind()).rope(q, k, positions, start, rope.for_rows(q), q_out, k_out, int(transposed))
    if type(r) is not int:
        return r

    def explain():
        _explain_rope(q, k, positions, rope)
        if k is None and k_out is not None:
            raise ValueError("k_out without k")
        _explain_result("q_out", q_out, q, k=k, k_out=k_out)
        _explain_result("k_out", k_out, k, q=q)
    _refused("rope_apply", r, explain)


def rotary(q, k, rope, positions=None, start: int = 0):
    """rope as a differentiable function of q and k."""
    r = (_bind or _load_bind()).rotary(q, k, positions, start, rope.for_rows(q))
    if type(r) is not int:
        return r
    _refused("rope_apply", r, lambda: _explain_rope(q, k, positions, rope))


# ------------------------------------------------------------------ paged 8-bit KV cache

def _explain_pools(k_pages, v_pages, k_scale, v_scale, layers=False):
    """Device and shape of a cache's pools; raises when they do not fit together."""
    import torch
    shape, dt, dev = k_pages.shape, k_pages.dtype, k_pages.get_device()
    if not (len(shape) in ((4, 5) if layers else (4,)) and k_pages.is_contiguous() and dev >= 0
            and dt in (torch.float8_e4m3fn, torch.uint8, torch.int8)):
        raise ValueError("k_pages must be a contiguous CUDA tensor of 8-bit values [n_pages, Hkv, page, "
                         f"D], not {dt} {tuple(shape)} on {k_pages.device}")
    _need("v_pages", v_pages, shape, dt, dev)
    _need("k_scale", k_scale, shape[:-2], torch.float32, dev)
    _need("v_scale", v_scale, shape[:-2], torch.float32, dev)
    return dev, shape


def _explain_table(table, lens, B, dev):
    import torch
    if table.dim() != 2:
        raise ValueError("table must be [B, max_pages]")
    _need("table", table, (B, table.shape[1]), torch.int32, dev)
    _need("lens", lens, (B,), torch.int32, dev)


def _need_word(name, t, dev):
    import torch
    if t is not None:
        _need(name, t, (1,), torch.int32, dev)


def kv8_append(k, v, k_pages, v_pages, k_scale, v_scale, table, lens, n_new=None, granted=None, rope=None,
               q=None, q_out=None):
    """Quantises new keys and values [B, Hkv, T, D] (any strides that are multiples
    of 8 with dense rows) into the paged cache (include/kvcache.h).  lens [B] are
    the lengths after the call; n_new [B] how many of the T tokens each sequence
    takes (None: all T).  granted [1] (written by kvp_reserve): nothing is appended
    where it is 0, since lens does not hold the tokens then.

    With rope (a rope.Rope) the keys are turned to the positions they take
    (include/rope.h), and with q [B, Hq, T, D] the step's queries as well: they are
    returned, in q_out if given (it may be q).  Nothing here is differentiable: a q that
    autograd follows is refused."""
    bind = _bind or _load_bind()
    if rope is None:
        if q is not None or q_out is not None:
            raise ValueError("queries are only turned with rope")
        rc = bind.kv8_append(k, v, k_pages, v_pages, k_scale, v_scale, table, lens, n_new, granted)
        if rc == ATTN_OK:
            return None
    else:
        rc = bind.kv8_append_rope(k, v, k_pages, v_pages, k_scale, v_scale, table, lens, n_new, granted,
                                  rope.for_rows(k), q, q_out)
        if type(rc) is not int:
            return rc

    def explain():
        import torch
        if rope is not None and rope.head_dim != k.shape[-1]:
            raise ValueError(f"the rotation is for head dim {rope.head_dim}, not {k.shape[-1]}")
        dev, (_, Hkv, _, D) = _explain_pools(k_pages, v_pages, k_scale, v_scale)
        _dtype_code(k)
        if not (k.dim() == 4 and v.shape == k.shape and v.dtype is k.dtype and k.shape[1] == Hkv
                and k.shape[3] == D and k.get_device() == dev and v.get_device() == dev):
            raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} must be [B, {Hkv}, T, {D}] on "
                             f"CUDA device {dev}")
        strides = [tuple(0 if n == 1 else s for n, s in zip(t.shape, t.stride())) for t in (k, v)]
        if strides[0] != strides[1] or k.stride(3) != 1 or v.stride(3) != 1:
            raise ValueError("k and v must have the same strides and dense rows")
        _explain_table(table, lens, k.shape[0], dev)
        if n_new is not None:
            _need("n_new", n_new, (k.shape[0],), torch.int32, dev)
        _need_word("granted", granted, dev)
        if q is None:
            if q_out is not None:
                raise ValueError("q_out without q")
        else:
            if not (q.dim() == 4 and q.dtype is k.dtype and q.shape[0] == k.shape[0]
                    and q.shape[2:] == k.shape[2:] and q.get_device() == dev):
                raise ValueError(f"q {tuple(q.shape)} must be a {k.dtype} tensor [{k.shape[0]}, Hq, "
                                 f"{k.shape[2]}, {D}] on CUDA device {dev}")
            if q_out is None and _followed(q):
                raise ValueError("q is turned behind autograd's back: call append under torch.no_grad(), or turn q by "
                                 "the rotation itself")
            _explain_result("q_out", q_out, q, k=k, v=v)
    _refused("kv8_append" if rope is None else "kv8_append_rope", rc, explain)


def _explain_cache_attn(q, k_pages, v_pages, k_scale, v_scale, table, lens, out, lse, workspace, n_new,
                        granted):
    """Device of a cache attention's arguments; raises when they do not fit together."""
    import torch
    dev, (_, _, _, D) = _explain_pools(k_pages, v_pages, k_scale, v_scale)
    _dtype_code(q)
    if q.dim() != 4 or q.shape[3] != D or not q.is_contiguous() or q.get_device() != dev:
        raise ValueError(f"q must be a contiguous tensor [B, Hq, Nq, {D}] on CUDA device {dev}")
    _explain_table(table, lens, q.shape[0], dev)
    if n_new is not None:
        _need("n_new", n_new, (q.shape[0],), torch.int32, dev)
    _need_word("granted", granted, dev)
    if out is not None:
        _need("out", out, q.shape, q.dtype, dev)
    if lse is not None:
        _need("lse", lse, q.shape[:3], torch.float32, dev)
    _need_workspace(workspace, dev)
    return dev


def kv8_attn(q, k_pages, v_pages, k_scale, v_scale, table, lens, scale: float | None = None,
             window: int = 0, sinks: int = 0, out=None, lse=None, workspace=None, n_new=None,
             granted=None):
    """Attention of the newest Nq positions of each sequence, q [B, Hq, Nq, D], over
    the paged cache (include/kvcache.h); returns (out, lse).  n_new [B]: only the
    first n_new of a sequence's queries are its newest positions, the others get 0
    and -inf, and so do all of them where granted [1] (written by kvp_reserve) is 0."""
    r = (_bind or _load_bind()).kv8_attn(q, k_pages, v_pages, k_scale, v_scale, table, lens, scale,
                                         window, sinks, out, lse, workspace, n_new, granted)
    if type(r) is tuple:
        return r

    def explain():
        _explain_cache_attn(q, k_pages, v_pages, k_scale, v_scale, table, lens, out, lse, workspace, n_new,
                            granted)
    _refused("kv8_attn", r, explain)


def kv8_attn_shared(q, k_pages, v_pages, k_scale, v_scale, table, lens, plan, scale: float | None = None,
                    out=None, lse=None, workspace=None, n_new=None, granted=None):
    """kv8_attn, without a window, for sequences that begin with the same pages: plan
    (kvp_find_shared's for this table) says which, and their common prefix is read once
    for all of them (include/kvcache.h).  n_new and granted as in kv8_attn."""
    r = (_bind or _load_bind()).kv8_attn_shared(q, k_pages, v_pages, k_scale, v_scale, table, lens, scale,
                                                plan, out, lse, workspace, n_new, granted)
    if type(r) is tuple:
        return r

    def explain():
        import torch
        dev = _explain_cache_attn(q, k_pages, v_pages, k_scale, v_scale, table, lens, out, lse, workspace,
                                  n_new, granted)
        words = load().kvp_plan_words(q.shape[0])
        if not isinstance(plan, torch.Tensor):
            raise ValueError("plan must be what kvp_find_shared returned")
        _need("plan", plan, (words,), torch.int32, dev)
    _refused("kv8_attn_shared", r, explain)


def kvp_find_shared(table, lens, page: int, min_saved: int = -1, plan=None):
    """Which sequences begin with the same pages: the plan of kv8_attn_shared (int32, written
    to plan if given).  Made after a fork and kept until the next one.  min_saved: positions that
    a group has to save (-1: as far as the attention finds it worth while;
    include/kvcache.h)."""
    r = (_bind or _load_bind()).kvp_find_shared(table, lens, page, min_saved, plan)
    if type(r) is not int:
        return r

    def explain():
        import torch
        if not table.is_cuda or table.dim() != 2:
            raise ValueError("table must be a CUDA tensor [B, max_pages]")
        dev = table.get_device()
        _need("table", table, table.shape, torch.int32, dev)
        _need("lens", lens, table.shape[:1], torch.int32, dev)
        if plan is not None:
            _need("plan", plan, (load().kvp_plan_words(table.shape[0]),), torch.int32, dev)
    _refused("kvp_find_shared", r, explain)


def kv8_copy_pages(k_pages, v_pages, k_scale, v_scale, src, dst, count, max_count: int | None = None):
    """Copies pages src[i] to dst[i] for i < min(count[0], max_count) in every layer
    of the pools ([n_layers, n_pages, Hkv, page, D], or without layers)."""
    rc = (_bind or _load_bind()).kv8_copy_pages(k_pages, v_pages, k_scale, v_scale, src, dst, count,
                                                max_count)
    if rc == ATTN_OK:
        return

    def explain():
        import torch
        dev, _ = _explain_pools(k_pages, v_pages, k_scale, v_scale, layers=True)
        _need("src", src, src.shape, torch.int32, dev)
        _need("dst", dst, dst.shape, torch.int32, dev)
        if count.dtype is not torch.int32 or count.numel() < 1 or count.get_device() != dev:
            raise ValueError(f"count must be an int32 tensor on CUDA device {dev}")
        room = min(src.numel(), dst.numel())
        if max_count is not None and max_count > room:
            raise ValueError(f"max_count {max_count} is past the {room} listed pairs")
    _refused("kv8_copy_pages", rc, explain)


def kvp_workspace_size(n_seqs: int, max_pages: int, n_pages: int) -> int:
    """Bytes of workspace the page bookkeeping calls need."""
    return load().kvp_workspace_size(n_seqs, max_pages, n_pages)


def _explain_book(table, refs, info, workspace, lists=(), **per_seq):
    """Raises when a bookkeeping call's tensors do not fit together: per_seq are int32
    [n_seqs], lists (name, tensor, least entries)."""
    import torch
    dev = table.get_device()
    if table.dim() != 2 or refs.dim() != 1 or dev < 0:
        raise ValueError("table must be a CUDA tensor [n_seqs, max_pages], refs [n_pages]")
    _need("table", table, table.shape, torch.int32, dev)
    _need("refs", refs, refs.shape, torch.int32, dev)
    _need("info", info, (4,), torch.int32, dev)
    for name, t in per_seq.items():
        _need(name, t, table.shape[:1], torch.int32, dev)
    for name, t, least in lists:
        _need(name, t, t.shape, torch.int32, dev)
        if t.numel() < least:
            raise ValueError(f"{name} needs {least} entries")
    _need_workspace(workspace, dev)


def kvp_reserve(table, lens, refs, n_new, page: int, info, window: int = 0, sinks: int = 0,
                workspace=None, granted=None):
    """Adds n_new [n_seqs] tokens to the sequences' lengths and pages for them to
    their tables; with a window first gives back the pages it has left behind
    (include/kvcache.h).  info [4] int32 receives (done, taken, given back, free),
    granted [1] int32, if given, done alone."""
    rc = (_bind or _load_bind()).kvp_reserve(table, lens, refs, n_new, page, info, window, sinks, workspace,
                                             granted)
    if rc != ATTN_OK:
        def explain():
            _explain_book(table, refs, info, workspace, lens=lens, n_new=n_new)
            _need_word("granted", granted, table.get_device())
        _refused("kvp_reserve", rc, explain)


def kvp_reassign(table, lens, refs, parents, page: int, copy_src, copy_dst, info, workspace=None):
    """Sequence c becomes what parents[c] was (c: kept, -1: freed); the pairs of
    pages to copy go to copy_src / copy_dst, info [4] int32 receives (done, pairs,
    given back, free) (include/kvcache.h)."""
    rc = (_bind or _load_bind()).kvp_reassign(table, lens, refs, parents, page, copy_src, copy_dst, info,
                                              workspace)
    if rc != ATTN_OK:
        n = table.shape[0]
        _refused("kvp_reassign", rc, lambda: _explain_book(
            table, refs, info, workspace, (("copy_src", copy_src, n), ("copy_dst", copy_dst, n)), lens=lens,
            parents=parents))


def kvp_compact(table, refs, move_src, move_dst, info, table_out=None, refs_out=None,
                workspace=None):
    """Renumbers the held pages to the front of the pool (in place without table_out
    and refs_out); the moves go to move_src / move_dst, info [4] int32 receives (1,
    moves, held, free) (include/kvcache.h)."""
    table_out = table if table_out is None else table_out
    refs_out = refs if refs_out is None else refs_out
    rc = (_bind or _load_bind()).kvp_compact(table, refs, move_src, move_dst, info, table_out, refs_out,
                                             workspace)
    if rc != ATTN_OK:
        def explain():
            import torch
            n = refs.numel() // 2
            _explain_book(table, refs, info, workspace, (("move_src", move_src, n), ("move_dst", move_dst, n)))
            _need("table_out", table_out, table.shape, torch.int32, table.get_device())
            _need("refs_out", refs_out, refs.shape, torch.int32, table.get_device())
        _refused("kvp_compact", rc, explain)
