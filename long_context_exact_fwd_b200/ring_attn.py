"""ctypes binding of libringattn.so (include/ring_attn.h): argument marshalling only.

Every step of the operations runs in the library's CUDA kernels; this
module only checks tensor properties, allocates outputs with torch (device memory
plumbing) and passes raw pointers plus the current CUDA stream.  There is no fallback:
importing this module fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import List, NamedTuple, Optional, Tuple

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libringattn.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{_LIB_PATH} is missing: build it with `python -m long_context_exact_fwd_b200.build` "
        "(there is no CPU fallback)")
_lib = ctypes.CDLL(_LIB_PATH)

(RA_OK, RA_ERR_ARG, RA_ERR_SHAPE, RA_ERR_ALIGN, RA_ERR_WORKSPACE, RA_ERR_CUDA, RA_ERR_TIMEOUT, RA_ERR_DEVICE,
 RA_ERR_PAGES) = range(9)
RA_BF16, RA_F32 = 0, 1

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ip = ctypes.POINTER(ctypes.c_int)


def _sig(name, restype, *argtypes):
    fn = getattr(_lib, name)
    fn.restype = restype
    fn.argtypes = list(argtypes)
    return fn


_fwd = _sig("ring_attn_fwd", _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp)
_fwd_ex = _sig("ring_attn_fwd_ex", _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _vp)
_bwd_ws = _sig("ring_attn_bwd_workspace_size", _sz, _i, _i, _i, _i)
_split_ws = _sig("ring_attn_fwd_split_workspace_size", _sz, _i, _i, _i, _i, _i)
_fwd_split = _sig("ring_attn_fwd_split", _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _sz, _vp)
_fwd_partial = _sig("ring_attn_fwd_partial", _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp)
_bwd = _sig("ring_attn_bwd", _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _sz, _vp)
_bwd_ex = _sig("ring_attn_bwd_ex", _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp,
               _sz, _vp)
_merge_ex = _sig("ring_attn_merge_ex", _i, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _vp)
_ring_order = _sig("ring_attn_ring_order", _i, _i, _i, _i, _ip, _i)
_visit_tiles = _sig("ring_attn_visit_tiles", _i, _i, _i, _i, _i, _i, _ip, _i)
_device_status = _sig("ring_attn_device_status", _i, _vp)
_kernel_status = _sig("ring_attn_kernel_status", _i, _vp)
_strerror = _sig("ring_attn_strerror", ctypes.c_char_p, _i)
_version = _sig("ring_attn_version", _i)
_last_cuda = _sig("ring_attn_last_cuda_error", _i, ctypes.POINTER(ctypes.c_char_p))
_bwd_visit_tiles = _sig("ring_attn_bwd_visit_tiles", _i, _i, _i, _i, _i, _i, _ip, _i)
_launch_count = _sig("ring_attn_launch_count", ctypes.c_ulonglong)
_bwd_acc = _sig("ring_attn_bwd_accumulate", _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                _i, _vp, _sz, _vp)
_bwd_noalloc = _sig("ring_attn_bwd_noalloc", _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp)
_noalloc_max = _sig("ring_attn_bwd_noalloc_max_bytes", _sz)
_ffn_ws = _sig("ring_attn_ffn_workspace_size", _sz, _i, _i, _i, _i)
_ffn_fwd = _sig("ring_attn_ffn_fwd", _i, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _i, _vp, _vp, _sz, _vp)
_ffn_block = _sig("ring_attn_ffn_block", _i, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _i, _vp, _vp, _sz, _vp)
_ll = ctypes.c_longlong


class _CacheStruct(ctypes.Structure):   # ra_cache
    _fields_ = ([(n, _vp) for n in ("k", "v", "k_scale", "v_scale", "table", "lens", "refs")]
                + [(n, _i) for n in ("layers", "pages", "heads", "page", "head_dim", "slots", "max_pages")])


_llp, _cp = ctypes.POINTER(_ll), ctypes.POINTER(_CacheStruct)
_rope = _sig("ring_attn_rope", _i, _vp, _vp, _i, _llp, _vp, _vp, _i, _llp, _i, _i, _i, _vp, _i, _i, _f, _vp, _ll, _ll,
             _ll, _i, _i, _vp)
_cache_pages_ws = _sig("ring_attn_cache_pages_workspace_size", _sz, _i, _i)
_cache_reserve = _sig("ring_attn_cache_reserve", _i, _cp, _vp, _vp, _i, _vp, _sz, _vp)
_cache_reserve_ex = _sig("ring_attn_cache_reserve_ex", _i, _cp, _vp, _vp, _i, _vp, _vp, _sz, _vp)
_cache_append = _sig("ring_attn_cache_append", _i, _cp, _i, _vp, _vp, _i, _i, _vp, _llp, _vp, _llp, _vp)
_cache_read = _sig("ring_attn_cache_read", _i, _cp, _i, _vp, _vp, _i, _i, _vp, _vp, _vp)
_cache_read_ex = _sig("ring_attn_cache_read_ex", _i, _cp, _i, _vp, _vp, _i, _i, _vp, _vp, _i, _i, _vp)
_cache_attend_ws = _sig("ring_attn_cache_attend_workspace_size", _sz, _i, _i, _i, _i)
_cache_attend = _sig("ring_attn_cache_attend", _i, _cp, _i, _vp, _vp, _i, _i, _i, _vp, _llp, _f, _i, _vp, _i, _vp, _vp,
                     _sz, _vp)
_cache_attend_ex = _sig("ring_attn_cache_attend_ex", _i, _cp, _i, _vp, _vp, _i, _i, _i, _vp, _llp, _f, _i, _vp, _i, _vp, _i,
                        _i, _vp, _sz, _vp)
_cache_fork = _sig("ring_attn_cache_fork", _i, _cp, _vp, _vp, _i, _vp, _sz, _vp)
_cache_trim = _sig("ring_attn_cache_trim", _i, _cp, _vp, _vp, _i, _vp)
_cache_compact = _sig("ring_attn_cache_compact", _i, _cp, _vp, _sz, _vp)
_exp2_check = _sig("ring_attn_exp2_check", _i, _vp, _vp, _vp, ctypes.c_longlong, _vp)
_wait_selftest = _sig("ring_attn_wait_selftest", _i, ctypes.c_longlong, _vp)


class RingAttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        msg = f"{where}: status {code} ({strerror(code)})"
        if code == RA_ERR_CUDA:
            err, site = last_cuda_error()
            msg += f"; last CUDA failure {err} in {site}"
        super().__init__(msg)


def last_cuda_error() -> Tuple[int, str]:
    site = ctypes.c_char_p()
    code = _last_cuda(ctypes.byref(site))
    return int(code), (site.value or b"").decode()


def strerror(code: int) -> str:
    return _strerror(code).decode()


def version() -> int:
    return _version()


def lib_path() -> str:
    return _LIB_PATH


def _check(code: int, where: str) -> None:
    if code != RA_OK:
        raise RingAttnError(code, where)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: torch.Tensor, name: str, dtype=None, shape=None) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    # the library launches on the current device (and uses its static scratch there)
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device} but the current device is cuda:{torch.cuda.current_device()}; "
                         "make the tensors' device current (torch.cuda.device) before the call")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, D: int, causal: bool = True,
        scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
        lse: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Ring-attention forward.  q, k, v: [B, H, S, Dh] bf16 (or float32) CUDA tensors.
    Returns (o [B, H, S, Dh] in the input dtype, lse [B, H, S] float32)."""
    if q.dim() != 4:
        raise ValueError("q must be [B, H, S, Dh]")
    B, H, S, Dh = q.shape
    dt = q.dtype
    if dt not in (torch.bfloat16, torch.float32):
        raise ValueError("inputs must be bfloat16 or float32")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, dt, q.shape)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device)
    _need(out, "out", dt, q.shape)
    _need(lse, "lse", torch.float32, (B, H, S))
    code = _fwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, S, Dh, D,
                   1 if causal else 0, RA_BF16 if dt == torch.bfloat16 else RA_F32,
                   float(scale) if scale else 0.0, _stream(stream))
    _check(code, "ring_attn_fwd")
    return out, lse


def fwd_split_workspace_bytes(B: int, H: int, S: int, Dh: int, n_parts: int) -> int:
    return int(_split_ws(B, H, S, Dh, n_parts))


def split_parts_hint(B: int, H: int, S: int, device=None) -> int:
    """Pieces per query pair worth using: 2 while the forward has fewer than two 256-row work
    items per SM (measured on B200: H=1 S=64K +50 %, H=2 S=32K +31 %; from four items per SM
    on, splitting only adds the merge), else 1."""
    sms = torch.cuda.get_device_properties(device if device is not None else torch.cuda.current_device()) \
        .multi_processor_count
    items = B * H * ((S + 255) // 256)
    return 2 if items < 2 * sms else 1


def fwd_split(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, D: int, causal: bool = True,
              n_parts: Optional[int] = None, workspace: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
              stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Forward with each query pair's ring cut into n_parts pieces merged through their
    log-sum-exp (ring_attn_fwd_split); n_parts None picks split_parts_hint.  q, k, v:
    [B, H, S, Dh] bf16.  Returns (o, lse); after the call `workspace` (if given) holds the
    partials."""
    if q.dim() != 4:
        raise ValueError("q must be [B, H, S, Dh]")
    B, H, S, Dh = q.shape
    if n_parts is None:
        n_parts = split_parts_hint(B, H, S, q.device)
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, torch.bfloat16, q.shape)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device) if lse is None else lse
    _need(out, "out", torch.bfloat16, q.shape)
    _need(lse, "lse", torch.float32, (B, H, S))
    need = fwd_split_workspace_bytes(B, H, S, Dh, n_parts)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _need(workspace, "workspace")
    code = _fwd_split(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, S, Dh, D,
                      1 if causal else 0, n_parts, workspace.data_ptr(),
                      workspace.numel() * workspace.element_size(), _stream(stream))
    _check(code, "ring_attn_fwd_split")
    return out, lse


def fwd_partial(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, D: int, causal: bool = True,
                out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Forward with a float32 output (ring_attn_fwd_partial): (o [B, H, S, Dh] f32, lse
    [B, H, S] f32), one part for merge().  q, k, v: [B, H, S, Dh] bf16."""
    if q.dim() != 4:
        raise ValueError("q must be [B, H, S, Dh]")
    B, H, S, Dh = q.shape
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(t, name, torch.bfloat16, q.shape)
    out = torch.empty(q.shape, dtype=torch.float32, device=q.device) if out is None else out
    lse = torch.empty((B, H, S), dtype=torch.float32, device=q.device) if lse is None else lse
    _need(out, "out", torch.float32, q.shape)
    _need(lse, "lse", torch.float32, (B, H, S))
    code = _fwd_partial(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), B, H, S, Dh, D,
                        1 if causal else 0, _stream(stream))
    _check(code, "ring_attn_fwd_partial")
    return out, lse


def bwd_workspace_bytes(B: int, H: int, S: int, Dh: int) -> int:
    return int(_bwd_ws(B, H, S, Dh))


def bwd(q, k, v, o, lse, do, D: int, causal: bool = True, dq=None, dk=None, dv=None,
        workspace: Optional[torch.Tensor] = None, stream=None, scale: Optional[float] = None):
    """Ring-attention backward (bf16, Dh 64 or 128; ring_attn_bwd_ex).  `scale` must be the
    forward's (None: 1/sqrt(Dh)).  Returns (dq, dk, dv), each [B, H, S, Dh] bf16."""
    B, H, S, Dh = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do)):
        _need(t, name, torch.bfloat16, q.shape)
    _need(lse, "lse", torch.float32, (B, H, S))
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _need(t, name, torch.bfloat16, q.shape)
    need = bwd_workspace_bytes(B, H, S, Dh)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _need(workspace, "workspace")
    code = _bwd_ex(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), do.data_ptr(),
                   dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, S, Dh, D, 1 if causal else 0,
                   float(scale) if scale else 0.0, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                   _stream(stream))
    _check(code, "ring_attn_bwd_ex")
    return dq, dk, dv


def bwd_accumulate(q, k, v, o, lse, do, D: int, causal: bool, dq32: torch.Tensor, dk32: torch.Tensor,
                   dv32: torch.Tensor, workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward whose gradients are added to float32 accumulators (ring_attn_bwd_accumulate):
    dq32 += dQ, dk32 += dK, dv32 += dV, each [B, H, S, Dh] float32 cleared by the caller
    before the first call."""
    B, H, S, Dh = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do)):
        _need(t, name, torch.bfloat16, q.shape)
    _need(lse, "lse", torch.float32, (B, H, S))
    for name, t in (("dq32", dq32), ("dk32", dk32), ("dv32", dv32)):
        _need(t, name, torch.float32, q.shape)
    need = bwd_workspace_bytes(B, H, S, Dh)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _need(workspace, "workspace")
    code = _bwd_acc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), do.data_ptr(),
                    dq32.data_ptr(), dk32.data_ptr(), dv32.data_ptr(), B, H, S, Dh, D, 1 if causal else 0,
                    workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(code, "ring_attn_bwd_accumulate")
    return dq32, dk32, dv32


def bwd_noalloc(q, k, v, o, lse, do, D: int, causal: bool = True, dq=None, dk=None, dv=None, stream=None):
    """Backward through ring_attn_bwd_noalloc: no workspace argument; the library's static
    device scratch (bwd_noalloc_max_bytes()) holds the dQ accumulator.  Calls that overlap
    on the GPU race on that scratch."""
    B, H, S, Dh = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do)):
        _need(t, name, torch.bfloat16, q.shape)
    _need(lse, "lse", torch.float32, (B, H, S))
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _need(t, name, torch.bfloat16, q.shape)
    code = _bwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), do.data_ptr(),
                        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, S, Dh, D, 1 if causal else 0,
                        _stream(stream))
    _check(code, "ring_attn_bwd_noalloc")
    return dq, dk, dv


def ffn_workspace_bytes(B: int, S: int, D: int, f: int) -> int:
    return int(_ffn_ws(B, S, D, f))


def ffn(o: torch.Tensor, w1: torch.Tensor, b1: torch.Tensor, w2: torch.Tensor, b2: torch.Tensor, D: int,
        block: Optional[int] = None, out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
        stream=None) -> torch.Tensor:
    """Blockwise feedforward after attention (ring_attn_ffn_fwd, or ring_attn_ffn_block for one
    ring block): o [B, H, S, Dh] bf16 attention output; w1 [f, H*Dh], w2 [H*Dh, f] bf16; b1 [f],
    b2 [H*Dh] float32.  Returns y [B, S, H*Dh] bf16 = gelu(x w1^T + b1) w2^T + b2 with
    x[b, s] the heads of token s side by side (only block `block`'s rows are written when given)."""
    if o.dim() != 4:
        raise ValueError("o must be [B, H, S, Dh]")
    B, H, S, Dh = o.shape
    h, f = H * Dh, w1.shape[0]
    _need(o, "o", torch.bfloat16)
    _need(w1, "w1", torch.bfloat16, (f, h))
    _need(w2, "w2", torch.bfloat16, (h, f))
    _need(b1, "b1", torch.float32, (f,))
    _need(b2, "b2", torch.float32, (h,))
    out = torch.empty((B, S, h), dtype=torch.bfloat16, device=o.device) if out is None else out
    _need(out, "out", torch.bfloat16, (B, S, h))
    if workspace is None:
        workspace = torch.empty(max(ffn_workspace_bytes(B, S, D, f), 1), dtype=torch.uint8, device=o.device)
    _need(workspace, "workspace")
    wsb = workspace.numel() * workspace.element_size()
    if block is None:
        code = _ffn_fwd(o.data_ptr(), B, H, S, Dh, D, w1.data_ptr(), b1.data_ptr(), w2.data_ptr(), b2.data_ptr(), f,
                        out.data_ptr(), workspace.data_ptr(), wsb, _stream(stream))
        _check(code, "ring_attn_ffn_fwd")
    else:
        code = _ffn_block(o.data_ptr(), B, H, S, Dh, D, int(block), w1.data_ptr(), b1.data_ptr(), w2.data_ptr(),
                          b2.data_ptr(), f, out.data_ptr(), workspace.data_ptr(), wsb, _stream(stream))
        _check(code, "ring_attn_ffn_block")
    return out


# ---------------------------------------------------------------------------- rotary positions
class RopePlan(NamedTuple):
    """What rope() goes by: per pair the turn per position (theta / 2 pi in units of 2^-64 turn, as
    int64 bits, on the device), the pairing and the amplitude.  Made once by rope_plan()."""
    steps: torch.Tensor
    rot: int
    interleaved: bool
    amplitude: float


def rope_inv_freq(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                  original_length: int = 0, fast: float = 32.0, slow: float = 1.0) -> Tuple[torch.Tensor, float]:
    """Inverse frequencies theta_i = base^(-2i / rot), i < rot / 2 (float64, CPU), and the amplitude,
    for contexts `factor` times as long as trained on:
      "none"    as they are;
      "linear"  theta / factor (positions interpolated);
      "base"    base grown to base * factor^(rot / (rot - 2)): the slowest pair is stretched by `factor`, the
                fastest not at all;
      "ramp"    by how often a pair turns over `original_length` positions: from `fast` turns on theta, up to
                `slow` turns theta / factor, linear between; amplitude 0.1 ln(factor) + 1 (the YaRN rule,
                arXiv 2309.00071)."""
    if rot <= 0 or rot % 2:
        raise ValueError(f"rot must be positive and even, got {rot}")
    if not (base > 0 and math.isfinite(base)) or not (factor > 0 and math.isfinite(factor)):
        raise ValueError("base and factor must be positive and finite")
    if scaling == "base":
        if rot < 4:
            raise ValueError('scaling "base" needs rot >= 4')
        base = base * factor ** (rot / (rot - 2))
    theta = torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    if scaling in ("none", "base"):
        return theta, 1.0
    if scaling == "linear":
        return theta / factor, 1.0
    if scaling == "ramp":
        if original_length <= 0 or not fast > slow:
            raise ValueError('scaling "ramp" needs original_length > 0 and fast > slow')
        turns = original_length * theta / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        return theta / factor * (1 - keep) + theta * keep, 0.1 * math.log(factor) + 1.0
    raise ValueError(f"unknown scaling {scaling!r}")


@functools.lru_cache(maxsize=64)
def _pi(bits: int) -> int:
    """pi * 2^bits to a unit or two, by Machin's formula: pi = 16 atan(1/5) - 4 atan(1/239)."""
    def atan(x):   # of 1 / x, 32 bits to spare
        power = (1 << (bits + 32)) // x
        total, n = power, 1
        while power:
            power //= -x * x
            n += 2
            total += power // n
        return total
    return (16 * atan(5) - 4 * atan(239)) >> 32


def _step(theta: float) -> int:
    """theta / 2 pi in units of 2^-64 turn, whole turns dropped, to the nearest unit.  In integers: a quotient of
    doubles would be off by up to 2^-53 of itself, hundreds of units."""
    bits = 128 + max(0, math.frexp(theta)[1])
    n, d = theta.as_integer_ratio()
    den = d * _pi(bits)
    return ((n << (64 + bits)) + den) // (2 * den) % (1 << 64)


def rope_plan(inv_freq: torch.Tensor, layout: str = "half", amplitude: float = 1.0, device=None) -> RopePlan:
    """The plan for rope(): inv_freq [rot / 2] (radians per position, finite), layout "half" (pairs
    i, i + rot / 2) or "interleaved" (pairs 2i, 2i + 1)."""
    if layout not in ("half", "interleaved"):
        raise ValueError(f'layout must be "half" or "interleaved", got {layout!r}')
    if inv_freq.dim() != 1 or inv_freq.numel() == 0:
        raise ValueError("inv_freq must be [rot / 2]")
    if not math.isfinite(amplitude):
        raise ValueError("amplitude must be finite")
    steps = []
    for w in inv_freq.detach().double().cpu().tolist():
        if not math.isfinite(w):
            raise ValueError("inv_freq must be finite")
        u = _step(w)
        steps.append(u - (1 << 64) if u >= 1 << 63 else u)
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return RopePlan(torch.tensor(steps, dtype=torch.int64).to(device), 2 * len(steps), layout == "interleaved",
                    float(amplitude))


def _need_on(t: torch.Tensor, name: str, dev: int) -> None:
    if t.get_device() != dev:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        raise ValueError(f"{name} is on {t.device} but the current device is cuda:{dev}; "
                         "make the tensors' device current (torch.cuda.device) before the call")


def _need_rows(t: torch.Tensor, name: str, dev: int, dtype, shape=None) -> Tuple[int, ...]:
    """As _need, for [B, heads, T, Dh] tensors that may be views: only the last dimension has to be
    contiguous.  Returns the other three strides."""
    _need_on(t, name, dev)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 4 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must have shape {'[B, heads, T, Dh]' if shape is None else tuple(shape)}, "
                         f"got {tuple(t.shape)}")
    st = t.stride()
    if st[3] != 1 and t.shape[3] > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return st[:3]


def _need_dense(t: torch.Tensor, name: str, dev: int, dtype, shape) -> None:
    _need_on(t, name, dev)
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")


@functools.lru_cache(maxsize=1024)
def _strides(*strides):
    """Strides as the C calls take them (read only, so one array serves every call with the same)."""
    return (_ll * len(strides))(*strides)


def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _on(stream):
    """Context in which tensors are allocated for work on `stream`, so that their memory is handed out
    again only behind that work."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _new(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with _on(stream):
        return like.new_empty(shape, dtype=dtype)


def rope(q: torch.Tensor, plan: RopePlan, k: Optional[torch.Tensor] = None, pos: Optional[torch.Tensor] = None,
         offset: int = 0, inverse: bool = False, out: Optional[torch.Tensor] = None,
         k_out: Optional[torch.Tensor] = None, stream=None):
    """Rotary positions (ring_attn_rope) on q [B, Hq, S, Dh] and, in the same launch, k [B, Hk, S, Dh];
    bf16 or float32, views with a contiguous last dimension (a fused projection's columns) included.
    Position of token s: pos[b, s] (int64, [B, S] or [S]), or offset + s.  `out` / `k_out` may be the
    inputs themselves.  inverse=True turns back: the gradient of the inputs from that of the outputs.
    Returns the rotated q, or (q, k)."""
    dt, dev = q.dtype, torch.cuda.current_device()
    if dt != torch.bfloat16 and dt != torch.float32:
        raise ValueError("inputs must be bfloat16 or float32")
    q_st = _need_rows(q, "q", dev, dt)
    B, Hq, S, Dh = q.shape
    if plan.rot > Dh:
        raise ValueError(f"the plan rotates {plan.rot} columns, heads have {Dh}")
    _need_dense(plan.steps, "plan.steps", dev, torch.int64, (plan.rot // 2,))
    pos_ptr, pos_b, pos_s = None, 0, 0
    if pos is not None:
        _need_on(pos, "pos", dev)
        if pos.dtype != torch.int64:
            raise ValueError(f"pos must be torch.int64, got {pos.dtype}")
        if pos.shape == (B, S):
            pos_b, pos_s = pos.stride()
        elif pos.shape == (S,):
            pos_s = pos.stride(0)
        else:
            raise ValueError(f"pos must have shape {(S,)} or {(B, S)}, got {tuple(pos.shape)}")
        pos_ptr = pos.data_ptr()
    if out is None:
        out = _new(q, (B, Hq, S, Dh), dt, stream)
    o_st = _need_rows(out, "out", dev, dt, q.shape)
    k_ptr, k_out_ptr, Hk, k_strides = None, None, 0, None
    if k is not None:
        Hk = k.shape[1] if k.dim() == 4 else 0
        k_st = _need_rows(k, "k", dev, dt, (B, Hk, S, Dh))
        if k_out is None:
            k_out = _new(q, (B, Hk, S, Dh), dt, stream)
        k_strides = _strides(*k_st, *_need_rows(k_out, "k_out", dev, dt, k.shape))
        k_ptr, k_out_ptr = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    code = _rope(q.data_ptr(), out.data_ptr(), Hq, _strides(*q_st, *o_st), k_ptr, k_out_ptr, Hk, k_strides, B, S, Dh,
                 plan.steps.data_ptr(), plan.rot, plan.interleaved, plan.amplitude, pos_ptr, pos_b, pos_s, int(offset),
                 bool(inverse), RA_BF16 if dt == torch.bfloat16 else RA_F32, _raw_stream(stream, dev))
    _check(code, "ring_attn_rope")
    return out if k is None else (out, k_out)


# ---------------------------------------------------------------------------- 8-bit key/value cache
class KVCache:
    """A paged key/value cache in 8 bits (ra_cache): checks its tensors once and keeps them.
      k, v              uint8 [layers, pages, heads, page, Dh] (bits of torch.float8_e4m3fn)
      k_scale, v_scale  float32 [layers, pages, heads], powers of two: value = code * scale
      table             int32 [slots, max_pages], page numbers, -1: none
      lens, refs        int32 [slots] tokens held, [pages] holders of a page
    kv_cache() makes an empty one."""
    __slots__ = ("k", "v", "k_scale", "v_scale", "table", "lens", "refs", "_c", "_ref")

    def __init__(self, k, v, k_scale, v_scale, table, lens, refs):
        if k.dim() != 5 or table.dim() != 2:
            raise ValueError("k must be [layers, pages, heads, page, Dh] and table [slots, max_pages]")
        L, P, H, page, Dh = k.shape
        N, M = table.shape
        for name, t, dt, shape in (("k", k, torch.uint8, k.shape), ("v", v, torch.uint8, k.shape),
                                   ("k_scale", k_scale, torch.float32, (L, P, H)),
                                   ("v_scale", v_scale, torch.float32, (L, P, H)),
                                   ("table", table, torch.int32, (N, M)), ("lens", lens, torch.int32, (N,)),
                                   ("refs", refs, torch.int32, (P,))):
            _need(t, name, dt, shape)
        if page not in (16, 32, 64, 128) or Dh not in (64, 128):
            raise ValueError(f"pages of 16, 32, 64 or 128 tokens and heads of 64 or 128, got {page} and {Dh}")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.table, self.lens, self.refs = table, lens, refs
        self._c = _CacheStruct(*(t.data_ptr() for t in (k, v, k_scale, v_scale, table, lens, refs)), L, P, H, page, Dh,
                               N, M)
        self._ref = ctypes.byref(self._c)

    def _at(self) -> int:
        """The current device, which has to be the cache's."""
        dev = torch.cuda.current_device()
        _need_on(self.k, "the cache", dev)
        return dev


def kv_cache(layers: int, pages: int, heads: int, page: int, Dh: int, slots: int, max_pages: int,
             device=None) -> KVCache:
    """An empty cache: `pages` pages of `page` tokens shared by `slots` sequences of up to max_pages pages."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    z = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)  # noqa: E731
    codes = [torch.zeros((layers, pages, heads, page, Dh), dtype=torch.uint8, device=device) for _ in range(2)]
    scales = [torch.full((layers, pages, heads), 2.0 ** -117, dtype=torch.float32, device=device) for _ in range(2)]
    return KVCache(*codes, *scales, z(slots, max_pages) - 1, z(slots), z(pages))


def _batch(t: torch.Tensor, name: str, dev: int, B: int) -> int:
    _need_on(t, name, dev)
    if t.dtype != torch.int32 or t.shape != (B,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {B} entries, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


@functools.lru_cache(maxsize=1024)
def cache_pages_workspace_bytes(B: int, pages: int) -> int:
    return int(_cache_pages_ws(B, pages))


@functools.lru_cache(maxsize=1024)
def cache_attend_workspace_bytes(T: int, Hq: int, Hkv: int, Dh: int) -> int:
    return int(_cache_attend_ws(T, Hq, Hkv, Dh))


def _workspace(workspace, need: int, like: torch.Tensor, dev: int, stream):
    if workspace is None:
        workspace = _new(like, (max(need, 1),), torch.uint8, stream)
        return workspace, need
    _need_on(workspace, "workspace", dev)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.numel() * workspace.element_size()


def cache_reserve(cache: KVCache, slots: torch.Tensor, n_new: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                  stream=None, granted: Optional[torch.Tensor] = None) -> None:
    """Room for n_new[b] more tokens of slots[b] (int32, on the device), once for all layers; lens grow
    (ring_attn_cache_reserve_ex).  Too few pages, or a slot out of range: device_status(), and 0 in `granted` (int32
    [B], may be n_new) where there was no room.  A step that goes on without asking, one captured in a graph above
    all, passes `granted` as the n_new of the calls that follow: cache_append() would write over older tokens."""
    dev, B = cache._at(), slots.shape[0]
    s, n = _batch(slots, "slots", dev, B), _batch(n_new, "n_new", dev, B)
    ws, size = _workspace(workspace, cache_pages_workspace_bytes(B, cache._c.pages), cache.k, dev, stream)
    g = None if granted is None else _batch(granted, "granted", dev, B)
    _check(_cache_reserve_ex(cache._ref, s, n, B, g, ws.data_ptr(), size, _raw_stream(stream, dev)),
           "ring_attn_cache_reserve_ex")


def cache_append(cache: KVCache, layer: int, slots: torch.Tensor, n_new: Optional[torch.Tensor], k: torch.Tensor,
                 v: torch.Tensor, stream=None) -> None:
    """Writes the last n_new[b] tokens (None: T) of slots[b] into one layer: k, v [B, heads, T, Dh] bf16,
    views with a contiguous last dimension included (ring_attn_cache_append)."""
    dev = cache._at()
    k_st = _need_rows(k, "k", dev, torch.bfloat16)
    v_st = _need_rows(v, "v", dev, torch.bfloat16, k.shape)
    B, H, T, Dh = k.shape
    if H != cache._c.heads or Dh != cache._c.head_dim:
        raise ValueError(f"k must be [B, {cache._c.heads}, T, {cache._c.head_dim}], got {tuple(k.shape)}")
    s = _batch(slots, "slots", dev, B)
    n = None if n_new is None else _batch(n_new, "n_new", dev, B)
    code = _cache_append(cache._ref, layer, s, n, B, T, k.data_ptr(), _strides(*k_st), v.data_ptr(), _strides(*v_st),
                         _raw_stream(stream, dev))
    _check(code, "ring_attn_cache_append")


def cache_read(cache: KVCache, layer: int, slots: torch.Tensor, length: int, start: Optional[torch.Tensor] = None,
               k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One layer's keys and values, exact in bf16, [B, heads, length, Dh]: positions start[b] (None: 0) ..
    of slots[b], zero where the sequence holds none (ring_attn_cache_read_ex).  Rows of padding (slot -1) and of
    entries that are left out are zero in a fresh output and stay as they were in a given k or v."""
    dev, B = cache._at(), slots.shape[0]
    s = _batch(slots, "slots", dev, B)
    at = None if start is None else _batch(start, "start", dev, B)
    shape = (B, cache._c.heads, length, cache._c.head_dim)
    fill_k, fill_v = k is None, v is None
    if fill_k:
        k = _new(cache.k, shape, torch.bfloat16, stream)
    if fill_v:
        v = _new(cache.k, shape, torch.bfloat16, stream)
    _need_dense(k, "k", dev, torch.bfloat16, shape)
    _need_dense(v, "v", dev, torch.bfloat16, shape)
    _check(_cache_read_ex(cache._ref, layer, s, at, B, length, k.data_ptr(), v.data_ptr(), fill_k, fill_v,
                          _raw_stream(stream, dev)), "ring_attn_cache_read_ex")
    return k, v


def cache_attend(cache: KVCache, layer: int, slots: torch.Tensor, n_new: Optional[torch.Tensor], q: torch.Tensor,
                 scale: Optional[float] = None, causal: bool = True, out_dtype=torch.bfloat16,
                 workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of each sequence's last n_new[b] tokens (None: T) over one layer of the cache
    (ring_attn_cache_attend_ex): q [B, Hq, T, Dh] bf16, views with a contiguous last dimension included, Hq a
    multiple of the cache's heads.  Returns (o [B, Hq, T, Dh] bf16 or float32, lse [B, Hq, T] float32) as
    fwd() does; a float32 o is one part for merge().  Rows t >= n_new[b], of padding (slot -1) and of entries that
    are left out are 0 and -inf in fresh outputs and stay as they were in a given out or lse."""
    dev = cache._at()
    q_st = _need_rows(q, "q", dev, torch.bfloat16)
    B, Hq, T, Dh = q.shape
    heads = cache._c.heads
    if Dh != cache._c.head_dim or Hq % heads:
        raise ValueError(f"q must be [B, a multiple of {heads}, T, {cache._c.head_dim}], got {tuple(q.shape)}")
    if out_dtype != torch.bfloat16 and out_dtype != torch.float32:
        raise ValueError("out_dtype must be bfloat16 or float32")
    s = _batch(slots, "slots", dev, B)
    n = None if n_new is None else _batch(n_new, "n_new", dev, B)
    ws, size = _workspace(workspace, cache_attend_workspace_bytes(T, Hq, heads, Dh), q, dev, stream)
    fill_o, fill_lse = out is None, lse is None
    if fill_o:
        out = _new(q, (B, Hq, T, Dh), out_dtype, stream)
    else:
        _need_dense(out, "out", dev, out_dtype, (B, Hq, T, Dh))
    if fill_lse:
        lse = _new(q, (B, Hq, T), torch.float32, stream)
    else:
        _need_dense(lse, "lse", dev, torch.float32, (B, Hq, T))
    code = _cache_attend_ex(cache._ref, layer, s, n, B, T, Hq, q.data_ptr(), _strides(*q_st), float(scale) if scale else 0.0,
                         bool(causal), out.data_ptr(), RA_BF16 if out_dtype == torch.bfloat16 else RA_F32,
                         lse.data_ptr(), fill_o, fill_lse, ws.data_ptr(), size, _raw_stream(stream, dev))
    _check(code, "ring_attn_cache_attend_ex")
    return out, lse


def cache_fork(cache: KVCache, src: torch.Tensor, dst: torch.Tensor, workspace: Optional[torch.Tensor] = None,
               stream=None) -> None:
    """The empty slots dst[b] share the pages of src[b] from here on (ring_attn_cache_fork); a page that
    both hold is copied when cache_reserve() makes room in it."""
    dev, B = cache._at(), src.shape[0]
    a, d = _batch(src, "src", dev, B), _batch(dst, "dst", dev, B)
    ws, size = _workspace(workspace, cache_pages_workspace_bytes(B, cache._c.pages), cache.k, dev, stream)
    _check(_cache_fork(cache._ref, a, d, B, ws.data_ptr(), size, _raw_stream(stream, dev)), "ring_attn_cache_fork")


def cache_trim(cache: KVCache, slots: torch.Tensor, keep: Optional[torch.Tensor] = None, stream=None) -> None:
    """Keeps the first keep[b] tokens of slots[b] (None: 0, the sequence is freed) and gives up the pages
    behind them (ring_attn_cache_trim)."""
    dev, B = cache._at(), slots.shape[0]
    s = _batch(slots, "slots", dev, B)
    n = None if keep is None else _batch(keep, "keep", dev, B)
    _check(_cache_trim(cache._ref, s, n, B, _raw_stream(stream, dev)), "ring_attn_cache_trim")


def cache_free(cache: KVCache, slots: torch.Tensor, stream=None) -> None:
    """Frees the sequences slots[b]: cache_trim() to nothing."""
    cache_trim(cache, slots, None, stream)


def cache_compact(cache: KVCache, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Moves the pages in use to the lowest page numbers, all layers (ring_attn_cache_compact)."""
    dev = cache._at()
    ws, size = _workspace(workspace, cache_pages_workspace_bytes(0, cache._c.pages), cache.k, dev, stream)
    _check(_cache_compact(cache._ref, ws.data_ptr(), size, _raw_stream(stream, dev)), "ring_attn_cache_compact")


def bwd_noalloc_max_bytes() -> int:
    return int(_noalloc_max())


def merge(o_parts: torch.Tensor, lse_parts: torch.Tensor, out_dtype=torch.bfloat16,
          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None):
    """LSE merge of P partials: o_parts [P, B, H, S, Dh] f32, lse_parts [P, B, H, S] f32."""
    P, B, H, S, Dh = o_parts.shape
    _need(o_parts, "o_parts", torch.float32)
    _need(lse_parts, "lse_parts", torch.float32, (P, B, H, S))
    if out is None:
        out = torch.empty((B, H, S, Dh), dtype=out_dtype, device=o_parts.device)
    if lse is None:
        lse = torch.empty((B, H, S), dtype=torch.float32, device=o_parts.device)
    _need(out, "out", out_dtype, (B, H, S, Dh))
    _need(lse, "lse", torch.float32, (B, H, S))
    code = _merge_ex(o_parts.data_ptr(), lse_parts.data_ptr(), P, out.data_ptr(), lse.data_ptr(), B, H, S, Dh,
                     RA_BF16 if out_dtype == torch.bfloat16 else RA_F32, _stream(stream))
    _check(code, "ring_attn_merge")
    return out, lse


def ring_order(D: int, r: int, causal: bool) -> List[int]:
    """Host-side ring schedule of the library (blocks visited by position r, in order)."""
    buf = (ctypes.c_int * max(D, 1))()
    n = _ring_order(D, r, 1 if causal else 0, buf, D)
    if n < 0:
        raise RingAttnError(-n, "ring_attn_ring_order")
    return list(buf[:n])


def visit_tiles(S: int, D: int, causal: bool, q0: int, rows: int) -> List[int]:
    """Host-side copy of the forward kernel's key-tile visit order for one query tile."""
    cap = S // 128 + 2
    buf = (ctypes.c_int * cap)()
    n = _visit_tiles(S, D, 1 if causal else 0, q0, rows, buf, cap)
    if n < 0:
        raise RingAttnError(-n, "ring_attn_visit_tiles")
    return list(buf[:n])


def bwd_visit_tiles(S: int, D: int, causal: bool, k0: int, rows: int = 128) -> List[int]:
    """Host-side copy of the backward kernel's query-tile visit order for one key tile."""
    cap = S // max(rows, 1) + 2
    buf = (ctypes.c_int * cap)()
    n = _bwd_visit_tiles(S, D, 1 if causal else 0, k0, rows, buf, cap)
    if n < 0:
        raise RingAttnError(-n, "ring_attn_bwd_visit_tiles")
    return list(buf[:n])


def exp2_check(x: torch.Tensor, stream=None):
    """Evaluate the kernels' two base-2 exponentials on x (float32, CUDA): returns
    (polynomial on the FMA pipes, hardware ex2.approx)."""
    _need(x, "x", torch.float32)
    y1, y2 = torch.empty_like(x), torch.empty_like(x)
    _check(_exp2_check(x.data_ptr(), y1.data_ptr(), y2.data_ptr(), x.numel(), _stream(stream)), "ring_attn_exp2_check")
    return y1, y2


def wait_selftest(timeout_s: float = 0.05, stream=None) -> None:
    """Run the bounded-wait self-test kernel (it records RA_ERR_TIMEOUT on purpose)."""
    _check(_wait_selftest(int(timeout_s * 1e9), _stream(stream)), "ring_attn_wait_selftest")


def launch_count() -> int:
    """Kernels launched by the library since it was loaded."""
    return int(_launch_count())


def device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) what kernels recorded: RA_ERR_TIMEOUT if a wait gave up,
    otherwise RA_ERR_PAGES if a cache call left an entry out, otherwise 0."""
    return int(_device_status(_stream(stream)))


def kernel_status(stream=None) -> int:
    """device_status() of RA_ERR_TIMEOUT alone; RA_ERR_PAGES is left for the cache's caller."""
    return int(_kernel_status(_stream(stream)))


# raw entry points (for tests of the C ABI itself)
raw = _lib
