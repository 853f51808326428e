"""Python binding of libdashattn (the DashAttention forward and backward for B200).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/dashattn.h``.  PyTorch is used
for device memory and the current CUDA stream.  The library must have been
built (``python -m sparse_hierarchical_attention_mean_b200._build``); loading
fails loudly otherwise -- there is no fallback implementation.

Layouts (FlashAttention convention, last dim contiguous):
q, out [B, S, H, d]; k, v [B, S, Hkv, d]; summaries [B, Hkv, T, d] fp32.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
import struct

import torch
from torch.autograd import forward_ad

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdashattn.so")

DASH_OK = 0
_STATUS = {
    0: "DASH_OK",
    1: "DASH_ERR_INVALID_ARGUMENT",
    2: "DASH_ERR_UNSUPPORTED",
    3: "DASH_ERR_WORKSPACE_TOO_SMALL",
    4: "DASH_ERR_CUDA",
    5: "DASH_ERR_DEVICE_TIMEOUT",
    6: "DASH_ERR_OUT_OF_PAGES",
}
_DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}

# Every symbol include/dashattn.h declares.
EXPORTED = (
    "dash_attn_version",
    "dash_attn_last_error",
    "dash_attn_fwd_workspace_size",
    "dash_attn_fwd_workspace_lists",
    "dash_attn_decode_workspace_lists",
    "dash_attn_fwd",
    "dash_attn_summarize",
    "dash_attn_summarize_sdpa",
    "dash_attn_fwd_ex",
    "dash_attn_sparse_ex",
    "dash_attn_sparse_mask",
    "dash_attn_debug_sparse_stalled",
    "dash_attn_decode_ex",
    "dash_attn_lists_to_mask",
    "dash_attn_cp_scores",
    "dash_attn_cp_lists",
    "dash_attn_cp_attend",
    "dash_attn_cp_attend_workspace_size",
    "dash_attn_cp_attend_ex",
    "dash_attn_cp_merge",
    "dash_attn_summarize_paged",
    "dash_attn_decode_paged",
    "dash_attn_decode_workspace_size",
    "dash_attn_decode",
    "dash_attn_route_workspace_size",
    "dash_attn_route",
    "dash_attn_sparse_workspace_size",
    "dash_attn_sparse",
    "dash_attn_get_device_status",
    "dash_attn_decode_noalloc",
    "dash_attn_decode_noalloc_status",
    "dash_attn_bwd_workspace_size",
    "dash_attn_bwd",
    "dash_attn_window_fwd_workspace_size",
    "dash_attn_window_fwd",
    "dash_attn_window_bwd_workspace_size",
    "dash_attn_window_bwd",
    "dash_attn_window_decode_workspace_size",
    "dash_attn_window_decode",
    "dash_attn_window_decode_paged",
    "dash_attn_pages_workspace_size",
    "dash_attn_pages_fork",
    "dash_attn_pages_free",
    "dash_attn_pages_grow",
    "dash_attn_pages_compact",
    "dash_attn_pages_copy",
)


class DashError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


class DashOptions(ctypes.Structure):
    _fields_ = [("sigma", ctypes.c_float), ("qbar", ctypes.c_void_p)]


class DashTensor(ctypes.Structure):
    _fields_ = [
        ("data", ctypes.c_void_p),
        ("dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("b", ctypes.c_int64),
        ("s", ctypes.c_int64),
        ("h", ctypes.c_int64),
        ("d", ctypes.c_int64),
        ("stride_b", ctypes.c_int64),
        ("stride_s", ctypes.c_int64),
        ("stride_h", ctypes.c_int64),
    ]


def _load() -> ctypes.CDLL:
    if not os.path.exists(_LIB_PATH):
        raise ImportError(
            f"{_LIB_PATH} is missing: build it with `python -m sparse_hierarchical_attention_mean_b200._build`"
        )
    lib = ctypes.CDLL(_LIB_PATH)
    T = ctypes.POINTER(DashTensor)
    O = ctypes.POINTER(DashOptions)
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    sig = {
        "dash_attn_version": (i32, []),
        "dash_attn_last_error": (ctypes.c_char_p, []),
        "dash_attn_fwd_workspace_size": (sz, [T, T, i32]),
        "dash_attn_fwd_workspace_lists": (i32, [T, T, i32, vp, vp, vp, vp]),
        "dash_attn_decode_workspace_lists": (i32, [T, T, i32, i64, vp, vp, vp]),
        "dash_attn_fwd": (i32, [T, T, T, vp, f32, i32, i32, T, vp, sz, vp]),
        "dash_attn_summarize": (i32, [T, vp, vp, i32, vp, i64, i64, vp]),
        "dash_attn_summarize_sdpa": (i32, [T, vp, vp, vp, i32, vp, i64, i64, vp]),
        "dash_attn_decode_workspace_size": (sz, [T, T, i32, i64]),
        "dash_attn_decode": (i32, [T, T, T, vp, vp, i64, f32, i32, T, vp, sz, vp]),
        "dash_attn_route_workspace_size": (sz, [T, i64, i64, i32]),
        "dash_attn_route": (i32, [T, vp, i64, i64, vp, f32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
        "dash_attn_sparse_workspace_size": (sz, [T, T, i32, i64]),
        "dash_attn_sparse": (i32, [T, T, T, vp, vp, vp, i64, i32, i32, T, vp, sz, vp]),
        "dash_attn_fwd_ex": (i32, [T, T, T, vp, f32, i32, i32, T, vp, sz, O, vp]),
        "dash_attn_sparse_ex": (i32, [T, T, T, vp, vp, vp, i64, i32, i32, T, vp, sz, O, vp]),
        "dash_attn_sparse_mask": (i32, [T, T, T, vp, i64, vp, i64, i32, i32, T, vp, sz, O, vp]),
        "dash_attn_debug_sparse_stalled": (i32, [T, T, T, vp, vp, vp, i64, i32, i32, T, vp, sz, i64, vp]),
        "dash_attn_decode_ex": (i32, [T, T, T, vp, vp, i64, f32, i32, T, vp, sz, O, vp]),
        "dash_attn_lists_to_mask": (i32, [vp, vp, i64, i64, vp, i64, vp]),
        "dash_attn_cp_scores": (i32, [T, i64, vp, i64, i64, i64, vp, i64, f32, i32, vp, i64, vp]),
        "dash_attn_cp_lists": (i32, [T, i64, vp, vp, i64, f32, i32, vp, vp, vp, i64, vp]),
        "dash_attn_cp_attend": (i32, [T, T, T, i64, vp, i64, vp, vp, vp, i64, i32, O, vp, vp]),
        "dash_attn_cp_attend_workspace_size": (sz, [i64, i64, i64, i64, i32, i64]),
        "dash_attn_cp_attend_ex": (i32, [T, T, T, i64, vp, i64, vp, vp, vp, i64, i32, O, vp, vp, sz, vp]),
        "dash_attn_cp_merge": (i32, [vp, i64, T, vp]),
        "dash_attn_summarize_paged": (i32, [T, vp, i64, i64, vp, vp, vp, i32, vp, i64, i64, vp]),
        "dash_attn_decode_paged": (i32, [T, T, T, vp, i64, vp, vp, i64, f32, i32, T, vp, sz, O, vp]),
        "dash_attn_get_device_status": (i32, [vp, vp]),
        "dash_attn_decode_noalloc": (i32, [T, T, T, vp, vp, i64, f32, i32, T, vp]),
        "dash_attn_decode_noalloc_status": (i32, [vp]),
        "dash_attn_bwd_workspace_size": (sz, [T, T, i32]),
        "dash_attn_bwd": (i32, [T, T, T, vp, T, T, f32, i32, i32, O, T, T, T, vp, vp, sz, vp]),
        # tensor descriptors as plain pointers: the binding passes them packed (_packed)
        "dash_attn_window_fwd_workspace_size": (sz, [vp, vp]),
        "dash_attn_window_fwd": (i32, [vp, vp, vp, vp, i64, i64, vp, vp, vp, vp, sz, vp]),
        "dash_attn_window_bwd_workspace_size": (sz, [vp, vp, i64, i64]),
        "dash_attn_window_bwd": (i32, [vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, vp, vp, vp, vp, sz, vp]),
        "dash_attn_window_decode_workspace_size": (sz, [i64, i64, i64]),
        "dash_attn_window_decode": (i32, [vp, vp, vp, vp, i64, i64, vp, vp, vp, sz, vp]),
        "dash_attn_window_decode_paged": (i32, [vp, vp, vp, vp, i64, vp, i64, i64, vp, vp, vp, sz, vp]),
        "dash_attn_pages_workspace_size": (sz, [i64, i64, i64]),
        "dash_attn_pages_fork": (i32, [vp, i64, i64, vp, vp, i64, vp, vp, i64, i32, vp, sz, vp]),
        "dash_attn_pages_free": (i32, [vp, i64, i64, vp, vp, i64, vp, i64, i32, vp, sz, vp]),
        "dash_attn_pages_grow": (i32, [vp, i64, i64, vp, vp, i64, vp, i32, vp, vp, vp, sz, vp]),
        "dash_attn_pages_compact": (i32, [vp, i64, i64, vp, vp, i64, i32, vp, vp, vp, vp, vp, vp, sz, vp]),
        "dash_attn_pages_copy": (i32, [vp, i64, vp, vp, i64, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


class _Lazy:
    """Loads the library on first use (so the build step can import this package)."""

    _cdll = None

    def __getattr__(self, name):
        if _Lazy._cdll is None:
            _Lazy._cdll = _load()
        fn = getattr(_Lazy._cdll, name)
        setattr(self, name, fn)  # the next lookup does not come here
        return fn


_lib = _Lazy()


def library_path() -> str:
    return _LIB_PATH


def load() -> ctypes.CDLL:
    """Loads (once) and returns the library; raises ImportError if it is missing."""
    _lib.dash_attn_version  # noqa: B018
    return _Lazy._cdll


def version() -> int:
    return _lib.dash_attn_version()


def _check(status: int) -> None:
    if status != DASH_OK:
        raise DashError(status, _lib.dash_attn_last_error().decode())


def _desc(t: torch.Tensor) -> DashTensor:
    if t.dim() != 4:
        raise ValueError("expected a [B, S, H, d] tensor")
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA device tensors")
    if t.stride(3) != 1:
        raise ValueError("the last dimension must be contiguous")
    if t.dtype not in _DTYPE:
        raise ValueError(f"unsupported dtype {t.dtype}")
    b, s, h, d = t.shape
    return DashTensor(t.data_ptr(), _DTYPE[t.dtype], 0, b, s, h, d, t.stride(0), t.stride(1), t.stride(2))


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _options(sigma: float, qbar: torch.Tensor | None):
    """None for the defaults (sigma 1, mean pooling), else a pointer to DashOptions."""
    if sigma == 1.0 and qbar is None:
        return None
    if qbar is not None:
        assert qbar.is_cuda and qbar.is_contiguous() and qbar.dtype == torch.float32
    return ctypes.byref(DashOptions(float(sigma), None if qbar is None else qbar.data_ptr()))


def _workspace(nbytes: int, device, given: torch.Tensor | None) -> torch.Tensor:
    if given is not None:
        return given
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def n_blocks(seq: int, block: int) -> int:
    return -(-seq // block)


# ------------------------------------------------------------------ stage 0


def summarize(k: torch.Tensor, w_s: torch.Tensor, block: int, seqlens: torch.Tensor | None = None,
              summaries: torch.Tensor | None = None, first_block: int = 0, stream=None,
              qbar: torch.Tensor | None = None) -> torch.Tensor:
    """Block summaries [B, Hkv, t_cap, d] fp32 (see dash_attn_summarize).

    qbar: optional fp32 [Hkv, d] learned summary queries (dash_attn_summarize_sdpa).
    """
    B, S, Hkv, d = k.shape
    if summaries is None:
        summaries = torch.zeros((B, Hkv, n_blocks(S, block), d), dtype=torch.float32, device=k.device)
    assert summaries.is_contiguous() and summaries.dtype == torch.float32
    kd = _desc(k)
    if qbar is None:
        _check(_lib.dash_attn_summarize(ctypes.byref(kd), _ptr(seqlens), w_s.data_ptr(), block,
                                        summaries.data_ptr(), summaries.shape[2], first_block, _stream(stream)))
    else:
        assert qbar.is_contiguous() and qbar.dtype == torch.float32 and tuple(qbar.shape) == (Hkv, d)
        _check(_lib.dash_attn_summarize_sdpa(ctypes.byref(kd), _ptr(seqlens), w_s.data_ptr(), qbar.data_ptr(),
                                             block, summaries.data_ptr(), summaries.shape[2], first_block,
                                             _stream(stream)))
    return summaries


# ------------------------------------------------------------------ stage 1


def route_workspace_size(q: torch.Tensor, kv_heads: int, t_cap: int, decode: bool) -> int:
    qd = _desc(q)
    return _lib.dash_attn_route_workspace_size(ctypes.byref(qd), kv_heads, t_cap, 1 if decode else 0)


def route(q: torch.Tensor, summaries: torch.Tensor, alpha: float, block: int, causal: bool = True,
          seqlens: torch.Tensor | None = None, want_tau: bool = False, want_p: bool = False,
          idx=None, logp=None, cnt=None, workspace=None, stream=None) -> dict:
    """Stage 1 alone; returns idx, logp [B, Hkv, Sq, t_cap], cnt [B, Hkv, Sq] (+ tau, p).

    idx / logp / cnt / workspace may be passed in to reuse buffers.
    """
    B, Sq, H, d = q.shape
    _, Hkv, t_cap, _ = summaries.shape
    dev = q.device
    if idx is None:
        idx = torch.full((B, Hkv, Sq, t_cap), -1, dtype=torch.int32, device=dev)
    if logp is None:
        logp = torch.zeros((B, Hkv, Sq, t_cap), dtype=torch.float32, device=dev)
    if cnt is None:
        cnt = torch.zeros((B, Hkv, Sq), dtype=torch.int32, device=dev)
    tau = torch.zeros((B, H, Sq), dtype=torch.float32, device=dev) if want_tau else None
    p = torch.zeros((B, H, Sq, t_cap), dtype=torch.float32, device=dev) if want_p else None
    ws = None
    if seqlens is not None:
        ws = _workspace(route_workspace_size(q, Hkv, t_cap, True), dev, workspace)
    elif q.dtype != torch.float32:
        ws = _workspace(route_workspace_size(q, Hkv, t_cap, False), dev, workspace)  # split summaries
    qd = _desc(q)
    _check(_lib.dash_attn_route(ctypes.byref(qd), summaries.data_ptr(), Hkv, t_cap, _ptr(seqlens), alpha, block,
                                1 if causal else 0, idx.data_ptr(), logp.data_ptr(), cnt.data_ptr(), _ptr(tau),
                                _ptr(p), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)))
    return {"idx": idx, "logp": logp, "cnt": cnt, "tau": tau, "p": p, "workspace": ws}


# ------------------------------------------------------------------ stage 2


def sparse_workspace_size(q: torch.Tensor, k: torch.Tensor, block: int, t_cap: int) -> int:
    qd, kd = _desc(q), _desc(k)
    return _lib.dash_attn_sparse_workspace_size(ctypes.byref(qd), ctypes.byref(kd), block, t_cap)


def sparse(q, k, v, idx, logp, cnt, block: int, causal: bool = True, out=None, workspace=None,
           stream=None, sigma: float = 1.0) -> torch.Tensor:
    """Stage 2 alone on caller-given routing (layout of :func:`route`); sigma: prior strength."""
    out = torch.empty_like(q) if out is None else out
    t_cap = idx.shape[-1]
    ws = _workspace(sparse_workspace_size(q, k, block, t_cap), q.device, workspace)
    qd, kd, vd, od = _desc(q), _desc(k), _desc(v), _desc(out)
    opts = _options(sigma, None)
    args = (ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), idx.data_ptr(), logp.data_ptr(), cnt.data_ptr(),
            t_cap, block, 1 if causal else 0, ctypes.byref(od), ws.data_ptr(), ws.numel())
    if opts is None:
        _check(_lib.dash_attn_sparse(*args, _stream(stream)))
    else:
        _check(_lib.dash_attn_sparse_ex(*args, opts, _stream(stream)))
    return out


def sparse_mask(q, k, v, mask: torch.Tensor, logp_dense: torch.Tensor, block: int, causal: bool = True, out=None,
                workspace=None, sigma: float = 1.0, stream=None) -> torch.Tensor:
    """Stage 2 on bit-packed masks [B, Hkv, S, n_words] (int32 bit patterns) and a dense log p_bar
    [B, Hkv, S, t_cap] (see dash_attn_sparse_mask)."""
    assert mask.is_contiguous() and mask.dtype == torch.int32 and logp_dense.is_contiguous()
    assert logp_dense.dtype == torch.float32
    out = torch.empty_like(q) if out is None else out
    t_cap, n_words = logp_dense.shape[-1], mask.shape[-1]
    ws = _workspace(sparse_workspace_size(q, k, block, t_cap), q.device, workspace)
    qd, kd, vd, od = _desc(q), _desc(k), _desc(v), _desc(out)
    _check(_lib.dash_attn_sparse_mask(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), mask.data_ptr(), n_words,
                                      logp_dense.data_ptr(), t_cap, block, 1 if causal else 0, ctypes.byref(od),
                                      ws.data_ptr(), ws.numel(), ctypes.byref(DashOptions(float(sigma), None)),
                                      _stream(stream)))
    return out


def debug_sparse_stalled(q, k, v, idx, logp, cnt, block: int, causal: bool, out, workspace, wait_cycles: int,
                         stream=None) -> None:
    """Stage 2 with its copies withheld and short waits (see dash_attn_debug_sparse_stalled): a test of
    the timeout path; the workspace status word then reads DASH_ERR_DEVICE_TIMEOUT."""
    qd, kd, vd, od = _desc(q), _desc(k), _desc(v), _desc(out)
    _check(_lib.dash_attn_debug_sparse_stalled(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), idx.data_ptr(),
                                               logp.data_ptr(), cnt.data_ptr(), idx.shape[-1], block,
                                               1 if causal else 0, ctypes.byref(od), workspace.data_ptr(),
                                               workspace.numel(), wait_cycles, _stream(stream)))


def lists_to_mask(idx: torch.Tensor, cnt: torch.Tensor, n_words: int | None = None, stream=None) -> torch.Tensor:
    """Bit-packed active-block masks [..., n_words] (int32 bit patterns) from lists idx [..., t_cap], cnt [...]."""
    t_cap = idx.shape[-1]
    n_words = -(-t_cap // 32) if n_words is None else n_words
    rows = cnt.numel()
    mask = torch.empty(tuple(cnt.shape) + (n_words,), dtype=torch.int32, device=idx.device)
    assert idx.is_contiguous() and cnt.is_contiguous() and idx.dtype == torch.int32 and cnt.dtype == torch.int32
    _check(_lib.dash_attn_lists_to_mask(idx.data_ptr(), cnt.data_ptr(), rows, t_cap, mask.data_ptr(), n_words,
                                        _stream(stream)))
    return mask


# ------------------------------------------------------------------ full forward


def fwd_workspace_size(q: torch.Tensor, k: torch.Tensor, block: int) -> int:
    qd, kd = _desc(q), _desc(k)
    n = _lib.dash_attn_fwd_workspace_size(ctypes.byref(qd), ctypes.byref(kd), block)
    if n == 0:
        raise DashError(1, "arguments rejected by dash_attn_fwd_workspace_size")
    return n


def fwd(q, k, v, w_s, alpha: float, block: int, causal: bool = True, out=None, workspace=None,
        stream=None, sigma: float = 1.0, qbar: torch.Tensor | None = None) -> torch.Tensor:
    """Full prefill forward (stages 0-2); see dash_attn_fwd (and dash_attn_fwd_ex for sigma / qbar)."""
    out = torch.empty_like(q) if out is None else out
    ws = _workspace(fwd_workspace_size(q, k, block), q.device, workspace)
    qd, kd, vd, od = _desc(q), _desc(k), _desc(v), _desc(out)
    opts = _options(sigma, qbar)
    args = (ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), w_s.data_ptr(), alpha, block, 1 if causal else 0,
            ctypes.byref(od), ws.data_ptr(), ws.numel())
    if opts is None:
        _check(_lib.dash_attn_fwd(*args, _stream(stream)))
    else:
        _check(_lib.dash_attn_fwd_ex(*args, opts, _stream(stream)))
    return out


def _view(ws: torch.Tensor, offset: int, shape, dtype) -> torch.Tensor:
    n = 1
    for e in shape:
        n *= e
    nbytes = n * torch.tensor([], dtype=dtype).element_size()
    return ws[offset:offset + nbytes].view(dtype).view(*shape)


def fwd_lists(workspace: torch.Tensor, q: torch.Tensor, k: torch.Tensor, block: int) -> dict:
    """Views into a fwd workspace of the call's summaries and routing lists (dash_attn_fwd_workspace_lists)."""
    qd, kd = _desc(q), _desc(k)
    off = [ctypes.c_size_t() for _ in range(4)]
    _check(_lib.dash_attn_fwd_workspace_lists(ctypes.byref(qd), ctypes.byref(kd), block,
                                              *[ctypes.byref(o) for o in off]))
    B, S, _, d = q.shape
    Hkv, T = k.shape[2], n_blocks(S, block)
    return {"summaries": _view(workspace, off[0].value, (B, Hkv, T, d), torch.float32),
            "idx": _view(workspace, off[1].value, (B, Hkv, S, T), torch.int32),
            "logp": _view(workspace, off[2].value, (B, Hkv, S, T), torch.float32),
            "cnt": _view(workspace, off[3].value, (B, Hkv, S), torch.int32)}


# ------------------------------------------------------------------ backward


def bwd_workspace_size(q: torch.Tensor, k: torch.Tensor, block: int) -> int:
    qd, kd = _desc(q), _desc(k)
    n = _lib.dash_attn_bwd_workspace_size(ctypes.byref(qd), ctypes.byref(kd), block)
    if n == 0:
        raise DashError(1, "arguments rejected by dash_attn_bwd_workspace_size")
    return n


def bwd(q, k, v, w_s, out, dout, alpha: float, block: int, causal: bool = True, sigma: float = 1.0,
        grads=None, workspace=None, stream=None) -> dict:
    """Gradients of sum(dout * out) (see dash_attn_bwd): dq, dk, dv fp32 and dw_s [d, d] fp32.

    grads: optional dict of preallocated fp32 dq / dk / dv / dw_s.
    """
    d = q.shape[-1]
    g = grads or {}
    dq = g.get("dq", torch.empty(q.shape, dtype=torch.float32, device=q.device))
    dk = g.get("dk", torch.empty(k.shape, dtype=torch.float32, device=q.device))
    dv = g.get("dv", torch.empty(v.shape, dtype=torch.float32, device=q.device))
    dw_s = g.get("dw_s", torch.empty((d, d), dtype=torch.float32, device=q.device))
    ws = _workspace(bwd_workspace_size(q, k, block), q.device, workspace)
    descs = [_desc(t) for t in (q, k, v, out, dout, dq, dk, dv)]
    qd, kd, vd, od, dod, dqd, dkd, dvd = descs
    opts = ctypes.byref(DashOptions(float(sigma), None))
    _check(_lib.dash_attn_bwd(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), w_s.data_ptr(), ctypes.byref(od),
                              ctypes.byref(dod), alpha, block, 1 if causal else 0, opts, ctypes.byref(dqd),
                              ctypes.byref(dkd), ctypes.byref(dvd), dw_s.data_ptr(), ws.data_ptr(), ws.numel(),
                              _stream(stream)))
    return {"dq": dq, "dk": dk, "dv": dv, "dw_s": dw_s}


class _DashAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, w_s, alpha, block, causal, sigma):
        out = fwd(q, k, v, w_s, alpha, block, causal, sigma=sigma)
        ctx.save_for_backward(q, k, v, w_s, out)
        ctx.args = (alpha, block, causal, sigma)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, w_s, out = ctx.saved_tensors
        alpha, block, causal, sigma = ctx.args
        g = bwd(q, k, v, w_s, out, dout.contiguous(), alpha, block, causal, sigma)
        return (g["dq"].to(q.dtype), g["dk"].to(k.dtype), g["dv"].to(v.dtype), g["dw_s"].to(w_s.dtype),
                None, None, None, None)


def attention(q, k, v, w_s, alpha: float, block: int, causal: bool = True, sigma: float = 1.0) -> torch.Tensor:
    """Differentiable DashAttention prefill (f16/bf16): forward by dash_attn_fwd_ex, gradients by dash_attn_bwd."""
    return _DashAttention.apply(q, k, v, w_s, alpha, block, causal, sigma)


# ------------------------------------------------------------------ decode


def decode_workspace_size(q: torch.Tensor, kcache: torch.Tensor, block: int, t_cap: int) -> int:
    qd, kd = _desc(q), _desc(kcache)
    n = _lib.dash_attn_decode_workspace_size(ctypes.byref(qd), ctypes.byref(kd), block, t_cap)
    if n == 0:
        raise DashError(1, "arguments rejected by dash_attn_decode_workspace_size")
    return n


def decode(q, kcache, vcache, seqlens, summaries, alpha: float, block: int, out=None, workspace=None,
           stream=None, sigma: float = 1.0) -> torch.Tensor:
    """One decode step for q [B, 1, H, d] (see dash_attn_decode); sigma: prior strength."""
    out = torch.empty_like(q) if out is None else out
    t_cap = summaries.shape[2]
    ws = _workspace(decode_workspace_size(q, kcache, block, t_cap), q.device, workspace)
    qd, kd, vd, od = _desc(q), _desc(kcache), _desc(vcache), _desc(out)
    opts = _options(sigma, None)
    args = (ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), seqlens.data_ptr(), summaries.data_ptr(), t_cap,
            alpha, block, ctypes.byref(od), ws.data_ptr(), ws.numel())
    if opts is None:
        _check(_lib.dash_attn_decode(*args, _stream(stream)))
    else:
        _check(_lib.dash_attn_decode_ex(*args, opts, _stream(stream)))
    return out


def decode_lists(workspace: torch.Tensor, q: torch.Tensor, kcache: torch.Tensor, block: int, t_cap: int) -> dict:
    """Views into a decode workspace of the step's routing lists (dash_attn_decode_workspace_lists)."""
    qd, kd = _desc(q), _desc(kcache)
    off = [ctypes.c_size_t() for _ in range(3)]
    _check(_lib.dash_attn_decode_workspace_lists(ctypes.byref(qd), ctypes.byref(kd), block, t_cap,
                                                 *[ctypes.byref(o) for o in off]))
    B, Hkv = q.shape[0], kcache.shape[2]
    return {"idx": _view(workspace, off[0].value, (B, Hkv, t_cap), torch.int32),
            "logp": _view(workspace, off[1].value, (B, Hkv, t_cap), torch.float32),
            "cnt": _view(workspace, off[2].value, (B, Hkv), torch.int32)}


def decode_noalloc(q, kcache, vcache, seqlens, summaries, alpha: float, block: int, out=None,
                   stream=None) -> torch.Tensor:
    """One decode step without a workspace (see dash_attn_decode_noalloc).

    For callers that may not allocate device memory while they run: the
    library keeps a fixed 16 MiB scratch array per GPU.  Only ``out`` is
    allocated here when it is not given.  Concurrent calls on one device race.
    """
    out = torch.empty_like(q) if out is None else out
    qd, kd, vd, od = _desc(q), _desc(kcache), _desc(vcache), _desc(out)
    _check(_lib.dash_attn_decode_noalloc(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), seqlens.data_ptr(),
                                         summaries.data_ptr(), summaries.shape[2], alpha, block, ctypes.byref(od),
                                         _stream(stream)))
    return out


def decode_noalloc_status(stream=None) -> int:
    """Status word of the last decode_noalloc call on the current device (synchronises)."""
    return _lib.dash_attn_decode_noalloc_status(_stream(stream))


def device_status(workspace: torch.Tensor, stream=None) -> int:
    """Status word of the last call that used ``workspace`` (synchronises)."""
    return _lib.dash_attn_get_device_status(workspace.data_ptr(), _stream(stream))



# ------------------------------------------------------------------ context-parallel decode


def cp_scores(q, summaries, block_lo: int, block_hi: int, seqlens, lmax: int, alpha: float, block: int,
              scores: torch.Tensor, stream=None) -> torch.Tensor:
    """This rank's routing logits into ``scores`` [B, Hkv, G, t_cap] (see dash_attn_cp_scores)."""
    B, Hkv, summ_cap, d = summaries.shape
    qd = _desc(q)
    _check(_lib.dash_attn_cp_scores(ctypes.byref(qd), Hkv, summaries.data_ptr(), summ_cap, block_lo, block_hi,
                                    seqlens.data_ptr(), lmax, alpha, block, scores.data_ptr(), scores.shape[3],
                                    _stream(stream)))
    return scores


def cp_lists(q, kv_heads: int, scores, seqlens, lmax: int, alpha: float, block: int, stream=None) -> dict:
    """alpha-entmax, GQA mean and ascending lists from whole score vectors (see dash_attn_cp_lists)."""
    B, Hkv, G, t_cap = scores.shape
    dev = q.device
    idx = torch.full((B, Hkv, t_cap), -1, dtype=torch.int32, device=dev)
    logp = torch.zeros((B, Hkv, t_cap), dtype=torch.float32, device=dev)
    cnt = torch.zeros((B, Hkv), dtype=torch.int32, device=dev)
    qd = _desc(q)
    _check(_lib.dash_attn_cp_lists(ctypes.byref(qd), kv_heads, scores.data_ptr(), seqlens.data_ptr(), lmax, alpha,
                                   block, idx.data_ptr(), logp.data_ptr(), cnt.data_ptr(), t_cap, _stream(stream)))
    return {"idx": idx, "logp": logp, "cnt": cnt}


def cp_attend(q, kshard, vshard, tok_lo: int, seqlens, lmax: int, lists: dict, block: int, sigma: float = 1.0,
              part=None, stream=None) -> torch.Tensor:
    """Partials [B, H, d + 2] of this rank's tokens (see dash_attn_cp_attend)."""
    B, _, H, d = q.shape
    part = torch.empty((B, H, d + 2), dtype=torch.float32, device=q.device) if part is None else part
    qd, kd, vd = _desc(q), _desc(kshard), _desc(vshard)
    t_cap = lists["idx"].shape[-1]
    _check(_lib.dash_attn_cp_attend(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), tok_lo, seqlens.data_ptr(),
                                    lmax, lists["idx"].data_ptr(), lists["logp"].data_ptr(), lists["cnt"].data_ptr(),
                                    t_cap, block, _options(sigma, None), part.data_ptr(), _stream(stream)))
    return part


def cp_attend_workspace_size(B: int, H: int, Hkv: int, d: int, block: int, t_cap: int) -> int:
    """Bytes of workspace dash_attn_cp_attend_ex needs."""
    return int(_lib.dash_attn_cp_attend_workspace_size(B, H, Hkv, d, block, t_cap))


def cp_attend_ex(q, kshard, vshard, tok_lo: int, seqlens, lmax: int, lists: dict, block: int, sigma: float = 1.0,
                 part=None, workspace=None, stream=None) -> torch.Tensor:
    """Partials [B, H, d + 2] of this rank's tokens on the split-KV path (see dash_attn_cp_attend_ex)."""
    B, _, H, d = q.shape
    Hkv = kshard.shape[2]
    t_cap = lists["idx"].shape[-1]
    part = torch.empty((B, H, d + 2), dtype=torch.float32, device=q.device) if part is None else part
    n_ws = cp_attend_workspace_size(B, H, Hkv, d, block, t_cap)
    if workspace is None:
        workspace = torch.empty(n_ws, dtype=torch.uint8, device=q.device)
    qd, kd, vd = _desc(q), _desc(kshard), _desc(vshard)
    _check(_lib.dash_attn_cp_attend_ex(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), tok_lo,
                                       seqlens.data_ptr(), lmax, lists["idx"].data_ptr(), lists["logp"].data_ptr(),
                                       lists["cnt"].data_ptr(), t_cap, block, _options(sigma, None), part.data_ptr(),
                                       workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                       _stream(stream)))
    return part


def cp_merge(parts: torch.Tensor, out: torch.Tensor, stream=None) -> torch.Tensor:
    """Merge partials [R, B, H, d + 2] into out [B, 1, H, d] (see dash_attn_cp_merge)."""
    assert parts.is_contiguous() and parts.dtype == torch.float32
    od = _desc(out)
    _check(_lib.dash_attn_cp_merge(parts.data_ptr(), parts.shape[0], ctypes.byref(od), _stream(stream)))
    return out


# ------------------------------------------------------------------ paged KV cache


def summarize_paged(k_pages, block_table, seqlens, w_s, block: int, summaries=None, t_cap: int | None = None,
                    first_block: int = 0, qbar=None, stream=None) -> torch.Tensor:
    """Summaries [B, Hkv, t_cap, d] from a paged cache (see dash_attn_summarize_paged)."""
    n_pages, page, Hkv, d = k_pages.shape
    B, max_blocks = block_table.shape
    t_cap = max_blocks if t_cap is None else t_cap
    if summaries is None:
        summaries = torch.zeros((B, Hkv, t_cap, d), dtype=torch.float32, device=k_pages.device)
    kd = _desc(k_pages)
    _check(_lib.dash_attn_summarize_paged(ctypes.byref(kd), block_table.data_ptr(), max_blocks, B, seqlens.data_ptr(),
                                          w_s.data_ptr(), _ptr(qbar), block, summaries.data_ptr(), summaries.shape[2],
                                          first_block, _stream(stream)))
    return summaries


def decode_paged(q, k_pages, v_pages, block_table, seqlens, summaries, alpha: float, block: int, out=None,
                 workspace=None, sigma: float = 1.0, stream=None) -> torch.Tensor:
    """One decode step against a paged cache (see dash_attn_decode_paged)."""
    out = torch.empty_like(q) if out is None else out
    B, max_blocks = block_table.shape
    t_cap = summaries.shape[2]
    qd, kd, vd, od = _desc(q), _desc(k_pages), _desc(v_pages), _desc(out)
    # the workspace is that of a dense cache of the same B, Hkv, d (only the shape enters the size query)
    dk = DashTensor(k_pages.data_ptr(), kd.dtype, 0, B, max_blocks * block, kd.h, kd.d,
                    kd.h * kd.d * max_blocks * block, kd.h * kd.d, kd.d)
    nbytes = _lib.dash_attn_decode_workspace_size(ctypes.byref(qd), ctypes.byref(dk), block, t_cap)
    ws = _workspace(nbytes, q.device, workspace)
    _check(_lib.dash_attn_decode_paged(ctypes.byref(qd), ctypes.byref(kd), ctypes.byref(vd), block_table.data_ptr(),
                                       max_blocks, seqlens.data_ptr(), summaries.data_ptr(), t_cap, alpha, block,
                                       ctypes.byref(od), ws.data_ptr(), ws.numel(), _options(sigma, None),
                                       _stream(stream)))
    return out


# ------------------------------------------------------------------ dense / sliding-window attention


class _On:
    """Device and stream of a call: every tensor on one device, buffers allocated for the stream they are used on.

    ``with _On(stream, first, ...) as handle``: the cudaStream_t to launch on.  The common case (no stream given,
    tensors on the current device) costs a microsecond; a one-token step is bound by the host otherwise.
    """

    __slots__ = ("_dev", "_stream", "_stack")

    def __init__(self, stream, first, *others):
        dev = first.get_device()
        if dev < 0:
            raise ValueError("tensors must be CUDA device tensors")
        for t in others:
            if t is not None and t.get_device() != dev:
                raise ValueError(f"tensors on different devices: {first.device} and {t.device}")
        if stream is not None and stream.device != first.device:
            raise ValueError(f"a stream of {stream.device} for tensors on {first.device}")
        self._dev, self._stream, self._stack = dev, stream, None

    def __enter__(self):
        if self._stream is not None or self._dev != torch.cuda.current_device():
            self._stack = contextlib.ExitStack()
            self._stack.enter_context(torch.cuda.device(self._dev))
            self._stack.enter_context(torch.cuda.stream(self._stream))
        return torch._C._cuda_getCurrentRawStream(self._dev)

    def __exit__(self, *error):
        if self._stack is not None:
            self._stack.close()
        return False


_PACK = struct.Struct("=qiiqqqqqqq").pack  # dash_tensor_t


def _packed(t: torch.Tensor) -> bytes:
    """A dash_tensor_t as bytes, with the checks of :func:`_desc`."""
    shape = t.shape
    if len(shape) != 4:
        raise ValueError("expected a [B, S, H, d] tensor")
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA device tensors")
    sb, ss, sh, sd = t.stride()
    if sd != 1:
        raise ValueError("the last dimension must be contiguous")
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return _PACK(t.data_ptr(), code, 0, *shape, sb, ss, sh)


def _array(t: torch.Tensor | None, name: str, shape, dtype=torch.int32):
    """Device pointer of a contiguous array of the given shape (None: not given)."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)}")
    return t.data_ptr()


def _scratch(nbytes: int, what: str, device, given: torch.Tensor | None):
    """A workspace and its size in bytes."""
    if nbytes == 0:
        raise DashError(1, f"arguments rejected by {what}: {_lib.dash_attn_last_error().decode()}")
    if given is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes
    if not given.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return given, given.numel() * given.element_size()


def window_fwd_workspace_size(q: torch.Tensor, k: torch.Tensor) -> int:
    return _lib.dash_attn_window_fwd_workspace_size(_packed(q), _packed(k))


def window_fwd(q, k, v, window: int = 0, sinks: int = 0, seqlens: torch.Tensor | None = None, out=None,
               return_lse: bool = False, lse=None, rest=None, workspace=None, stream=None):
    """Causal attention over a sliding window and the first ``sinks`` tokens (see dash_attn_window_fwd).

    window 0: every earlier token.  seqlens: optional int32 [B], the valid tokens of each sequence of a padded
    batch.  rest: optional tensor like out (f16 / bf16) that receives what rounding took from it.  Returns out
    [B, S, H, d], and with ``return_lse`` the log-sum-exp [B, H, S] fp32 too.
    """
    with _On(stream, q, k, v, seqlens, out, lse, rest, workspace) as s:
        qd, kd = _packed(q), _packed(k)
        B, S, H, _ = q.shape
        out = torch.empty_like(q) if out is None else out
        if return_lse and lse is None:
            lse = q.new_empty((B, H, S), dtype=torch.float32)
        ws, room = _scratch(_lib.dash_attn_window_fwd_workspace_size(qd, kd), "dash_attn_window_fwd_workspace_size",
                            q.device, workspace)
        _check(_lib.dash_attn_window_fwd(qd, kd, _packed(v), _array(seqlens, "seqlens", (B,)), window, sinks,
                                         _packed(out), None if rest is None else _packed(rest),
                                         _array(lse, "lse", (B, H, S), torch.float32), ws.data_ptr(), room, s))
    return (out, lse) if return_lse else out


def window_bwd_workspace_size(q: torch.Tensor, k: torch.Tensor, window: int = 0, sinks: int = 0) -> int:
    return _lib.dash_attn_window_bwd_workspace_size(_packed(q), _packed(k), window, sinks)


def window_bwd(q, k, v, out, lse, dout, window: int = 0, sinks: int = 0, seqlens: torch.Tensor | None = None,
               grads=None, rest=None, workspace=None, stream=None) -> dict:
    """Gradients of sum(dout * out) (see dash_attn_window_bwd): dq, dk, dv in the inputs' type.

    out, lse (and rest, if it was asked for): those of :func:`window_fwd`.  grads: optional dict of preallocated dq / dk / dv.
    """
    g = grads or {}
    with _On(stream, q, k, v, out, lse, dout, seqlens, rest, workspace, *g.values()) as s:
        B, S, H, _ = q.shape
        dq, dk, dv = (g[n] if n in g else torch.empty_like(t) for n, t in (("dq", q), ("dk", k), ("dv", v)))
        qd, kd = _packed(q), _packed(k)
        ws, room = _scratch(_lib.dash_attn_window_bwd_workspace_size(qd, kd, window, sinks),
                            "dash_attn_window_bwd_workspace_size", q.device, workspace)
        _check(_lib.dash_attn_window_bwd(qd, kd, _packed(v), _packed(out), None if rest is None else _packed(rest),
                                         _array(lse, "lse", (B, H, S), torch.float32), _packed(dout),
                                         _array(seqlens, "seqlens", (B,)), window, sinks, _packed(dq), _packed(dk),
                                         _packed(dv), ws.data_ptr(), room, s))
    return {"dq": dq, "dk": dk, "dv": dv}


def _readable(t: torch.Tensor) -> torch.Tensor:
    """t, or a copy of it where its strides or its address are not ones that the kernels read."""
    *outer, last = t.stride()
    if last == 1 and all(x > 0 and x * t.element_size() % 16 == 0 for x in outer) and t.data_ptr() % 16 == 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)


class _WindowAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, window, sinks, seqlens):
        if not any(ctx.needs_input_grad[:3]):
            return window_fwd(q, k, v, window, sinks, seqlens)
        rest = torch.empty_like(q) if q.dtype != torch.float32 else None
        out, lse = window_fwd(q, k, v, window, sinks, seqlens, return_lse=True, rest=rest)
        ctx.save_for_backward(q, k, v, out, lse, rest, seqlens)
        ctx.args = (window, sinks)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse, rest, seqlens = ctx.saved_tensors
        g = window_bwd(q, k, v, out, lse, _readable(dout), *ctx.args, seqlens, rest=rest)
        return g["dq"], g["dk"], g["dv"], None, None, None


def window_attention(q, k, v, window: int = 0, sinks: int = 0, seqlens: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable :func:`window_fwd` (reverse mode): by dash_attn_window_fwd and dash_attn_window_bwd.

    In a captured step, as for any operator of torch, the leaves must have no eager graph alive when the capture
    starts: the gradients would be accumulated on the stream of that graph, outside the capture.
    """
    # without gradients there is nothing to keep for a backward; a tangent is the function's to refuse
    if not torch.is_grad_enabled() and not any(forward_ad.unpack_dual(t).tangent is not None for t in (q, k, v)):
        return window_fwd(q, k, v, window, sinks, seqlens)
    return _WindowAttention.apply(q, k, v, window, sinks, seqlens)


def window_decode_workspace_size(heads: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace the one-token calls need on the current device (whatever the batch and the lengths)."""
    return _lib.dash_attn_window_decode_workspace_size(heads, kv_heads, head_dim)


def window_decode(q, kcache, vcache, seqlens, window: int = 0, sinks: int = 0, out=None, return_lse: bool = False,
                  lse=None, workspace=None, stream=None):
    """Attention of one new token per sequence, q [B, 1, H, d], over its cache (see dash_attn_window_decode)."""
    return _window_decode(q, kcache, vcache, None, seqlens, window, sinks, out, return_lse, lse, workspace, stream)


def window_decode_paged(q, k_pages, v_pages, block_table, seqlens, window: int = 0, sinks: int = 0, out=None,
                        return_lse: bool = False, lse=None, workspace=None, stream=None):
    """:func:`window_decode` against a paged cache (see dash_attn_window_decode_paged)."""
    return _window_decode(q, k_pages, v_pages, block_table, seqlens, window, sinks, out, return_lse, lse, workspace,
                          stream)


def _window_decode(q, k, v, table, seqlens, window, sinks, out, return_lse, lse, workspace, stream):
    with _On(stream, q, k, v, table, seqlens, out, lse, workspace) as s:
        qd, kd, vd = _packed(q), _packed(k), _packed(v)
        B, _, H, d = q.shape
        out = torch.empty_like(q) if out is None else out
        if return_lse and lse is None:
            lse = q.new_empty((B, H), dtype=torch.float32)
        ws, room = _scratch(_lib.dash_attn_window_decode_workspace_size(H, k.shape[2], d),
                            "dash_attn_window_decode_workspace_size", q.device, workspace)
        tail = (_array(seqlens, "seqlens", (B,)), window, sinks, _packed(out),
                _array(lse, "lse", (B, H), torch.float32), ws.data_ptr(), room, s)
        if table is None:
            _check(_lib.dash_attn_window_decode(qd, kd, vd, *tail))
        else:
            if table.dim() != 2:
                raise ValueError("block_table must be [B, max_blocks]")
            most = table.shape[1]
            _check(_lib.dash_attn_window_decode_paged(qd, kd, vd, _array(table, "block_table", (B, most)), most,
                                                      *tail))
    return (out, lse) if return_lse else out


# ------------------------------------------------------------------ cache pages


def _pages_state(block_table, seqlens, refs):
    """The arguments (table, batch, max_blocks, seqlens, refs, n_pages) of the calls on a block table."""
    if block_table.dim() != 2 or refs.dim() != 1:
        raise ValueError("block_table must be [batch, max_blocks] and refs [n_pages]")
    batch, most = block_table.shape
    return (_array(block_table, "block_table", (batch, most)), batch, most, _array(seqlens, "seqlens", (batch,)),
            _array(refs, "refs", (refs.shape[0],)), refs.shape[0])


def pages_workspace_size(batch: int, max_blocks: int, n_pages: int) -> int:
    return _lib.dash_attn_pages_workspace_size(batch, max_blocks, n_pages)


def _pages_scratch(state, device, given):
    return _scratch(_lib.dash_attn_pages_workspace_size(state[1], state[2], state[5]),
                    "dash_attn_pages_workspace_size", device, given)


def pages_fork(block_table, seqlens, refs, src, dst, block: int, workspace=None, stream=None) -> None:
    """Sequences dst[i] become copies of src[i] that share their pages, in place (see dash_attn_pages_fork)."""
    with _On(stream, block_table, seqlens, refs, src, dst, workspace) as s:
        state = _pages_state(block_table, seqlens, refs)
        n = dst.numel()
        ws, room = _pages_scratch(state, block_table.device, workspace)
        _check(_lib.dash_attn_pages_fork(*state, _array(src, "src", (n,)), _array(dst, "dst", (n,)), n, block,
                                         ws.data_ptr(), room, s))


def pages_free(block_table, seqlens, refs, slots, block: int, workspace=None, stream=None) -> None:
    """The sequences slots[i] give back their pages, in place (see dash_attn_pages_free)."""
    with _On(stream, block_table, seqlens, refs, slots, workspace) as s:
        state = _pages_state(block_table, seqlens, refs)
        n = slots.numel()
        ws, room = _pages_scratch(state, block_table.device, workspace)
        _check(_lib.dash_attn_pages_free(*state, _array(slots, "slots", (n,)), n, block, ws.data_ptr(), room, s))


class Grown(tuple):
    """copy_src, copy_dst of :func:`pages_grow`, with the workspace whose status word says whether the pool sufficed."""

    workspace: torch.Tensor


def pages_grow(block_table, seqlens, refs, n_new, block: int, workspace=None, stream=None) -> Grown:
    """Room for n_new[b] more tokens of every sequence, in place (see dash_attn_pages_grow).

    Returns copy_src, copy_dst [batch]: the page copies to make with :func:`pages_copy` before the new tokens are
    written (-1: none).  When the pool has too few free pages nothing changes, the lengths neither, and
    ``device_status(result.workspace)`` is 6 (DASH_ERR_OUT_OF_PAGES): where the pool can run out, look at it before
    the tokens are written (it synchronises), or count the free pages beforehand.
    """
    with _On(stream, block_table, seqlens, refs, n_new, workspace) as s:
        state = _pages_state(block_table, seqlens, refs)
        batch = state[1]
        src, dst = torch.empty_like(n_new), torch.empty_like(n_new)
        ws, room = _pages_scratch(state, block_table.device, workspace)
        _check(_lib.dash_attn_pages_grow(*state, _array(n_new, "n_new", (batch,)), block, src.data_ptr(),
                                         dst.data_ptr(), ws.data_ptr(), room, s))
    grown = Grown((src, dst))
    grown.workspace = ws
    return grown


def pages_compact(block_table, seqlens, refs, block: int, inplace: bool = False, workspace=None, stream=None) -> dict:
    """The pages in use move to the low end of the pool (see dash_attn_pages_compact).

    Returns table and refs after it (the inputs themselves with ``inplace``), the moves src, dst [n_pages // 2] to
    make with :func:`pages_copy` (-1 past their number) and info [2] = {moves, pages in use}.  Pages that other tables
    or owners hold (counted in refs) move too: their entries equal to src[i] have to become dst[i].
    """
    with _On(stream, block_table, seqlens, refs, workspace) as s:
        state = _pages_state(block_table, seqlens, refs)
        dev, n_pages = block_table.device, state[5]
        table_out = block_table if inplace else torch.empty_like(block_table)
        refs_out = refs if inplace else torch.empty_like(refs)
        src, dst, info = (refs.new_empty(n) for n in (n_pages // 2, n_pages // 2, 2))
        ws, room = _pages_scratch(state, dev, workspace)
        _check(_lib.dash_attn_pages_compact(*state, block, table_out.data_ptr(), refs_out.data_ptr(), src.data_ptr(),
                                            dst.data_ptr(), info.data_ptr(), ws.data_ptr(), room, s))
    return {"table": table_out, "refs": refs_out, "src": src, "dst": dst, "info": info}


def pages_copy(pools, src, dst, stream=None) -> None:
    """Page src[i] of every pool [n_pages, s, h, d] to page dst[i] (see dash_attn_pages_copy)."""
    pools = list(pools)
    if not pools:
        raise ValueError("no pools")
    with _On(stream, *pools, src, dst) as s:
        n = src.numel()
        _check(_lib.dash_attn_pages_copy(b"".join(map(_packed, pools)), len(pools), _array(src, "src", (n,)),
                                         _array(dst, "dst", (n,)), n, s))
