"""Masked attention: an interval of keys per query row (causal, prefix, document
and window masks), a tanh cap on the scores, a bias that falls with distance,
and query heads that share key heads.  Bindings of ``sigattn_fwd_span``,
``sigattn_bwd_span`` and ``sigattn_mask_spans`` (include/sigattn.h).

    x_ij = cap tanh(alpha q_i . k_j / cap) - slopes[h] |i - j| + b
    O_i  = sum over lo_i <= j < hi_i of sigma(x_ij) v_j
"""
from __future__ import annotations

import ctypes

import torch

_vp, _ci, _cf, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t


def register(lib):
    """Argument types of this module's entry points."""
    lib.sigattn_fwd_span.argtypes = [_vp] * 6 + [_ci] * 5 + [_cf, _cf, _vp, _cf, _vp, _ci, _vp]
    lib.sigattn_bwd_span.argtypes = [_vp] * 9 + [_ci] * 5 + [_cf, _cf, _vp, _cf, _vp, _vp, _sz, _ci, _vp]
    lib.sigattn_bwd_span_workspace_bytes.argtypes = [_ci, _ci, _ci]
    lib.sigattn_bwd_span_workspace_bytes.restype = _sz
    lib.sigattn_mask_spans.argtypes = [_vp, _vp, _vp, _ci, _ci, _ci, _ci, _vp, _vp]
    for f in (lib.sigattn_fwd_span, lib.sigattn_bwd_span, lib.sigattn_mask_spans):
        f.restype = _ci


class on_device:
    """Makes a tensor's device the current one for a call, when it is not."""

    __slots__ = ("index", "before")

    def __init__(self, t):
        self.index = t.get_device()

    def __enter__(self):
        self.before = torch._C._cuda_getDevice()
        if self.before != self.index:
            torch._C._cuda_setDevice(self.index)

    def __exit__(self, *exc):
        if self.before != self.index:
            torch._C._cuda_setDevice(self.before)
        return False


def check_pair(q, keys, what="k and v"):
    """q [Z, L, H, D] and the tensors of its shared key heads [Z, L, Hk, D]."""
    if q.dim() != 4:
        raise ValueError("tensors must be [Z, L, H, D]")
    if not q.is_cuda:
        raise ValueError("sigattn tensors must live on a CUDA device (no CPU fallback)")
    if not q.is_contiguous():
        raise ValueError("tensors must be contiguous [Z, L, H, D]")
    Z, L, H, D = q.shape
    ref = keys[0]
    for t in keys:
        if t.dim() != 4 or t.shape != ref.shape or t.shape[:2] != q.shape[:2] or t.shape[3] != D:
            raise ValueError(f"{what} must be [Z, L, Hk, D] with the queries' Z, L and D")
        if t.dtype != q.dtype or t.device != q.device:
            raise ValueError("all tensors must share dtype and device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous [Z, L, Hk, D]")
    Hk = ref.shape[2]
    if H and (Hk == 0 or H % Hk):
        raise ValueError(f"{H} query heads cannot share {Hk} key heads evenly")


def check_like(ref, tensors):
    for t in tensors:
        if t.shape != ref.shape or t.dtype != ref.dtype or t.device != ref.device or not t.is_contiguous():
            raise ValueError("outputs and gradients must be contiguous, with the shape, dtype and device "
                             "of the tensor they belong to")


def check_ints(t, shape, device, name):
    if not (t.dtype == torch.int32 and tuple(t.shape) == tuple(shape) and t.is_contiguous()
            and t.device == device):
        raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor on the tensors' device")


def check_floats(t, count, device, name):
    if not (t.dtype == torch.float32 and t.dim() == 1 and t.shape[0] == count and t.is_contiguous()
            and t.device == device):
        raise ValueError(f"{name} must be a contiguous float32 [{count}] tensor on the tensors' device")


def score_args(q, bias, cap, slopes):
    """(scalar bias, per-sample bias pointer, cap, slopes pointer) of a call."""
    bias_ptr = slopes_ptr = None
    if isinstance(bias, torch.Tensor):
        check_floats(bias, q.shape[0], q.device, "bias")
        bias_ptr, bias = bias.data_ptr(), 0.0
    if slopes is not None:
        check_floats(slopes, q.shape[2], q.device, "slopes")
        slopes_ptr = slopes.data_ptr()
    return float(bias), bias_ptr, float(cap), slopes_ptr


def _check_mask(q, seqlens, spans):
    check_ints(seqlens, q.shape[:1], q.device, "seqlens")
    if spans is not None:
        check_ints(spans, (q.shape[0], q.shape[1], 2), q.device, "spans")


def fwd_span(q, k, v, seqlens, alpha: float, bias, spans=None, cap: float = 0.0, slopes=None, out=None):
    """O [Z, L, H, D] of the masked attention.  ``k``, ``v``: [Z, L, Hk, D] with H
    a multiple of Hk.  ``seqlens``: int32 [Z] true lengths.  ``bias``: a number, or
    float32 [Z] with one bias per sample.  ``spans``: int32 [Z, L, 2], the keys
    [lo, hi) that each row sees (``mask_spans``; None: all).  ``cap``: 0 for none.
    ``slopes``: float32 [H], how fast a head's scores fall with |i - j|."""
    from . import _check, _dtype_code, _stream_ptr, load_library
    check_pair(q, [k, v])
    _check_mask(q, seqlens, spans)
    b, bias_ptr, cap, slopes_ptr = score_args(q, bias, cap, slopes)
    if out is None:
        out = torch.empty_like(q)
    else:
        check_like(q, [out])
    Z, L, H, D = q.shape
    with on_device(q):
        _check(load_library().sigattn_fwd_span(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), seqlens.data_ptr(),
            None if spans is None else spans.data_ptr(), Z, L, H, k.shape[2], D, float(alpha), b, bias_ptr,
            cap, slopes_ptr, _dtype_code(q), _stream_ptr(q)), "sigattn_fwd_span")
    return out


def bwd_span_workspace_bytes(Z: int, L: int, dtype) -> int:
    """Device workspace bytes of ``bwd_span``."""
    from . import _BF16, _FP32, load_library
    code = _FP32 if dtype == torch.float32 else _BF16
    return int(load_library().sigattn_bwd_span_workspace_bytes(int(Z), int(L), code))


def bwd_span(q, k, v, dout, seqlens, alpha: float, bias, spans=None, cap: float = 0.0, slopes=None,
             dq=None, dk=None, dv=None, workspace=None):
    """(dQ, dK, dV) of ``fwd_span`` given dout = dLoss/dO; P is recomputed, O is
    not needed.  ``workspace``: a device uint8 tensor of at least
    ``bwd_span_workspace_bytes`` bytes (allocated here when omitted)."""
    from . import _check, _dtype_code, _stream_ptr, load_library
    check_pair(q, [k, v])
    _check_mask(q, seqlens, spans)
    b, bias_ptr, cap, slopes_ptr = score_args(q, bias, cap, slopes)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    check_like(q, [dout, dq])
    check_like(k, [dk, dv])
    Z, L, H, D = q.shape
    code = _dtype_code(q)
    if workspace is None:
        lib = load_library()
        workspace = torch.empty(lib.sigattn_bwd_span_workspace_bytes(Z, L, code), dtype=torch.uint8,
                                device=q.device)
    elif workspace.device != q.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the tensors' device")
    with on_device(q):
        _check(load_library().sigattn_bwd_span(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
            dv.data_ptr(), seqlens.data_ptr(), None if spans is None else spans.data_ptr(), Z, L, H,
            k.shape[2], D, float(alpha), b, bias_ptr, cap, slopes_ptr, workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), code, _stream_ptr(q)), "sigattn_bwd_span")
    return dq, dk, dv


def mask_spans(seqlens, L: int, causal: bool = False, prefix=None, docs=None, window: int = 0, out=None):
    """int32 [Z, L, 2]: the keys [lo, hi) that each row of a padded batch sees.

    ``causal``: the keys up to the row itself.  ``prefix``: int32 [Z], the first
    prefix[z] tokens are seen by every row and the rest causally (implies
    ``causal``).  ``docs``: int32 [Z, L], a document id per token; a row sees only
    the run of equal ids around it, and a prefix counts from the run's start.
    ``window`` > 0: at most that many keys back (and, without ``causal``, forward),
    the row's own included."""
    from . import _check, _stream_ptr, load_library
    if not (isinstance(seqlens, torch.Tensor) and seqlens.is_cuda and seqlens.dim() == 1):
        raise ValueError("seqlens must be a contiguous int32 [Z] CUDA tensor")
    Z, L, window = seqlens.shape[0], int(L), int(window)
    check_ints(seqlens, (Z,), seqlens.device, "seqlens")
    if prefix is not None:
        check_ints(prefix, (Z,), seqlens.device, "prefix")
        if window:
            raise ValueError("a prefix and a window do not make one interval of keys")
        causal = True
    if docs is not None:
        check_ints(docs, (Z, L), seqlens.device, "docs")
    if out is None:
        out = torch.empty((Z, L, 2), dtype=torch.int32, device=seqlens.device)
    else:
        check_ints(out, (Z, L, 2), seqlens.device, "out")
    with on_device(seqlens):
        _check(load_library().sigattn_mask_spans(
            seqlens.data_ptr(), None if prefix is None else prefix.data_ptr(),
            None if docs is None else docs.data_ptr(), int(bool(causal)), window, Z, L, out.data_ptr(),
            _stream_ptr(seqlens)), "sigattn_mask_spans")
    return out
