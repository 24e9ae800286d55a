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

from . import _BF16, _FP32, _check, _dtype_code, _stream_ptr, load_library

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


_current_device = torch._C._cuda_getDevice


def run_on(device: int, f, args, name: str):
    """Calls entry point f with `device` as the current one."""
    if _current_device() == device:
        code = f(*args)
    else:
        with torch.cuda.device(device):
            code = f(*args)
    if code:
        _check(code, name)


def check_pair(q, keys, what="k and v"):
    """q [Z, L, H, D] and the tensors of its shared key heads [Z, L, Hk, D];
    returns (shape of q, Hk, device index)."""
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("tensors must be [Z, L, H, D]")
    device, dtype = q.get_device(), q.dtype
    if device < 0:
        raise ValueError("sigattn tensors must live on a CUDA device (no CPU fallback)")
    if not q.is_contiguous():
        raise ValueError("tensors must be contiguous [Z, L, H, D]")
    Z, L, H, D = shape
    first = keys[0].shape
    if len(first) != 4 or first[0] != Z or first[1] != L or first[3] != D:
        raise ValueError(f"{what} must be [Z, L, Hk, D] with the queries' Z, L and D")
    for t in keys:
        if t.shape != first:
            raise ValueError(f"{what} must be [Z, L, Hk, D] with the queries' Z, L and D")
        if t.dtype is not dtype or t.get_device() != device:
            raise ValueError("all tensors must share dtype and device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous [Z, L, Hk, D]")
    Hk = first[2]
    if H and (Hk == 0 or H % Hk):
        raise ValueError(f"{H} query heads cannot share {Hk} key heads evenly")
    return shape, Hk, device


def check_like(ref, tensors):
    for t in tensors:
        if t.shape != ref.shape or t.dtype is not ref.dtype or t.get_device() != ref.get_device() \
                or not t.is_contiguous():
            raise ValueError("outputs and gradients must be contiguous, with the shape, dtype and device "
                             "of the tensor they belong to")


def check_ints(t, shape, device, name):
    if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor on the tensors' device")


def check_floats(t, count, device, name):
    if t.dtype is not torch.float32 or t.shape != (count,) or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 [{count}] tensor on the tensors' device")


def score_args(Z, H, device, bias, cap, slopes):
    """(scalar bias, per-sample bias pointer, cap, slopes pointer) of a call."""
    bias_ptr = slopes_ptr = None
    if isinstance(bias, torch.Tensor):
        check_floats(bias, Z, device, "bias")
        bias_ptr, bias = bias.data_ptr(), 0.0
    if slopes is not None:
        check_floats(slopes, H, device, "slopes")
        slopes_ptr = slopes.data_ptr()
    return float(bias), bias_ptr, float(cap), slopes_ptr


def workspace_args(workspace, ref, device, size_of, args):
    """(tensor to hold until the launch, pointer, bytes) of the caller's workspace,
    or of one allocated for the call: its memory goes back to the allocator of the
    current stream, in whose order it may be used again."""
    if workspace is None:
        need = size_of(*args)
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=ref.device)
        return workspace, workspace.data_ptr(), need
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the tensors' device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _mask_args(Z, L, device, seqlens, spans):
    """(lengths pointer, spans pointer) of a call."""
    check_ints(seqlens, (Z,), device, "seqlens")
    if spans is None:
        return seqlens.data_ptr(), None
    check_ints(spans, (Z, L, 2), device, "spans")
    return seqlens.data_ptr(), spans.data_ptr()


def fwd_span(q, k, v, seqlens, alpha: float, bias, spans=None, cap: float = 0.0, slopes=None, out=None):
    """O [Z, L, H, D] of the masked attention.  ``k``, ``v``: [Z, L, Hk, D] with H
    a multiple of Hk.  ``seqlens``: int32 [Z] true lengths.  ``bias``: a number, or
    float32 [Z] with one bias per sample.  ``spans``: int32 [Z, L, 2], the keys
    [lo, hi) that each row sees (``mask_spans``; None: all).  ``cap``: 0 for none.
    ``slopes``: float32 [H], how fast a head's scores fall with |i - j|."""
    (Z, L, H, D), Hk, device = check_pair(q, (k, v))
    lens_ptr, spans_ptr = _mask_args(Z, L, device, seqlens, spans)
    b, bias_ptr, cap, slopes_ptr = score_args(Z, H, device, bias, cap, slopes)
    if out is None:
        out = torch.empty_like(q)
    else:
        check_like(q, (out,))
    run_on(device, load_library().sigattn_fwd_span,
           (q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lens_ptr, spans_ptr, Z, L, H, Hk, D,
            float(alpha), b, bias_ptr, cap, slopes_ptr, _dtype_code(q), _stream_ptr(q)), "sigattn_fwd_span")
    return out


def bwd_span_workspace_bytes(Z: int, L: int, dtype) -> int:
    """Device workspace bytes of ``bwd_span``."""
    code = _FP32 if dtype == torch.float32 else _BF16
    return int(load_library().sigattn_bwd_span_workspace_bytes(int(Z), int(L), code))


def bwd_span(q, k, v, dout, seqlens, alpha: float, bias, spans=None, cap: float = 0.0, slopes=None,
             dq=None, dk=None, dv=None, workspace=None):
    """(dQ, dK, dV) of ``fwd_span`` given dout = dLoss/dO; P is recomputed, O is
    not needed.  ``workspace``: a device uint8 tensor of at least
    ``bwd_span_workspace_bytes`` bytes (allocated here when omitted)."""
    (Z, L, H, D), Hk, device = check_pair(q, (k, v))
    lens_ptr, spans_ptr = _mask_args(Z, L, device, seqlens, spans)
    b, bias_ptr, cap, slopes_ptr = score_args(Z, H, device, bias, cap, slopes)
    check_like(q, (dout,) if dq is None else (dout, dq))
    check_like(k, [t for t in (dk, dv) if t is not None])
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    lib, code = load_library(), _dtype_code(q)
    workspace, ws_ptr, ws_bytes = workspace_args(workspace, q, device, lib.sigattn_bwd_span_workspace_bytes,
                                                 (Z, L, code))
    run_on(device, lib.sigattn_bwd_span,
           (q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
            lens_ptr, spans_ptr, Z, L, H, Hk, D, float(alpha), b, bias_ptr, cap, slopes_ptr, ws_ptr, ws_bytes, code,
            _stream_ptr(q)), "sigattn_bwd_span")
    return dq, dk, dv


def mask_spans(seqlens, L: int, causal: bool = False, prefix=None, docs=None, window: int = 0, out=None):
    """int32 [Z, L, 2]: the keys [lo, hi) that each row of a padded batch sees.

    ``causal``: the keys up to the row itself.  ``prefix``: int32 [Z], the first
    prefix[z] tokens are seen by every row and the rest causally (implies
    ``causal``).  ``docs``: int32 [Z, L], a document id per token; a row sees only
    the run of equal ids around it, and a prefix counts from the run's start.
    ``window`` > 0: at most that many keys back (and, without ``causal``, forward),
    the row's own included."""
    device = seqlens.get_device()
    if device < 0 or seqlens.dim() != 1:
        raise ValueError("seqlens must be a contiguous int32 [Z] CUDA tensor")
    Z, L, window = seqlens.shape[0], int(L), int(window)
    check_ints(seqlens, (Z,), device, "seqlens")
    if prefix is not None:
        check_ints(prefix, (Z,), device, "prefix")
        if window:
            raise ValueError("a prefix and a window do not make one interval of keys")
        causal = True
    if docs is not None:
        check_ints(docs, (Z, L), device, "docs")
    if out is None:
        out = torch.empty((Z, L, 2), dtype=torch.int32, device=seqlens.device)
    else:
        check_ints(out, (Z, L, 2), device, "out")
    run_on(device, load_library().sigattn_mask_spans,
           (seqlens.data_ptr(), None if prefix is None else prefix.data_ptr(),
            None if docs is None else docs.data_ptr(), int(bool(causal)), window, Z, L, out.data_ptr(),
            _stream_ptr(seqlens)), "sigattn_mask_spans")
    return out
