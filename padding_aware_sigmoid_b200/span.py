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

from . import _BF16, _FP32, _check, _stream_ptr, load_library, native

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


def fwd_span(q, k, v, seqlens, alpha: float, bias, spans=None, cap: float = 0.0, slopes=None, out=None):
    """O [Z, L, H, D] of the masked attention.  ``k``, ``v``: [Z, L, Hk, D] with H
    a multiple of Hk.  ``seqlens``: int32 [Z] true lengths.  ``bias``: a number, or
    float32 [Z] with one bias per sample.  ``spans``: int32 [Z, L, 2], the keys
    [lo, hi) that each row sees (``mask_spans``; None: all).  ``cap``: 0 for none.
    ``slopes``: float32 [H], how fast a head's scores fall with |i - j|.  ``out``
    must not overlap the inputs."""
    return native().fwd_span(q, k, v, seqlens, alpha, bias, spans, cap, slopes, out)


def bwd_span_workspace_bytes(Z: int, L: int, dtype) -> int:
    """Device workspace bytes of ``bwd_span``."""
    code = _FP32 if dtype == torch.float32 else _BF16
    return int(load_library().sigattn_bwd_span_workspace_bytes(int(Z), int(L), code))


def bwd_span(q, k, v, dout, seqlens, alpha: float, bias, spans=None, cap: float = 0.0, slopes=None,
             dq=None, dk=None, dv=None, workspace=None):
    """(dQ, dK, dV) of ``fwd_span`` given dout = dLoss/dO; P is recomputed, O is
    not needed.  ``workspace``: a device uint8 tensor of at least
    ``bwd_span_workspace_bytes`` bytes (allocated here when omitted).  The outputs
    must not overlap the inputs or one another."""
    return native().bwd_span(q, k, v, dout, seqlens, alpha, bias, spans, cap, slopes, dq, dk, dv, workspace)


def _check_ints(t, shape, device, name):
    if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 {list(shape)} tensor on the tensors' device")


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
    Z, L = seqlens.shape[0], int(L)
    window = max(-1, min(int(window), L))     # wider windows hide nothing; the library takes an int
    _check_ints(seqlens, (Z,), device, "seqlens")
    if prefix is not None:
        _check_ints(prefix, (Z,), device, "prefix")
        if window:
            raise ValueError("a prefix and a window do not make one interval of keys")
        causal = True
    if docs is not None:
        _check_ints(docs, (Z, L), device, "docs")
    if out is None:
        out = torch.empty((Z, L, 2), dtype=torch.int32, device=seqlens.device)
    else:
        _check_ints(out, (Z, L, 2), device, "out")
    with torch.cuda.device(device):
        _check(load_library().sigattn_mask_spans(
            seqlens.data_ptr(), None if prefix is None else prefix.data_ptr(),
            None if docs is None else docs.data_ptr(), int(bool(causal)), window, Z, L, out.data_ptr(),
            _stream_ptr(seqlens)), "sigattn_mask_spans")
    return out
