"""A paged cache of keys and values: appending to it with the position rotation
applied on the way, and attention against it, with a prefix that the whole batch
shares.  Bindings of ``sigattn_cache_append`` and ``sigattn_fwd_paged``
(include/sigattn.h)."""
from __future__ import annotations

import ctypes

import torch

from . import _BF16, _FP32, load_library, native

_vp, _ci, _cf, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t

PAGED_MAX_Z = 4096   # SIGATTN_PAGED_MAX_Z


def register(lib):
    """Argument types of this module's entry points."""
    lib.sigattn_cache_append.argtypes = [_vp] * 11 + [_ci] * 8 + [_vp, _ci, _ci, _ci, _vp]
    lib.sigattn_fwd_paged.argtypes = [_vp] * 9 + [_ci] * 9 + [_cf, _cf, _vp, _cf, _vp, _vp, _sz, _ci, _vp]
    lib.sigattn_fwd_paged_workspace_bytes.argtypes = [_ci] * 6
    lib.sigattn_fwd_paged_workspace_bytes.restype = _sz
    lib.sigattn_cache_append.restype = lib.sigattn_fwd_paged.restype = _ci


def cache_append(k, v, k_pages, v_pages, page_table, cache_lens, seqlens_new, inv_freq=None,
                 interleaved: bool = False, q=None, prefix_len=None, q_out=None, lens_out=None):
    """Writes new tokens into the cache and returns (rotated queries or None, new
    lengths int32 [Z]).

    ``k``, ``v``: [Z, L, Hk, D], of which sample z has seqlens_new[z] tokens; they go
    behind its cache_lens[z] places.  ``inv_freq``: float32 [rot / 2], the turn per
    position of each pair of the first rot entries of a head (a multiple of 16);
    None for no rotation.  ``interleaved``: pairs (2 i, 2 i + 1) instead of (i, i +
    rot / 2).  ``q``: [Z, L, H, D] queries to rotate as well.  ``prefix_len``: int32
    [1], tokens that stand before every sample's own.  ``lens_out`` may be
    ``cache_lens`` itself for single tokens (L = 1) and overlaps no length otherwise."""
    return native().cache_append(k, v, k_pages, v_pages, page_table, cache_lens, seqlens_new, inv_freq, interleaved, q,
                                 prefix_len, q_out, lens_out)


def fwd_paged_workspace_bytes(Z: int, L: int, H: int, Hk: int, D: int, dtype) -> int:
    """Device workspace bytes of ``fwd_paged``."""
    code = _FP32 if dtype == torch.float32 else _BF16
    return int(load_library().sigattn_fwd_paged_workspace_bytes(int(Z), int(L), int(H), int(Hk), int(D), code))


def fwd_paged(q, k_pages, v_pages, page_table, seqlens_k, seqlens_q, alpha: float, bias, prefix_table=None,
              prefix_len=None, cap: float = 0.0, slopes=None, out=None, workspace=None):
    """O [Z, L, H, D] of new tokens against a paged cache.

    Sample z has seqlens_k[z] own tokens in the pages page_table[z]; its
    seqlens_q[z] <= L queries are the last of them, each seeing its own tokens up
    to itself.  ``prefix_table`` (int32 [prefix_pages]) and ``prefix_len`` (int32
    [1]): the pages and length of a prefix that every query sees, read for up to 256
    rows of the batch at a time (bf16).  ``bias``, ``cap`` and ``slopes`` as in ``fwd_span``, distances
    counted in positions with the prefix first.  ``workspace``: a device uint8
    tensor of at least ``fwd_paged_workspace_bytes`` bytes (allocated here when
    omitted).  ``out`` may be ``q`` and overlaps no input otherwise."""
    return native().fwd_paged(q, k_pages, v_pages, page_table, seqlens_k, seqlens_q, alpha, bias, prefix_table,
                              prefix_len, cap, slopes, out, workspace)
