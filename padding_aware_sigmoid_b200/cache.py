"""A paged cache of keys and values: appending to it with the position rotation
applied on the way, and attention against it, with a prefix that the whole batch
shares.  Bindings of ``sigattn_cache_append`` and ``sigattn_fwd_paged``
(include/sigattn.h)."""
from __future__ import annotations

import ctypes

import torch

from . import _BF16, _FP32, _dtype_code, _stream_ptr, load_library
from .span import check_floats, check_ints, check_like, check_pair, run_on, score_args, workspace_args

_vp, _ci, _cf, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t

PAGED_MAX_Z = 4096   # SIGATTN_PAGED_MAX_Z


def register(lib):
    """Argument types of this module's entry points."""
    lib.sigattn_cache_append.argtypes = [_vp] * 11 + [_ci] * 8 + [_vp, _ci, _ci, _ci, _vp]
    lib.sigattn_fwd_paged.argtypes = [_vp] * 9 + [_ci] * 9 + [_cf, _cf, _vp, _cf, _vp, _vp, _sz, _ci, _vp]
    lib.sigattn_fwd_paged_workspace_bytes.argtypes = [_ci] * 6
    lib.sigattn_fwd_paged_workspace_bytes.restype = _sz
    lib.sigattn_cache_append.restype = lib.sigattn_fwd_paged.restype = _ci


_PAGE_SIZES = (16, 32, 64, 128, 256)


def _check_pages(dtype, device, D, k_pages, v_pages, Hk=None):
    """Cache pages [pages, page_size, Hk, D] beside the call's tensors; returns their shape."""
    shape = k_pages.shape
    if len(shape) != 4 or shape[3] != D or v_pages.shape != shape or (Hk is not None and shape[2] != Hk):
        raise ValueError("k_pages and v_pages must be [pages, page_size, Hk, D]")
    for t in (k_pages, v_pages):
        if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
            raise ValueError("k_pages and v_pages must be contiguous, with the tensors' dtype and device")
    if shape[1] not in _PAGE_SIZES:
        raise ValueError(f"page_size must be 16, 32, 64, 128 or 256, got {shape[1]}")
    return shape


def _check_table(page_table, Z, device):
    """Checks the page table and returns its width."""
    if page_table.dim() != 2:
        raise ValueError("page_table must be a contiguous int32 [Z, max_pages] tensor")
    most = page_table.shape[1]
    check_ints(page_table, (Z, most), device, "page_table")
    return most


def cache_append(k, v, k_pages, v_pages, page_table, cache_lens, seqlens_new, inv_freq=None,
                 interleaved: bool = False, q=None, prefix_len=None, q_out=None, lens_out=None):
    """Writes new tokens into the cache and returns (rotated queries or None, new
    lengths int32 [Z]).

    ``k``, ``v``: [Z, L, Hk, D], of which sample z has seqlens_new[z] tokens; they go
    behind its cache_lens[z] places.  ``inv_freq``: float32 [rot / 2], the turn per
    position of each pair of the first rot entries of a head (a multiple of 16);
    None for no rotation.  ``interleaved``: pairs (2 i, 2 i + 1) instead of (i, i +
    rot / 2).  ``q``: [Z, L, H, D] queries to rotate as well.  ``prefix_len``: int32
    [1], tokens that stand before every sample's own."""
    if q is not None:
        (Z, L, H, D), Hk, device = check_pair(q, (k, v))
    else:
        (Z, L, Hk, D), _, device = check_pair(k, (v,), "v")
        H = 0
    if k.shape != v.shape:
        raise ValueError("k and v must be [Z, L, Hk, D]")
    pages, page_size, _, _ = _check_pages(k.dtype, device, D, k_pages, v_pages, Hk)
    most = _check_table(page_table, Z, device)
    check_ints(cache_lens, (Z,), device, "cache_lens")
    check_ints(seqlens_new, (Z,), device, "seqlens_new")
    if prefix_len is not None:
        check_ints(prefix_len, (1,), device, "prefix_len")
    rot, freq_ptr = 0, None
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        check_floats(inv_freq, rot // 2, device, "inv_freq")
        if rot % 16 or rot > D:
            raise ValueError(f"inv_freq must turn a multiple of 16 entries of a head, at most {D}, got {rot}")
        freq_ptr = inv_freq.data_ptr()
    q_ptr = out_ptr = None
    if q is not None:
        if q_out is None:
            q_out = torch.empty_like(q)
        else:
            check_like(q, (q_out,))
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    if lens_out is None:
        lens_out = torch.empty_like(cache_lens)
    else:
        check_ints(lens_out, (Z,), device, "lens_out")
        if L > 1 and lens_out.data_ptr() == cache_lens.data_ptr():
            raise ValueError("lens_out can be cache_lens itself only for single tokens")
    run_on(device, load_library().sigattn_cache_append,
           (k.data_ptr(), v.data_ptr(), q_ptr, out_ptr, k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
            cache_lens.data_ptr(), seqlens_new.data_ptr(), None if prefix_len is None else prefix_len.data_ptr(),
            lens_out.data_ptr(), Z, L, H, Hk, D, pages, page_size, most, freq_ptr, rot, 1 if interleaved else 0,
            _dtype_code(k), _stream_ptr(k)), "sigattn_cache_append")
    return (None if q is None else q_out), lens_out


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
    [1]): the pages and length of a prefix that every query sees, read once for
    the batch.  ``bias``, ``cap`` and ``slopes`` as in ``fwd_span``, distances
    counted in positions with the prefix first.  ``workspace``: a device uint8
    tensor of at least ``fwd_paged_workspace_bytes`` bytes (allocated here when
    omitted)."""
    shape, device = q.shape, q.get_device()
    if len(shape) != 4:
        raise ValueError("q must be [Z, L, H, D]")
    if device < 0:
        raise ValueError("sigattn tensors must live on a CUDA device (no CPU fallback)")
    if not q.is_contiguous():
        raise ValueError("q must be contiguous [Z, L, H, D]")
    Z, L, H, D = shape
    pages, page_size, Hk, _ = _check_pages(q.dtype, device, D, k_pages, v_pages)
    if H and (Hk == 0 or H % Hk):
        raise ValueError(f"{H} query heads cannot share {Hk} key heads evenly")
    most = _check_table(page_table, Z, device)
    check_ints(seqlens_k, (Z,), device, "seqlens_k")
    check_ints(seqlens_q, (Z,), device, "seqlens_q")
    if (prefix_table is None) != (prefix_len is None):
        raise ValueError("prefix_table and prefix_len go together")
    prefix_pages, table_ptr, len_ptr = 0, None, None
    if prefix_table is not None:
        prefix_pages = prefix_table.numel()
        check_ints(prefix_table, (prefix_pages,), device, "prefix_table")
        check_ints(prefix_len, (1,), device, "prefix_len")
        table_ptr, len_ptr = prefix_table.data_ptr(), prefix_len.data_ptr()
    b, bias_ptr, cap, slopes_ptr = score_args(Z, H, device, bias, cap, slopes)
    if out is None:
        out = torch.empty_like(q)
    else:
        check_like(q, (out,))
    lib, code = load_library(), _dtype_code(q)
    workspace, ws_ptr, ws_bytes = workspace_args(workspace, q, device, lib.sigattn_fwd_paged_workspace_bytes,
                                                 (Z, L, H, Hk, D, code))
    run_on(device, lib.sigattn_fwd_paged,
           (q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), out.data_ptr(), page_table.data_ptr(),
            seqlens_k.data_ptr(), seqlens_q.data_ptr(), table_ptr, len_ptr, Z, L, H, Hk, D, pages, page_size, most,
            prefix_pages, float(alpha), b, bias_ptr, cap, slopes_ptr, ws_ptr, ws_bytes, code, _stream_ptr(q)),
           "sigattn_fwd_paged")
    return out
