"""Refusals of the paged cache's entry points, without a GPU."""
import ctypes

import pytest
import torch

from tests.test_span_cpu import sa  # noqa: F401  (the built package)

P = ctypes.c_void_p(16)


def _append(lib, k=P, q=P, q_out=P, kp=P, table=P, lens=P, out=P, Z=1, L=4, H=4, Hk=2, D=64, page=16, most=2, freq=P, rot=32,
            dtype=0):
    return lib.sigattn_cache_append(k, P, q, q_out, kp, P, table, lens, P, None, out, Z, L, H, Hk, D, 8, page, most, freq, rot,
                                    0, dtype, None)


def _paged(lib, q=P, kp=P, table=P, nk=P, pre=P, plen=P, Z=1, L=1, H=4, Hk=2, D=64, page=16, most=2, ahead=2, cap=0.0, ws=P,
           nbytes=1 << 40, dtype=0):
    return lib.sigattn_fwd_paged(q, kp, P, P, table, nk, P, pre, plen, Z, L, H, Hk, D, 8, page, most, ahead, 1.0, 0.0, None,
                                 cap, None, ws, nbytes, dtype, None)


def test_append_refusals(sa):  # noqa: F811
    lib = sa.load_library()
    assert _append(lib, D=96) == 2 and _append(lib, dtype=9) == 3
    for page in (0, 8, 24, 512):
        assert _append(lib, page=page) == 1
    assert _append(lib, H=3) == 1 and _append(lib, Hk=0) == 1 and _append(lib, Z=-1) == 1
    assert _append(lib, rot=8) == 1 and _append(lib, rot=80) == 1 and _append(lib, rot=-16) == 1
    assert _append(lib, freq=None) == 1
    assert _append(lib, k=None) == 1 and _append(lib, table=None) == 1 and _append(lib, lens=None) == 1
    assert _append(lib, out=None) == 1 and _append(lib, q_out=None) == 1 and _append(lib, kp=None) == 1
    assert _append(lib, k=ctypes.c_void_p(24)) == 5 and _append(lib, q_out=ctypes.c_void_p(24)) == 5
    assert _append(lib, Z=65536, L=65536) == 9 and _append(lib, most=2 ** 27) == 9
    assert _append(lib, Z=0) == 0


def test_paged_refusals(sa):  # noqa: F811
    lib = sa.load_library()
    assert _paged(lib, D=256) == 2 and _paged(lib, dtype=2) == 3 and _paged(lib, page=48) == 1
    assert _paged(lib, H=5) == 1 and _paged(lib, Hk=0) == 1 and _paged(lib, cap=-1.0) == 1
    assert _paged(lib, cap=float("nan")) == 1
    assert _paged(lib, q=None) == 1 and _paged(lib, kp=None) == 1 and _paged(lib, table=None) == 1 and _paged(lib, nk=None) == 1
    assert _paged(lib, pre=None) == 1
    need = lib.sigattn_fwd_paged_workspace_bytes(1, 1, 4, 2, 64, 0)
    assert need > 0 and lib.sigattn_fwd_paged_workspace_bytes(1, 1, 4, 2, 64, 1) == 0
    assert lib.sigattn_fwd_paged_workspace_bytes(1, 1, 4, 3, 64, 0) == 0
    assert _paged(lib, ws=None) == 1 and _paged(lib, nbytes=need - 1) == 1 and _paged(lib, ws=ctypes.c_void_p(20)) == 5
    assert _paged(lib, Z=4097) == 9 and _paged(lib, most=2 ** 27) == 9 and _paged(lib, Z=4096, most=2 ** 22) == 9
    assert _paged(lib, Z=0) == 0 and _paged(lib, L=0) == 0 and _paged(lib, H=0) == 0


def test_binding_refuses_cpu_tensors(sa):  # noqa: F811
    t = lambda h: torch.zeros(1, 4, h, 64, dtype=torch.bfloat16)      # noqa: E731
    n = torch.zeros(1, dtype=torch.int32)
    pages = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sa.cache_append(t(2), t(2), pages, pages, torch.zeros(1, 2, dtype=torch.int32), n, n)
    with pytest.raises(ValueError, match="CUDA"):
        sa.fwd_paged(t(2), pages, pages, torch.zeros(1, 2, dtype=torch.int32), n, n, 1.0, 0.0)
