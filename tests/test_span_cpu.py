"""Refusals of the masked attention's entry points, without a GPU: the C ABI's checks and the binding's."""
import ctypes
import os
import shutil

import pytest
import torch


@pytest.fixture(scope="module")
def sa():
    from padding_aware_sigmoid_b200 import build
    if not os.path.exists(build.OUT):
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("nvcc unavailable and library not built")
        build.build()
    import padding_aware_sigmoid_b200 as pkg
    return pkg


P = ctypes.c_void_p(16)


def _fwd(lib, q=P, seqlens=P, spans=P, Z=1, L=128, H=4, Hk=2, D=64, alpha=1.0, cap=0.0, dtype=0):
    return lib.sigattn_fwd_span(q, P, P, P, seqlens, spans, Z, L, H, Hk, D, alpha, 0.0, None, cap, None, dtype, None)


def _bwd(lib, dv=P, ws=P, nbytes=1 << 30, H=4, Hk=2, D=64, cap=0.0, dtype=0):
    return lib.sigattn_bwd_span(P, P, P, P, P, P, dv, P, P, 1, 128, H, Hk, D, 1.0, 0.0, None, cap, None, ws, nbytes, dtype,
                                None)


def test_forward_refusals(sa):
    lib = sa.load_library()
    assert _fwd(lib, D=96) == 2
    assert _fwd(lib, dtype=3) == 3
    assert _fwd(lib, Z=-1) == 1 and _fwd(lib, L=-1) == 1 and _fwd(lib, H=65536, Hk=1) == 1
    assert _fwd(lib, H=0, Hk=2) == 1
    assert _fwd(lib, H=4, Hk=3) == 1 and _fwd(lib, H=4, Hk=0) == 1 and _fwd(lib, H=2, Hk=4) == 1
    assert _fwd(lib, q=None) == 1 and _fwd(lib, seqlens=None) == 1
    assert _fwd(lib, q=ctypes.c_void_p(18)) == 5 and _fwd(lib, spans=ctypes.c_void_p(20)) == 5
    for cap in (-1.0, float("nan"), float("inf"), 1e-45):
        assert _fwd(lib, cap=cap, alpha=10.0) == 1
    assert _fwd(lib, Z=0) == 0 and _fwd(lib, L=0) == 0 and _fwd(lib, H=0, Hk=0) == 0
    assert _fwd(lib, Z=65535, L=2 ** 31 - 300, H=65535, Hk=1, dtype=1) == 9


def test_backward_refusals(sa):
    lib = sa.load_library()
    need = lib.sigattn_bwd_span_workspace_bytes(1, 128, 0)
    assert need == 128 * 8 + 16
    assert lib.sigattn_bwd_span_workspace_bytes(3, 129, 0) == 3 * 2 * (128 * 8 + 16)
    assert lib.sigattn_bwd_span_workspace_bytes(3, 129, 1) == 0 and lib.sigattn_bwd_span_workspace_bytes(0, 5, 0) == 0
    assert _bwd(lib, ws=None) == 1 and _bwd(lib, nbytes=need - 1) == 1
    assert _bwd(lib, ws=ctypes.c_void_p(24)) == 5
    assert _bwd(lib, dv=None) == 1 and _bwd(lib, dv=ctypes.c_void_p(8)) == 5
    assert _bwd(lib, H=4, Hk=3) == 1 and _bwd(lib, D=32) == 2 and _bwd(lib, cap=-2.0) == 1


def test_mask_refusals(sa):
    lib = sa.load_library()
    f = lib.sigattn_mask_spans
    assert f(P, None, None, 0, -1, 1, 8, P, None) == 1
    assert f(P, P, None, 0, 0, 1, 8, P, None) == 1          # a prefix without causal
    assert f(P, P, None, 1, 4, 1, 8, P, None) == 1          # a prefix with a window
    assert f(None, None, None, 1, 0, 1, 8, P, None) == 1 and f(P, None, None, 1, 0, 1, 8, None, None) == 1
    assert f(P, None, None, 1, 0, 1, 8, ctypes.c_void_p(12), None) == 5
    assert f(P, None, None, 1, 0, 0, 8, None, None) == 0


def test_binding_refuses_cpu_tensors_and_uneven_heads(sa):
    t = lambda h: torch.zeros(1, 8, h, 64, dtype=torch.bfloat16)      # noqa: E731
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sa.fwd_span(t(2), t(2), t(2), n, 1.0, 0.0)
    with pytest.raises(ValueError, match="CUDA"):
        sa.bwd_span(t(2), t(2), t(2), t(2), n, 1.0, 0.0)
    with pytest.raises(ValueError, match="CUDA"):
        sa.mask_spans(n, 8)


def test_masked_module_refuses_what_has_no_gradient(sa):
    with pytest.raises(ValueError, match="learned bias"):
        sa.SigmoidAttention(learnable_bias=True, bias=-1.0, cap=20.0)
    with pytest.raises(ValueError, match="cap"):
        sa.SigmoidAttention(cap=-1.0)
    m = sa.SigmoidAttention(learnable_bias=True, bias=-1.0)
    x = torch.zeros(1, 4, 2, 64)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="learned bias"):
        m(x, x[:, :, :1], x[:, :, :1], n)
    with pytest.raises(ValueError, match="one length"):
        sa.SigmoidAttention()(x, x[:, :, :1], x[:, :, :1], n, n.clone())
    assert sa.SigmoidAttention(slopes=[0.5, 0.25]).slopes.tolist() == [0.5, 0.25]
    assert not sa.SigmoidAttention(slopes=[0.5]).state_dict()
