"""GPU tests of the masked attention where it can go wrong beyond the usual cases: far caps, sigma' in the tail, modules cast to
another type, later queries of the same warp, infinities in live rows, many samples."""
import math

import numpy as np
import pytest
import torch

from tests import _compare as C
from tests import _span_ref as R

pytestmark = pytest.mark.gpu

sa = pytest.importorskip("padding_aware_sigmoid_b200")


@pytest.fixture
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sa.last_device_status()
    yield torch.device("cuda", 0)
    assert sa.last_device_status() == 0


@pytest.fixture
def exp_mode():
    old = sa.get_sigmoid_mode()
    sa.set_sigmoid_mode(sa.SIGMOID_EXP)
    yield
    sa.set_sigmoid_mode(old)


def _tensors(Z, L, H, Hk, D, dtype, dev, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda h, s: (torch.randn(Z, L, h, D, generator=g) * s).to(dtype).to(dev)      # noqa: E731
    return r(H, scale), r(Hk, scale), r(Hk, 1.0), r(H, 1.0)


def _seq(n, dev):
    return torch.as_tensor(np.asarray(n, np.int32), device=dev)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [30.0, 1000.0, 1e6, 1e12])
def test_far_caps_in_exp_mode(dev, exp_mode, D, cap):
    """A cap far above the scores is nearly the identity.  The bounds of tests/_span_ref.py hold for it: their share for the
    argument, 3e-4, is a score's error of 2^-20 of itself (scores here stay below 60) many times over."""
    Z, L, H, Hk = 2, 300, 4, 2
    n = [300, 211]
    q, k, v, do = _tensors(Z, L, H, Hk, D, torch.bfloat16, dev, 11, 2.0)
    spans = R.make_spans("causal", n, L).to(dev)
    alpha, bias = D ** -0.5, -3.0
    args = dict(spans=spans, cap=cap)
    got = (sa.fwd_span(q, k, v, _seq(n, dev), alpha, bias, **args), *sa.bwd_span(q, k, v, do, _seq(n, dev), alpha, bias, **args))
    ref, bound = R.reference(q, k, v, do, R.visible(spans, n, L), alpha, [bias] * Z, cap, None)
    for name, x in zip(("O", "dQ", "dK", "dV"), got):
        R.assert_within(x, ref[name], bound[name], name)
