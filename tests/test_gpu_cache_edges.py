"""GPU tests of the paged cache beyond the usual cases: places beyond 2^24, far caps, outputs over inputs, many heads and samples,
shared pages, infinities, and a decoding loop inside a graph."""
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


def _i(a, dev):
    return torch.as_tensor(np.asarray(a, np.int32), device=dev)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [1, 5, 30])
@pytest.mark.parametrize("cap", [30.0, 1e6, 1e12])
def test_far_caps(dev, exp_mode, D, rows, cap):
    """As test_far_caps_in_exp_mode of the masked forward, in each row tile of the tile kernel and, with 30 rows a sample, in the
    prefix kernel."""
    Z, H, Hk, page, prefix = 3, 4, 2, 16, 100
    own = np.asarray([rows, 90, 61])
    nq = np.minimum(own, rows)
    g = torch.Generator().manual_seed(D + rows)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(dev)      # noqa: E731
    table = np.arange(18).reshape(3, 6)
    pre = np.arange(18, 25)
    kp, vp, q = r(25, page, Hk, D) * 2, r(25, page, Hk, D), r(Z, rows, H, D) * 2
    alpha, bias = D ** -0.5, -3.0
    o = sa.fwd_paged(q, kp, vp, _i(table, dev), _i(own, dev), _i(nq, dev), alpha, bias, cap=cap, prefix_table=_i(pre, dev),
                     prefix_len=_i([prefix], dev)).cpu().double()
    kc, vc, qc = (t.cpu().double() for t in (kp, vp, q))
    for z in range(Z):
        m, n = int(nq[z]), int(own[z])
        k = torch.cat([kc[pre].flatten(0, 1)[:prefix], kc[table[z]].flatten(0, 1)[:n]]).repeat_interleave(H // Hk, 1).transpose(0, 1)
        v = torch.cat([vc[pre].flatten(0, 1)[:prefix], vc[table[z]].flatten(0, 1)[:n]]).repeat_interleave(H // Hk, 1).transpose(0, 1)
        i, j = prefix + n - m + torch.arange(m)[:, None], torch.arange(prefix + n)[None]
        P = torch.sigmoid(cap * torch.tanh(alpha * (qc[z, :m].transpose(0, 1) @ k.mT) / cap) + bias) * (j <= i)
        want = (P @ v).transpose(0, 1)
        bound = R.HALF_BF16 * want.abs() + (R.HALF_BF16 + 1.1e-3) * (P @ v.abs()).transpose(0, 1)
        off = (o[z, :m] - want).abs()
        assert (off <= bound).all(), f"sample {z}: {float((off / bound).max()):.3g} of the bound"


def test_append_refuses_lengths_over_lengths(dev):
    """lens_out may be cache_lens itself for single tokens; any other overlap with the lengths would be read after it is written."""
    Z, Hk, D, page = 4, 2, 64, 16
    kp = torch.zeros(8, page, Hk, D, dtype=torch.bfloat16, device=dev)
    vp, table = torch.zeros_like(kp), _i(np.arange(8).reshape(4, 2), dev)
    buf = _i(np.arange(3 * Z), dev)
    call = lambda L, have, add, out, **a: sa.cache_append(torch.zeros(Z, L, Hk, D, dtype=kp.dtype, device=dev),      # noqa: E731
                                                          torch.zeros(Z, L, Hk, D, dtype=kp.dtype, device=dev), kp, vp, table,
                                                          have, add, lens_out=out, **a)
    a, b, c = buf[:Z], buf[Z:2 * Z].fill_(1), buf[2 * Z:]
    for L, out in ((1, b), (2, a), (2, b), (1, buf[1:Z + 1]), (2, buf[Z - 1:2 * Z - 1])):
        with pytest.raises(ValueError, match="lens_out"):
            call(L, a, b, out)
    with pytest.raises(ValueError, match="lens_out"):
        call(1, a, b, c, prefix_len=c[1:2])
    call(1, a, b, c)
    assert c.tolist() == [1, 2, 3, 4]
    call(1, a, b, a)
    assert a.tolist() == [1, 2, 3, 4]
    call(2, a, b, c)
    assert c.tolist() == [2, 3, 4, 5]


def test_append_refuses_queries_half_over_themselves(dev):
    Z, L, H, D = 1, 4, 2, 64
    buf = torch.zeros(2 * Z * L * H * D, dtype=torch.bfloat16, device=dev)
    q, half = buf[:L * H * D].view(Z, L, H, D), buf[64:64 + L * H * D].view(Z, L, H, D)
    kp = torch.zeros(1, 16, H, D, dtype=torch.bfloat16, device=dev)
    k = torch.zeros_like(q)
    call = lambda **a: sa.cache_append(k, k, kp, kp.clone(), _i([[0]], dev), _i([0], dev), _i([L], dev), q=q, **a)      # noqa: E731
    with pytest.raises(ValueError, match="q_out"):
        call(q_out=half)
    call(q_out=q)


def test_too_many_empty_pages_are_refused_with_an_exception(dev):
    """A size that does not fit the library's int raises, from whatever place it is found in: 2^31 pages of no heads hold no byte."""
    pages = torch.empty(2 ** 31, 16, 0, 64, dtype=torch.bfloat16, device=dev)
    q = torch.empty(1, 1, 0, 64, dtype=torch.bfloat16, device=dev)
    one = _i([1], dev)
    with pytest.raises(ValueError, match="2\\^31"):
        sa.fwd_paged(q, pages, pages, _i([[0]], dev), one, one, 1.0, 0.0)
    with pytest.raises(ValueError, match="2\\^31"):
        sa.cache_append(q, q, pages, pages, _i([[0]], dev), one, one)


@pytest.mark.parametrize("where", ["own", "own, odd", "prefix, few rows", "prefix, many rows"])
def test_distances_beyond_two_to_the_24(dev, exp_mode, where):
    """Places that fp32 does not hold: distances to the nearest keys are exact all the same.  All pages of the long part are one page
    with zero keys, so that a key's weight is sigma(-distance); its values mark the place within the page, entry e every place that
    is e modulo 64.  Weights fall by e a place: those nearer than 64 decide each sum, and the rest is below e^-64 of them.
    Bounds: P within 1e-3 and 2^-8 of itself, and the result's rounding 2^-8 (tests/_span_ref.py)."""
    D, page, far = 64, 256, 2 ** 24 + (6 if where == "own, odd" else 5)
    H, L = (16, 8) if where == "prefix, many rows" else (1, 1)
    pages = -(-far // page)
    kp = torch.zeros(2, page, 1, D, dtype=torch.bfloat16, device=dev)
    vp = torch.zeros_like(kp)
    vp[0, torch.arange(page), 0, torch.arange(page) % D] = 1.0
    q = torch.zeros(1, L, H, D, dtype=torch.bfloat16, device=dev)
    slopes = torch.ones(H, device=dev)
    if where.startswith("own"):
        o = sa.fwd_paged(q, kp, vp, torch.zeros(1, pages, dtype=torch.int32, device=dev), _i([far], dev), _i([1], dev), 1.0, 0.0,
                         slopes=slopes)
    else:           # own tokens of zero values behind the prefix
        o = sa.fwd_paged(q, kp, vp, _i([[1]], dev), _i([L], dev), _i([L], dev), 1.0, 0.0, slopes=slopes,
                         prefix_table=torch.zeros(pages, dtype=torch.int32, device=dev), prefix_len=_i([far], dev))
    e = torch.arange(D)
    for l in range(L):
        last = far - 1                                           # the nearest key that is marked
        first = 0 if where.startswith("own") else l + 1                   # and its distance
        near = (last - e) % D                                    # of the nearest place that is e modulo 64, behind `last`
        want = torch.sigmoid(-(first + near).double())
        want = want + torch.sigmoid(-(first + near + 64).double())
        off = (o[0, l].double().cpu() - want).abs()
        assert (off <= (2.0 ** -7 + 1.1e-3) * want).all(), f"row {l}: {float((off / want).max()):.3g}"
