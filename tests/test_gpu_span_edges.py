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


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 40.0])
def test_the_tail_gradient_has_the_bias_it_states(dev, D, cap):
    """Rows long enough for sigma's tail form, every score at x = -3.5, where u = e^x = 0.0302: sigma' is formed with a relative
    error of -u^2 and no more.  What else moves an output averages out: roundings of dS and of the result, each within 2^-8 with
    mean 0, over more than 10^5 of them leave less than 1e-4.  A cap adds the hardware tanh's error: 2^-11 of the capped score
    of 5 (2.5e-3 of sigma), and twice that, of 1 - tanh^2 = 0.984, 1e-5."""
    Z, L, H = 1, 2048, 2
    g = torch.Generator().manual_seed(D)
    x = -3.5
    y = 5.0 if not cap else cap * math.atanh(5.0 / cap)          # the product that the cap takes to 5
    f = 1.0 if not cap else 1.0 - (5.0 / cap) ** 2
    alpha, bias = y / 5.0, -8.5
    u = math.exp(x)
    slope = u / (1 + u) ** 2 * f
    pos = lambda: (0.5 + 0.5 * torch.rand(Z, L, H, D, generator=g)).to(torch.bfloat16).to(dev)      # noqa: E731
    for side in ("dQ", "dK"):
        a, b = pos(), pos()
        one, other = torch.zeros_like(a), pos()                # their product is 2.5 * 2.0 whatever `other` holds
        one[..., 0], other[..., 0] = 2.5, 2.0
        q, k = (one, other) if side == "dQ" else (other, one)
        grads = sa.bwd_span(q, k, a, b, _seq([L], dev), alpha, bias, cap=cap)
        got = grads[0 if side == "dQ" else 1][..., 1:].double()
        vt, dt, ot = (t.double().transpose(1, 2) for t in (a, b, other))
        dp = dt @ vt.mT                                         # [Z, H, query, key]
        want = alpha * slope * ((dp if side == "dQ" else dp.mT) @ ot)
        off = (got.transpose(1, 2) / want[..., 1:] - 1.0).mean()
        assert abs(float(off)) <= u * u + 1e-4 + (2.5e-3 if cap else 0.0), f"{side}: off by {float(off):.2e} on average"


@pytest.mark.parametrize("cast", ["bfloat16", "half", "double", "to"])
def test_a_cast_module_keeps_its_slopes(dev, cast):
    """A module inside a model that is converted to another type runs with the slopes it was given, to the bit."""
    Z, L, H, Hk, D = 2, 200, 6, 2, 64
    q, k, v, do = _tensors(Z, L, H, Hk, D, torch.bfloat16, dev, 61)
    slopes = torch.linspace(0.4, 0.01, H)
    model = torch.nn.ModuleDict({"attn": sa.SigmoidAttention(bias=-3.0, cap=25.0, slopes=slopes)})
    model = model.to(dev, torch.bfloat16) if cast == "to" else getattr(model, cast)().to(dev)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    out = model["attn"](*leaves, _seq([200, 91], dev))
    out.backward(do)
    args = dict(cap=25.0, slopes=slopes.to(dev))
    assert torch.equal(out, sa.fwd_span(q, k, v, _seq([200, 91], dev), D ** -0.5, -3.0, **args))
    for leaf, want in zip(leaves, sa.bwd_span(q, k, v, do, _seq([200, 91], dev), D ** -0.5, -3.0, **args)):
        assert torch.equal(leaf.grad, want)


# lengths that end inside a warp's 32 rows and inside its octets of columns' work: the lanes of a block that shares a tile part there
@pytest.mark.parametrize("L", [1026, 1039, 1057, 1151])
@pytest.mark.parametrize("D", [64, 128])
def test_ragged_tiles_that_blocks_share(dev, exp_mode, D, L):
    """Z = 1, few heads: the blocks of a cluster add their sums (span_split.cuh), rows beyond L left out lane by lane."""
    H, Hk = 2, 1
    q, k, v, do = _tensors(1, L, H, Hk, D, torch.bfloat16, dev, L)
    spans = R.make_spans("causal", [L], L).to(dev)
    # the outputs end where a guard begins
    guard = lambda t: torch.full((t.numel() + 512,), 7.0, dtype=t.dtype, device=dev)      # noqa: E731
    bufs = [guard(t) for t in (q, q, k, v)]
    o, dq, dk, dv = (b[:t.numel()].view_as(t) for b, t in zip(bufs, (q, q, k, v)))
    sa.fwd_span(q, k, v, _seq([L], dev), D ** -0.5, -3.0, spans=spans, out=o)
    sa.bwd_span(q, k, v, do, _seq([L], dev), D ** -0.5, -3.0, spans=spans, dq=dq, dk=dk, dv=dv)
    ref, bound = R.reference(q, k, v, do, R.visible(spans, [L], L), D ** -0.5, [-3.0], 0.0, None)
    for name, x, b in zip(("O", "dQ", "dK", "dV"), (o, dq, dk, dv), bufs):
        R.assert_within(x, ref[name], bound[name], name)
        assert (b[-512:] == 7.0).all()


def test_outputs_over_inputs_are_refused(dev):
    Z, L, H, Hk, D = 2, 40, 4, 2, 64
    q, k, v, do = _tensors(Z, L, H, Hk, D, torch.bfloat16, dev, 63)
    seq = _seq([40, 7], dev)
    both = torch.empty(2, Z, L, H, D, dtype=q.dtype, device=dev)
    shifted = both.flatten()[64:64 + q.numel()].view_as(q)
    with pytest.raises(ValueError, match="overlap"):
        sa.fwd_span(q, k, v, seq, 0.1, 0.0, out=q)
    with pytest.raises(ValueError, match="overlap"):
        sa.fwd_span(both[0], k, v, seq, 0.1, 0.0, out=shifted)
    for outs in (dict(dq=q), dict(dq=do), dict(dk=k), dict(dk=v), dict(dv=v), dict(dk=(t := torch.empty_like(k)), dv=t)):
        with pytest.raises(ValueError, match="overlap"):
            sa.bwd_span(q, k, v, do, seq, 0.1, 0.0, **outs)
    sa.fwd_span(both[0].zero_(), k, v, seq, 0.1, 0.0, out=both[1])       # side by side is fine
    sa.bwd_span(q, k, k, q, seq, 0.1, 0.0)                               # so is an input given twice


def test_windows_beyond_32_bits_hide_nothing(dev):
    seq = _seq([40, 7], dev)
    docs = (torch.arange(50, device=dev, dtype=torch.int32) // 9).expand(2, 50).contiguous()
    for causal in (False, True):
        want = sa.mask_spans(seq, 50, causal=causal, docs=docs)
        for window in (50, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 40 + 1):
            assert torch.equal(sa.mask_spans(seq, 50, causal=causal, docs=docs, window=window), want)
    for window in (-1, -2 ** 31, -2 ** 32 + 3):
        with pytest.raises(sa.SigattnError):
            sa.mask_spans(seq, 50, window=window)


@pytest.mark.parametrize("cap,bias", [(0.0, -9.5), (20.0, -9.5), (20.0, -2.0)])
@pytest.mark.parametrize("D", [64, 128])
def test_later_queries_of_the_same_warp(dev, D, cap, bias):
    """Causal rows, the queries of rows 480 ... 511 behind row 490 made large.  What rows up to 490 yield does not depend on them to
    the bit in EXP mode; in TANH mode, which chooses a chunk's form for 32 rows at once, it stays within the bar of that mode."""
    Z, L, H = 1, 600, 2
    q, k, v, do = _tensors(Z, L, H, H, D, torch.bfloat16, dev, 15)
    seq = _seq([L], dev)
    spans = sa.mask_spans(seq, L, causal=True)
    large = q.clone()
    large[:, 491:512] *= 60.0
    call = lambda x: (sa.fwd_span(x, k, v, seq, D ** -0.5, bias, spans=spans, cap=cap),      # noqa: E731
                      sa.bwd_span(x, k, v, do, seq, D ** -0.5, bias, spans=spans, cap=cap)[0])
    ref, _ = R.reference(q, k, v, do, R.visible(spans, [L], L), D ** -0.5, [bias], cap, None)
    for got, name in zip(call(large), ("O", "dQ")):
        C.assert_close(got[:, :491].float().cpu().numpy(), ref[name][:, :491].numpy(), "bf16", name)
    old = sa.get_sigmoid_mode()
    try:
        sa.set_sigmoid_mode(sa.SIGMOID_EXP)
        for a, b in zip(call(q), call(large)):
            assert torch.equal(a[:, :491], b[:, :491])
            assert torch.equal(a[:, 512:], b[:, 512:])
    finally:
        sa.set_sigmoid_mode(old)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", [(3, 700, 8), (1, 1300, 2)])       # blocks of their own, and blocks that share tiles
def test_calls_in_a_row_on_one_workspace(dev, D, shape):
    """The backward's kernels overlap and hand tables over in the workspace: calls of unlike masks and lengths, one after the other
    on one workspace without a wait between them, equal the same calls alone."""
    Z, L, H = shape
    q, k, v, do = _tensors(Z, L, H, H, D, torch.bfloat16, dev, 45)
    kinds = []
    for mask, n in (("causal", [L] * Z), ("docs", [L // 2] * Z), ("window", [L - 1] * Z), ("scatter", [L] * Z), ("holes", [130] * Z)):
        kinds.append((R.make_spans(mask, n, L).to(dev), _seq(n, dev)))
    call = lambda s, n, **a: sa.bwd_span(q, k, v, do, n, 0.1, -3.0, spans=s, **a)      # noqa: E731
    want = []
    for s, n in kinds:
        want.append(call(s, n))
        torch.cuda.synchronize()
    ws = torch.empty(sa.bwd_span_workspace_bytes(Z, L, q.dtype), dtype=torch.uint8, device=dev)
    got = [(at, call(*kinds[at], workspace=ws)) for at in [0, 1, 2, 3, 4, 2, 0, 4, 1, 3] * 4]
    for at, outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, want[at]))


@pytest.mark.parametrize("mode", ["SIGMOID_TANH", "SIGMOID_EXP"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cap,sl,bias", [(0.0, False, -9.5), (0.0, False, -1.0), (20.0, False, -9.5), (20.0, True, -1.0)])
def test_infinities_and_nan_in_live_rows(dev, dtype, mode, cap, sl, bias):
    """A live key of infinite entries: sigma is 1 or 0 by the sign of the score, and O stays finite.  A query of NaN makes its own
    row NaN and no other."""
    Z, L, H, D = 1, 300, 2, 64
    q, k, v, _ = _tensors(Z, L, H, H, D, dtype, dev, 25)
    k[:, 100, :, 0], k[:, 207, :, 1] = float("inf"), float("-inf")
    slopes = torch.tensor([0.02, 0.001], device=dev) if sl else None
    seq = _seq([290], dev)
    alpha = D ** -0.5
    old = sa.get_sigmoid_mode()
    try:
        sa.set_sigmoid_mode(getattr(sa, mode))
        o = sa.fwd_span(q, k, v, seq, alpha, bias, cap=cap, slopes=slopes)
        bad = q.clone()
        bad[:, 77] = float("nan")
        ob = sa.fwd_span(bad, k, v, seq, alpha, bias, cap=cap, slopes=slopes)
    finally:
        sa.set_sigmoid_mode(old)
    ref, _ = R.reference(q, k, v, None, R.visible(None, [290], L), alpha, [bias], cap, slopes)
    kind = "fp32" if dtype == torch.float32 else "bf16"
    assert torch.isfinite(o).all()
    C.assert_close(o.float().cpu().numpy(), ref["O"].numpy(), kind, "O")
    assert torch.isnan(ob[:, 77]).all()
    others = torch.arange(L, device=dev) != 77
    C.assert_close(ob[:, others].float().cpu().numpy(), ref["O"][:, others.cpu()].numpy(), kind, "O beside a row of NaN")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_short_samples(dev, exp_mode, dtype):
    """More samples than are ranked by length, of 0 to 10 tokens."""
    Z, L, H, Hk, D = 200, 10, 4, 2, 64
    n = np.arange(Z) % 11
    q, k, v, do = _tensors(Z, L, H, Hk, D, dtype, dev, 35)
    spans = sa.mask_spans(_seq(n, dev), L, causal=True)
    bias = [-1.0] * Z
    got = (sa.fwd_span(q, k, v, _seq(n, dev), 0.125, -1.0, spans=spans), *sa.bwd_span(q, k, v, do, _seq(n, dev), 0.125, -1.0, spans=spans))
    ref, bound = R.reference(q, k, v, do, R.visible(spans, n, L), 0.125, bias, 0.0, None, dtype == torch.float32)
    for name, x in zip(("O", "dQ", "dK", "dV"), got):
        R.assert_within(x, ref[name], bound[name], name)


def test_caps_that_round_to_nothing_are_refused(dev):
    q, k, v, do = _tensors(1, 20, 2, 2, 64, torch.bfloat16, dev, 2)
    for cap in (1e-46, 1e-300):
        with pytest.raises(ValueError, match="cap"):
            sa.fwd_span(q, k, v, _seq([20], dev), 1.0, 0.0, cap=cap)
        with pytest.raises(ValueError, match="cap"):
            sa.bwd_span(q, k, v, do, _seq([20], dev), 1.0, 0.0, cap=cap)


@pytest.mark.parametrize("D", [64, 128])
def test_tensors_beyond_two_to_the_31_entries(dev, D):
    """Queries of more than 2^31 entries, their heads sharing one key head: with all scores 0 sigma is 1/2 and its derivative 1/4, and
    marked rows are counted (tests/test_gpu_span.py), the last samples' as the first's."""
    L, H = 2048, 128
    Z = 2 ** 31 // (L * H * D) + 2
    window = 40
    n = np.full(Z, L)
    n[-1] = L - 77
    seq = _seq(n, dev)
    spans = sa.mask_spans(seq, L, causal=True, window=window)
    q = torch.zeros(Z, L, H, D, dtype=torch.bfloat16, device=dev)
    assert q.numel() > 2 ** 31
    k, v = (torch.zeros(Z, L, 1, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    mark = (torch.arange(L, device=dev) % 5 == 0).to(q.dtype)
    q[..., 0] = (torch.arange(H, device=dev) % 64 == 3).to(q.dtype)
    k[..., 1] = mark[None, :, None]
    v[..., 2], v[..., 3] = 2.0, 2.0 * mark[None, :, None]
    do = torch.zeros_like(q)
    do[..., 2] = 1.0                                             # dP = 2, dS = 1/2
    do[..., 4] = q[..., 0] * 2.0
    o = sa.fwd_span(q, k, v, seq, 2.0, 0.0, spans=spans)
    dq, dk, dv = sa.bwd_span(q, k, v, do, seq, 2.0, 0.0, spans=spans)
    i = torch.arange(L, device=dev)
    for z in (0, 1, Z - 2, Z - 1):
        sees = ((i[None] <= i[:, None]) & (i[None] > i[:, None] - window) & (i[:, None] < int(n[z]))).float()
        rows, keys = sees @ mark.float(), sees.sum(0)
        for x, e in ((o, 3), (dq, 1)):
            assert torch.equal(x[z, :, :, e].float(), rows[:, None].expand(L, H))
            assert not x[z, :, :, 5:].any()
        assert torch.equal(dv[z, :, 0, 4].float(), 2.0 * keys)   # two marked heads
        assert torch.equal(dk[z, :, 0, 0].float(), 2.0 * keys)
        assert not dk[z, :, 0, 5:].any() and not dv[z, :, 0, 5:].any()


@pytest.mark.parametrize("mode", ["SIGMOID_TANH", "SIGMOID_EXP"])
@pytest.mark.parametrize("D", [64, 128])
def test_caps_on_both_sides_of_far(dev, D, mode):
    """A cap of 64 and the next fp32 above it, which the accurate form evaluates otherwise, with slopes and without, alone in a tile
    and shared: both within the bounds of their mode, and next to each other."""
    old = sa.get_sigmoid_mode()
    caps = (64.0, float(np.nextafter(np.float32(64.0), np.float32(65.0))))
    for (Z, L, H), sl in (((2, 260, 2), False), ((1, 1100, 2), True)):
        q, k, v, do = _tensors(Z, L, H, H, D, torch.bfloat16, dev, 5, 2.0)
        n = [L - 3] * Z
        spans = R.make_spans("causal", n, L).to(dev)
        slopes = torch.tensor([0.05, 0.001], device=dev) if sl else None
        ref, bound = R.reference(q, k, v, do, R.visible(spans, n, L), D ** -0.5, [-3.0] * Z, 64.0, slopes)
        for cap in caps:
            a = dict(spans=spans, cap=cap, slopes=slopes)
            try:
                sa.set_sigmoid_mode(getattr(sa, mode))
                got = (sa.fwd_span(q, k, v, _seq(n, dev), D ** -0.5, -3.0, **a), *sa.bwd_span(q, k, v, do, _seq(n, dev), D ** -0.5, -3.0, **a))
            finally:
                sa.set_sigmoid_mode(old)
            for name, x in zip(("O", "dQ", "dK", "dV"), got):
                if mode == "SIGMOID_EXP":
                    R.assert_within(x, ref[name], bound[name], name)
                else:
                    C.assert_close(x.float().cpu().numpy(), ref[name].numpy(), "bf16", name)
