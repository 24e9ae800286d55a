"""GPU tests of the masked attention: exact counts under every mask, numeric parity with the definition in 64 bits (bounds
derived in tests/_span_ref.py), NaN in padding, gradients against differences, capture, streams and the mask builder."""
import math

import numpy as np
import pytest
import torch

from tests import _compare as C
from tests import _span_ref as R

pytestmark = pytest.mark.gpu

sa = pytest.importorskip("padding_aware_sigmoid_b200")

MASKS = ["none", "full", "causal", "prefix", "docs", "docs_causal", "window", "holes", "scatter"]


@pytest.fixture
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield torch.device("cuda", 0)
    assert sa.last_device_status() == 0


@pytest.fixture
def exp_mode():
    old = sa.get_sigmoid_mode()
    sa.set_sigmoid_mode(sa.SIGMOID_EXP)
    yield
    sa.set_sigmoid_mode(old)


def _lens(Z, L, seed):
    g = np.random.default_rng(seed)
    n = g.integers(0, L + 1, size=Z).astype(np.int32)
    n[0] = L
    return n


def _spans(mask, n, L, dev, seed=3):
    return None if mask == "none" else R.make_spans(mask, n, L, seed).to(dev)


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("shape", [(3, 1, 2, 2, 64), (2, 77, 2, 1, 64), (3, 128, 2, 2, 128), (2, 129, 4, 2, 128),
                                   (2, 300, 6, 2, 64), (3, 515, 4, 1, 128), (2, 1100, 2, 2, 64)])
def test_visible_pairs_are_counted_exactly(dev, mask, shape):
    """With all scores 0 sigma is exactly 1/2 and its derivative 1/4, so marked keys and queries are counted: every output is
    a small integer that bf16 holds, and one wrong pair shows."""
    Z, L, H, Hk, D = shape
    n = _lens(Z, L, L + H)
    spans = _spans(mask, n, L, dev)
    g = np.random.default_rng(L * 7 + H)
    share = min(1.0, 40 / L)
    mark = lambda heads: torch.as_tensor((g.random((Z, L, heads)) < share).astype(np.float32))     # noqa: E731
    mq, mk, mv, mo = mark(H), mark(Hk), mark(Hk), mark(H)
    t = lambda heads: torch.zeros(Z, L, heads, D)      # noqa: E731
    q, k, v, do = t(H), t(Hk), t(Hk), t(H)
    q[..., 0], k[..., 1] = mq, mk                # q . k = 0
    v[..., 2], do[..., 2] = 2.0, 1.0             # dP = 2, dS = 1/2
    v[..., 3], do[..., 4] = 2.0 * mv, 2.0 * mo
    dt = torch.bfloat16
    q, k, v, do = (x.to(dev, dt) for x in (q, k, v, do))
    seq = torch.as_tensor(n, device=dev)
    out = torch.full_like(q, float("nan"))
    o = sa.fwd_span(q, k, v, seq, 2.0, 0.0, spans=spans, out=out)
    dq, dk, dv = sa.bwd_span(q, k, v, do, seq, 2.0, 0.0, spans=spans, dq=torch.full_like(q, float("nan")),
                             dk=torch.full_like(k, float("nan")), dv=torch.full_like(v, float("nan")))
    m = R.visible(spans, n, L).double()
    G = H // Hk
    fold = lambda x: x.view(Z, Hk, G, L).sum(2)        # noqa: E731
    up = lambda x: x.permute(0, 2, 1).double()         # noqa: E731
    want_o = (m[:, None] @ up(mv).repeat_interleave(G, 1)[..., None])[..., 0].permute(0, 2, 1)
    assert torch.equal(o[..., 3].cpu().double(), want_o)
    want_q = (m[:, None] @ up(mk).repeat_interleave(G, 1)[..., None])[..., 0].permute(0, 2, 1)
    assert torch.equal(dq[..., 1].cpu().double(), want_q)
    want_k = fold((m.mT[:, None] @ up(mq)[..., None])[..., 0]).permute(0, 2, 1)
    assert torch.equal(dk[..., 0].cpu().double(), want_k)
    want_v = fold((m.mT[:, None] @ up(mo)[..., None])[..., 0]).permute(0, 2, 1)
    assert torch.equal(dv[..., 4].cpu().double(), want_v)
    for x in (o, dq, dk, dv):
        assert not x[..., 5:].any()


def _tensors(Z, L, H, Hk, D, dtype, dev, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda h, s: (torch.randn(Z, L, h, D, generator=g) * s).to(dtype).to(dev)      # noqa: E731
    return r(H, scale), r(Hk, scale), r(Hk, 1.0), r(H, 1.0)


CASES = [  # Z, L, H, Hk, D, mask, cap, slopes
    (2, 1, 2, 1, 128, "causal", 0.0, False),
    (2, 200, 2, 2, 64, "none", 30.0, False),
    (3, 257, 4, 2, 128, "causal", 20.0, True),
    (2, 385, 3, 1, 64, "prefix", 0.0, True),
    (2, 640, 2, 2, 128, "docs", 50.0, False),
    (2, 511, 4, 4, 64, "docs_causal", 30.0, True),
    (1, 900, 2, 1, 128, "window", 0.0, True),
    (2, 300, 6, 2, 64, "holes", 0.0, False),
    (2, 260, 2, 1, 128, "scatter", 30.0, True),
]


def _run_case(case, dev, dtype, tanh):
    Z, L, H, Hk, D, mask, cap, sl = case
    n = _lens(Z, L, L)
    q, k, v, do = _tensors(Z, L, H, Hk, D, dtype, dev, L + D, 2.0 if cap else 1.0)
    spans = _spans(mask, n, L, dev)
    slopes = torch.linspace(0.5, 0.01, H, device=dev) if sl else None
    bias = -math.log(L) / 2 + 0.25 * np.arange(Z)
    bz = torch.as_tensor(bias.astype(np.float32), device=dev)
    seq = torch.as_tensor(n, device=dev)
    alpha = D ** -0.5
    o = sa.fwd_span(q, k, v, seq, alpha, bz, spans=spans, cap=cap, slopes=slopes)
    grads = sa.bwd_span(q, k, v, do, seq, alpha, bz, spans=spans, cap=cap, slopes=slopes)
    sees = R.visible(spans, n, L)
    ref, bound = R.reference(q, k, v, do, sees, alpha, bias.astype(np.float32), cap, slopes, dtype == torch.float32)
    for name, x in zip(("O", "dQ", "dK", "dV"), (o, *grads)):
        if tanh:
            C.assert_close(x.float().cpu().numpy(), ref[name].numpy(), "bf16", name)
        else:
            R.assert_within(x, ref[name], bound[name], name)
        dead = ~(sees.any(-1) if name in ("O", "dQ") else sees.any(1))
        assert not x[dead.to(dev)].any(), f"{name}: rows that take no part are not zero"


@pytest.mark.parametrize("case", CASES)
def test_parity_exp(dev, exp_mode, case):
    _run_case(case, dev, torch.bfloat16, False)


@pytest.mark.parametrize("case", CASES[1:])
def test_parity_tanh(dev, case):
    _run_case(case, dev, torch.bfloat16, True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,bias", [(1.5, -1.0), (6.0, -9.5), (15.0, -9.5), (40.0, -9.5), (40.0, -2.0), (1e6, 0.5)])
def test_forms_of_capped_scores(dev, D, cap, bias):
    """Scores far below the cap, around it and far beyond, within the same rows, in sigma's left tail and outside it: every form
    of the hardware-tanh mode, and the steps between them."""
    Z, L, H, Hk = 1, 1300, 2, 1
    q, k, v, do = _tensors(Z, L, H, Hk, D, torch.bfloat16, dev, 77)
    # keys of one stretch score large, queries of one stretch small
    k[:, 300:420] *= 4.0
    q[:, 700:1000] *= 0.1
    seq = torch.as_tensor(np.asarray([1290], np.int32), device=dev)
    spans = _spans("causal", [1290], L, dev)
    alpha = D ** -0.5
    args = dict(spans=spans, cap=cap)
    sees = R.visible(spans, [1290], L)
    ref, _ = R.reference(q, k, v, do, sees, alpha, [bias], cap, None)
    got = (sa.fwd_span(q, k, v, seq, alpha, bias, **args), *sa.bwd_span(q, k, v, do, seq, alpha, bias, **args))
    for name, x in zip(("O", "dQ", "dK", "dV"), got):
        C.assert_close(x.float().cpu().numpy(), ref[name].numpy(), "bf16", f"{name} at cap {cap}")


@pytest.mark.parametrize("case", CASES)
def test_parity_fp32(dev, case):
    _run_case(case, dev, torch.float32, False)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
def test_nan_in_padding_never_reaches_a_result(dev, dtype, D):
    Z, L, H, Hk = 3, 400, 4, 2
    n = np.asarray([400, 131, 0], np.int32)
    q, k, v, do = _tensors(Z, L, H, Hk, D, dtype, dev, 5)
    seq = torch.as_tensor(n, device=dev)
    for mask in ("none", "causal", "docs"):
        spans = _spans(mask, n, L, dev)
        clean = (sa.fwd_span(q, k, v, seq, 0.1, -2.0, spans=spans), *sa.bwd_span(q, k, v, do, seq, 0.1, -2.0, spans=spans))
        bad = []
        for t in (q, k, v, do):
            b = t.clone()
            for z in range(Z):
                b[z, n[z]:] = float("nan")
                b[z, n[z]:, :, ::3] = float("inf")
            bad.append(b)
        dirty = (sa.fwd_span(*bad[:3], seq, 0.1, -2.0, spans=spans), *sa.bwd_span(*bad, seq, 0.1, -2.0, spans=spans))
        for a, b in zip(clean, dirty):
            assert torch.equal(a, b)


def test_equals_the_padding_only_call_without_terms(dev, exp_mode):
    """No spans, no cap, no slopes, the EXP form: the same operation as fwd / bwd, to the bit (in TANH mode the masked kernels
    take a more accurate form in sigma's left tail), in a batch that fills the device: a smaller one adds its sums up in
    another order, over the blocks that share a tile."""
    Z, L, H, D = 24, 700, 16, 128
    q, k, v, do = _tensors(Z, L, H, H, D, torch.bfloat16, dev, 9)
    seq = torch.as_tensor(np.asarray([700, 333] * (Z // 2), np.int32), device=dev)
    assert torch.equal(sa.fwd(q, k, v, seq, seq, 0.09, -6.0), sa.fwd_span(q, k, v, seq, 0.09, -6.0))
    for a, b in zip(sa.bwd(q, k, v, do, seq, seq, 0.09, -6.0), sa.bwd_span(q, k, v, do, seq, 0.09, -6.0)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cap,sl", [(0.0, False), (4.0, True)])
def test_gradients_against_differences(dev, cap, sl):
    """fp32 path: central differences of <O, dO> along random directions.  The step's second-order error is h^2 / 6 of a third
    derivative of order 1, the values' rounding n 2^-24 / h: both below 1e-3 of the directional derivative's scale at h = 1e-2."""
    Z, L, H, Hk, D = 1, 90, 2, 1, 64
    n = np.asarray([83], np.int32)
    q, k, v, do = _tensors(Z, L, H, Hk, D, torch.float32, dev, 21)
    spans = _spans("docs_causal", n, L, dev)
    slopes = torch.tensor([0.3, 0.05], device=dev) if sl else None
    seq = torch.as_tensor(n, device=dev)
    f = lambda a, b, c: float((sa.fwd_span(a, b, c, seq, 0.125, -1.0, spans=spans, cap=cap, slopes=slopes).double() *   # noqa: E731
                               do.double()).sum())
    grads = sa.bwd_span(q, k, v, do, seq, 0.125, -1.0, spans=spans, cap=cap, slopes=slopes)
    for at, grad in enumerate(grads):
        d = torch.randn(grad.shape, generator=torch.Generator().manual_seed(at)).to(dev)
        h = 1e-2
        up, down = [q, k, v], [q, k, v]
        up[at], down[at] = up[at] + h * d, down[at] - h * d
        got = (f(*up) - f(*down)) / (2 * h)
        want = float((grad.double() * d.double()).sum())
        scale = float((grad.double() * d.double()).norm())
        assert abs(got - want) <= 2e-3 * max(scale, abs(want)) + 1e-3


def test_capture_and_replay_with_new_inputs(dev):
    Z, L, H, Hk, D = 2, 500, 4, 2, 64
    q, k, v, do = _tensors(Z, L, H, Hk, D, torch.bfloat16, dev, 31)
    seq = torch.as_tensor(np.asarray([500, 260], np.int32), device=dev)
    spans = sa.mask_spans(seq, L, causal=True)
    slopes = torch.full((H,), 0.1, device=dev)
    ws = torch.empty(sa.bwd_span_workspace_bytes(Z, L, q.dtype), dtype=torch.uint8, device=dev)
    outs = [torch.empty_like(t) for t in (q, q, k, v)]

    def step():
        sa.mask_spans(seq, L, causal=True, out=spans)
        sa.fwd_span(q, k, v, seq, 0.125, -3.0, spans=spans, cap=10.0, slopes=slopes, out=outs[0])
        sa.bwd_span(q, k, v, do, seq, 0.125, -3.0, spans=spans, cap=10.0, slopes=slopes, dq=outs[1], dk=outs[2],
                    dv=outs[3], workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        for t, u in zip((q, k, v, do), _tensors(Z, L, H, Hk, D, torch.bfloat16, dev, seed)):
            t.copy_(u)
        seq.copy_(torch.as_tensor(np.asarray([77 * seed, 500 - seed], np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in outs]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, outs))


def test_two_streams_at_once_and_repeats_are_bitwise_equal(dev):
    Z, L, H, Hk, D = 3, 777, 6, 2, 128
    q, k, v, do = _tensors(Z, L, H, Hk, D, torch.bfloat16, dev, 41)
    seq = torch.as_tensor(np.asarray([777, 400, 129], np.int32), device=dev)
    spans = _spans("docs_causal", [777, 400, 129], L, dev)
    call = lambda: (sa.fwd_span(q, k, v, seq, 0.1, -4.0, spans=spans, cap=30.0),      # noqa: E731
                    *sa.bwd_span(q, k, v, do, seq, 0.1, -4.0, spans=spans, cap=30.0))
    want = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(call())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))


def test_lengths_out_of_range_are_clamped_and_flagged():
    dev = torch.device("cuda", 0)
    q, k, v, do = _tensors(2, 100, 2, 2, 64, torch.bfloat16, dev, 51)
    seq = torch.as_tensor(np.asarray([150, -3], np.int32), device=dev)
    sa.last_device_status()
    o = sa.fwd_span(q, k, v, seq, 0.1, -1.0)
    assert sa.last_device_status() == 8
    fine = torch.as_tensor(np.asarray([100, 0], np.int32), device=dev)
    assert torch.equal(o, sa.fwd_span(q, k, v, fine, 0.1, -1.0))
    sa.bwd_span(q, k, v, do, seq, 0.1, -1.0)
    assert sa.last_device_status() == 8


def _by_rule(n, L, causal, prefix, docs, window):
    out = np.zeros((len(n), L, 2), np.int32)
    for z, m in enumerate(n):
        for i in range(m):
            lo, hi = 0, m
            if docs is not None:
                lo = i
                while lo > 0 and docs[z][lo - 1] == docs[z][i]:
                    lo -= 1
                hi = i + 1
                while hi < m and docs[z][hi] == docs[z][i]:
                    hi += 1
            end, start = hi, lo
            if causal:
                hi = min(end, i + 1 if prefix is None else max(i + 1, start + max(0, int(prefix[z]))))
            if window:
                lo = max(lo, i - window + 1)
                if not causal:
                    hi = min(hi, i + window)
            out[z, i] = (lo, hi) if lo < hi else (0, 0)
    return out


@pytest.mark.parametrize("L", [1, 33, 1024, 1025, 2500])
def test_mask_spans(dev, L):
    g = np.random.default_rng(L)
    n = [L, max(0, L // 3), 0]
    seq = torch.as_tensor(np.asarray(n, np.int32), device=dev)
    docs = np.cumsum(g.random((3, L)) < 0.01, axis=1).astype(np.int32) % 2       # ids come back: runs count, not ids
    dd = torch.as_tensor(docs, device=dev)
    pre = np.asarray([L // 2, 5, 2 ** 31 - 1], np.int32)
    pd = torch.as_tensor(pre, device=dev)
    for causal, prefix, doc, window in [(False, None, None, 0), (True, None, None, 0), (True, pre, None, 0),
                                        (False, None, docs, 0), (True, None, docs, 0), (True, pre, docs, 0),
                                        (True, None, docs, 17), (False, None, None, 1), (False, None, docs, 40),
                                        (True, None, None, 2 ** 31 - 1)]:
        got = sa.mask_spans(seq, L, causal=causal, prefix=None if prefix is None else pd,
                            docs=None if doc is None else dd, window=window)
        assert np.array_equal(got.cpu().numpy(), _by_rule(n, L, causal, prefix, doc, min(window, L)))


@pytest.mark.parametrize("per_sample", [False, True])
def test_module_runs_the_masked_attention_with_its_gradients(dev, per_sample):
    """The autograd module's outputs and gradients are the calls' own, for strided inputs and a strided output gradient too."""
    Z, L, H, Hk, D = 2, 200, 6, 2, 64
    q, k, v, do = _tensors(Z, L, H, Hk, D, torch.bfloat16, dev, 61)
    seq = torch.as_tensor(np.asarray([200, 91], np.int32), device=dev)
    spans = sa.mask_spans(seq, L, causal=True)
    slopes = torch.linspace(0.4, 0.01, H)
    attn = sa.SigmoidAttention(per_sample_bias=per_sample, bias=None if per_sample else -3.0, cap=25.0, slopes=slopes)
    leaves = [t.transpose(1, 2).contiguous().requires_grad_() for t in (q, k, v)]
    out = attn(*(t.transpose(1, 2) for t in leaves), seq, spans=spans)
    out.backward(do.transpose(1, 2).contiguous().transpose(1, 2))
    bias = sa.log_length_bias(seq) if per_sample else -3.0
    args = dict(spans=spans, cap=25.0, slopes=slopes.to(dev))
    assert torch.equal(out, sa.fwd_span(q, k, v, seq, D ** -0.5, bias, **args))
    for leaf, want in zip(leaves, sa.bwd_span(q, k, v, do, seq, D ** -0.5, bias, **args)):
        assert torch.equal(leaf.grad.transpose(1, 2), want)


def test_module_shares_key_heads_without_a_mask(dev):
    Z, L, H, Hk, D = 2, 130, 4, 1, 128
    q, k, v, do = _tensors(Z, L, H, Hk, D, torch.bfloat16, dev, 62)
    seq = torch.as_tensor(np.asarray([130, 7], np.int32), device=dev)
    out = sa.SigmoidAttention(bias=-2.0)(q, k, v, seq)
    assert torch.equal(out, sa.fwd_span(q, k, v, seq, D ** -0.5, -2.0))


def test_calls_refuse_what_does_not_fit(dev):
    Z, L, H, Hk, D = 2, 40, 4, 2, 64
    q, k, v, do = _tensors(Z, L, H, Hk, D, torch.bfloat16, dev, 63)
    seq = torch.as_tensor(np.asarray([40, 7], np.int32), device=dev)
    ok = lambda **a: sa.fwd_span(a.pop("q", q), a.pop("k", k), a.pop("v", v), a.pop("n", seq), 0.1, a.pop("b", 0.0), **a)  # noqa: E731
    ok()
    bad = [dict(q=q.float()), dict(k=k[:, :20]), dict(v=v[..., :32]), dict(q=q.transpose(1, 2)), dict(k=k.cpu()),
           dict(n=seq.long()), dict(n=seq[:1]), dict(spans=torch.zeros(Z, L, 2, device=dev)),
           dict(spans=torch.zeros(Z, L, 1, dtype=torch.int32, device=dev)), dict(slopes=torch.zeros(H - 1, device=dev)),
           dict(slopes=torch.zeros(H, device=dev, dtype=torch.float64)), dict(b=torch.zeros(Z + 1, device=dev)),
           dict(out=torch.empty_like(q).float()), dict(out=torch.empty_like(k)), dict(k=k[:, :, :1].expand(-1, -1, 3, -1).contiguous())]
    for args in bad:
        with pytest.raises(ValueError):
            ok(**args)
    with pytest.raises(TypeError):
        sa.fwd_span(q.half(), k.half(), v.half(), seq, 0.1, 0.0)
    for cap in (-1.0, float("nan"), float("inf")):
        with pytest.raises(sa.SigattnError):
            ok(cap=cap)
    with pytest.raises(sa.SigattnError):
        sa.bwd_span(q, k, v, do, seq, 0.1, 0.0, workspace=torch.empty(16, dtype=torch.uint8, device=dev))
    with pytest.raises(ValueError):
        sa.mask_spans(seq, L, prefix=seq, window=3)
    with pytest.raises(ValueError):
        sa.SigmoidAttention()(q, k, v, seq, seq.clone())
    assert sa.last_device_status() == 0


def test_long_rows_pass_the_tail_of_the_grid(dev):
    """More 128-row tiles than a grid's y and z sizes were chosen for, one head: the last rows count what they see."""
    Z, L, D = 1, 70000, 64
    n = np.asarray([L - 5], np.int32)
    seq = torch.as_tensor(n, device=dev)
    spans = sa.mask_spans(seq, L, causal=True, window=200)
    q = torch.zeros(Z, L, 1, D, device=dev, dtype=torch.bfloat16)
    v = torch.zeros_like(q)
    v[..., 0] = 2.0
    o = sa.fwd_span(q, q, v, seq, 1.0, 0.0, spans=spans)[0, :, 0, 0].float().cpu()
    want = torch.clamp(torch.arange(L) + 1, max=200).float()
    want[L - 5:] = 0
    assert torch.equal(o, want.to(torch.bfloat16).float())


def test_module_refuses_a_gradient_of_the_gradient(dev):
    q, k, v, do = _tensors(1, 64, 2, 2, 64, torch.bfloat16, dev, 71)
    seq = torch.as_tensor(np.asarray([50], np.int32), device=dev)
    q.requires_grad_()
    out = sa.SigmoidAttention(bias=-1.0, cap=5.0)(q, k, v, seq)
    dq, = torch.autograd.grad(out, q, do, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dq.float().sum(), q)


def test_captured_module_step_replays_with_new_inputs(dev):
    """Forward and backward of the module in one graph, warmed up on a side stream as PyTorch asks."""
    Z, L, H, Hk, D = 2, 300, 4, 2, 128
    q, k, v, do = _tensors(Z, L, H, Hk, D, torch.bfloat16, dev, 72)
    seq = torch.as_tensor(np.asarray([300, 140], np.int32), device=dev)
    spans = sa.mask_spans(seq, L, causal=True)
    attn = sa.SigmoidAttention(bias=-3.0, cap=20.0)
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]

    def step():
        out = attn(*leaves, seq, spans=spans)
        return (out.detach(), *torch.autograd.grad(out, leaves, do))

    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream(dev).wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (73, 74):
        new = _tensors(Z, L, H, Hk, D, torch.bfloat16, dev, seed)
        with torch.no_grad():
            for t, u in zip((*leaves, do), new):
                t.copy_(u)
        graph.replay()
        torch.cuda.synchronize()
        a = dict(spans=spans, cap=20.0)
        assert torch.equal(outs[0], sa.fwd_span(*new[:3], seq, D ** -0.5, -3.0, **a))
        for got, want in zip(outs[1:], sa.bwd_span(*new, seq, D ** -0.5, -3.0, **a)):
            assert torch.equal(got, want)


# few tiles with many steps: 2 or 4 blocks share each (span_split.cuh), some of them without a step of their own
SHARED = [(1, 2048, 2, 1, 128), (1, 2100, 2, 2, 64), (2, 1500, 2, 1, 64), (1, 1111, 6, 1, 128), (1, 4200, 3, 3, 128), (3, 1030, 2, 1, 64)]


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("shape", SHARED)
def test_blocks_that_share_a_tile_count_exactly(dev, mask, shape):
    test_visible_pairs_are_counted_exactly(dev, mask, shape)


@pytest.mark.parametrize("case", [(1, 1100, 2, 1, 64, "causal", 20.0, True), (1, 1200, 8, 1, 128, "window", 0.0, False),
                                  (1, 1025, 2, 2, 128, "prefix", 30.0, True), (1, 2060, 1, 1, 64, "docs_causal", 0.0, False)])
def test_parity_where_blocks_share_a_tile(dev, exp_mode, case):
    _run_case(case, dev, torch.bfloat16, False)


def test_shared_tiles_keep_nan_in_padding_out_and_repeat_to_the_bit(dev):
    Z, L, H, Hk, D = 2, 1400, 2, 1, 128
    n = np.asarray([1390, 700], np.int32)
    ts = _tensors(Z, L, H, Hk, D, torch.bfloat16, dev, 81)
    seq = torch.as_tensor(n, device=dev)
    spans = _spans("causal", n, L, dev)
    call = lambda q, k, v, do: (sa.fwd_span(q, k, v, seq, 0.1, -3.0, spans=spans, cap=20.0),      # noqa: E731
                                *sa.bwd_span(q, k, v, do, seq, 0.1, -3.0, spans=spans, cap=20.0))
    want = call(*ts)
    bad = [t.clone() for t in ts]
    for t in bad:
        for z in range(Z):
            t[z, n[z]:] = float("nan")
    for _ in range(3):
        for a, b in zip(want, call(*bad)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap,bias,sl", [(0.0, -9.5, False), (20.0, -9.5, False), (20.0, -2.0, False), (20.0, -9.5, True)])
def test_other_documents_and_padding_do_not_change_a_bit(dev, D, cap, bias, sl):
    """Documents of 100 to 700 tokens: what one of them yields stays the same, to the bit, whatever the others and the padding
    hold (large scores there choose other forms of the score function for their own chunks only)."""
    Z, L, H, Hk = 2, 1500, 4, 2
    n = np.asarray([1490, 1203], np.int32)
    ids = np.zeros((Z, L), np.int32)
    for z in range(Z):
        for edge in (100, 260, 900, 1150, 1300):
            ids[z, edge + 7 * z:] += 1
    seq = torch.as_tensor(n, device=dev)
    docs = torch.as_tensor(ids, device=dev)
    slopes = torch.linspace(0.1, 0.001, H, device=dev) if sl else None
    ts = _tensors(Z, L, H, Hk, D, torch.bfloat16, dev, 91)
    keep = (docs == 2) & (torch.arange(L, device=dev)[None] < seq[:, None])
    for causal in (False, True):
        spans = sa.mask_spans(seq, L, causal=causal, docs=docs)
        a = dict(spans=spans, cap=cap, slopes=slopes)
        call = lambda q, k, v, do: (sa.fwd_span(q, k, v, seq, D ** -0.5, bias, **a),      # noqa: E731
                                    *sa.bwd_span(q, k, v, do, seq, D ** -0.5, bias, **a))
        want = call(*ts)
        other = [torch.where(keep[..., None, None], t, u * 30)
                 for t, u in zip(ts, _tensors(Z, L, H, Hk, D, torch.bfloat16, dev, 92))]
        pad = torch.arange(L, device=dev)[None] >= seq[:, None]
        other = [t.masked_fill(pad[..., None, None], float("nan")) for t in other]
        for x, y in zip(want, call(*other)):
            assert torch.equal(x[keep], y[keep])
