"""GPU tests of the paged cache: appending with the rotation on the way, attention against it with a shared prefix, both
against their definitions in 64 bits, and a whole run from training form to decoding.

Bounds of fwd_paged: those of the masked forward in tests/_span_ref.py (P rounded to bf16 before its second product, sums of
partials in fp32, one rounding at the end).  Bounds of cache_append: a rotated entry is a cos - b sin in fp32 from angles of
64 bits, sincosf being within 2 ulp: 4 * 2^-23 (|a| + |b|), and the rounding to bf16, 2^-8 of the result."""
import math

import numpy as np
import pytest
import torch

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


def _pages(lens, page, spare=2, seed=0):
    """(page_table [Z, most], pages): a shuffled pool with a row of -1 behind each sample's pages."""
    g = np.random.default_rng(seed)
    need = [-(-int(n) // page) for n in lens]
    pool = g.permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(lens), max(1, max(need, default=0))), -1, np.int32)
    at = 0
    for z, m in enumerate(need):
        table[z, :m] = pool[at:at + m]
        at += m
    return table, len(pool)


def _i(a, dev):
    return torch.as_tensor(np.asarray(a, np.int32), device=dev)


def _turned(x, pos, inv_freq, interleaved):
    """64-bit rotation of [tokens, heads, D] and the bound's sum |a| + |b| per entry."""
    x = x.detach().cpu().double().clone()
    f = inv_freq.cpu().double()
    rot = 2 * len(f)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    w = torch.as_tensor(pos).double()[:, None] * f
    c, s = torch.cos(w)[:, None], torch.sin(w)[:, None]
    size = torch.zeros_like(x)
    size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    x0, x1 = x[..., a].clone(), x[..., b].clone()
    x[..., a], x[..., b] = x0 * c - x1 * s, x1 * c + x0 * s
    return x, size


APPENDS = [  # Z, L, H, Hk, D, page, rot, interleaved, prefix, dtype
    (1, 1, 2, 1, 64, 16, 64, False, 0, torch.bfloat16),
    (5, 1, 16, 4, 128, 64, 128, False, 70000, torch.bfloat16),
    (3, 77, 4, 2, 128, 16, 64, True, 5, torch.bfloat16),
    (2, 130, 12, 12, 64, 32, 16, False, 0, torch.bfloat16),
    (4, 33, 3, 3, 64, 128, 32, True, 1000003, torch.float32),
    (9, 500, 2, 2, 128, 256, 128, False, 1, torch.float32),
    (3, 50, 0, 2, 64, 16, 0, False, 0, torch.bfloat16),       # no queries, no rotation
]


@pytest.mark.parametrize("case", APPENDS)
def test_append(dev, case):
    Z, L, H, Hk, D, page, rot, inter, prefix, dt = case
    g = np.random.default_rng(L)
    have = g.integers(0, 200, size=Z)
    add = g.integers(0, L + 1, size=Z)
    add[0] = L
    if Z > 1:
        add[1], have[-1] = 0, 0
    table, count = _pages(have + add, page)
    gen = torch.Generator().manual_seed(L)
    r = lambda *s: torch.randn(*s, generator=gen).to(dt).to(dev)      # noqa: E731
    k, v = r(Z, L, Hk, D), r(Z, L, Hk, D)
    q = r(Z, L, H, D) if H else None
    kp, vp = r(count, page, Hk, D), r(count, page, Hk, D)
    kp[0, 0] = float("nan")              # whatever was there stays
    before = kp.clone(), vp.clone()
    inv = torch.as_tensor(10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2)), dtype=torch.float32, device=dev) if rot else None
    out, lens = sa.cache_append(k, v, kp, vp, _i(table, dev), _i(have, dev), _i(add, dev), inv_freq=inv, interleaved=inter, q=q,
                                prefix_len=_i([prefix], dev) if prefix else None,
                                q_out=torch.full_like(q, float("nan")) if H else None)
    assert lens.cpu().tolist() == (have + add).tolist()
    touched = torch.zeros(count, page, dtype=torch.bool)
    half = 2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -24
    for z in range(Z):
        m = int(add[z])
        at = np.arange(have[z], have[z] + m)
        pg, slot = table[z][at // page], at % page
        touched[pg, slot] = True
        assert torch.equal(vp[pg, slot], v[z, :m])
        for got, src in ((kp[pg, slot], k[z, :m]), (out[z, :m] if H else None, q[z, :m] if H else None)):
            if src is None:
                continue
            if not rot:
                assert torch.equal(got, src)
                continue
            want, size = _turned(src, prefix + at, inv, inter)
            off = (got.cpu().double() - want).abs()
            assert (off <= half * want.abs() + 4 * 2.0 ** -23 * size).all()
            assert torch.equal(got[..., rot:], src[..., rot:])
        if H:
            assert not out[z, m:].any()
    same = ~touched.to(dev)
    for now, was in ((kp, before[0]), (vp, before[1])):
        assert torch.equal(now[same].view(torch.uint8), was[same].view(torch.uint8))


def test_append_in_place_queries_and_lengths(dev):
    Z, H, Hk, D, page = 6, 4, 2, 64, 16
    have = np.asarray([0, 15, 16, 31, 47, 5])
    table, count = _pages(have + 3, page)
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(dev)      # noqa: E731
    kp, vp = r(count, page, Hk, D), r(count, page, Hk, D)
    kp2, vp2 = kp.clone(), vp.clone()
    inv = torch.logspace(0, -3, 32, device=dev)
    lens, lens2, one = _i(have, dev), _i(have, dev), _i([1] * Z, dev)
    for _ in range(3):
        k, v, q = r(Z, 1, Hk, D), r(Z, 1, Hk, D), r(Z, 1, H, D)
        q2 = q.clone()
        want, lens2 = sa.cache_append(k, v, kp2, vp2, _i(table, dev), lens2, one, inv_freq=inv, q=q2)
        sa.cache_append(k, v, kp, vp, _i(table, dev), lens, one, inv_freq=inv, q=q, q_out=q, lens_out=lens)
        assert torch.equal(q, want) and torch.equal(lens, lens2)
    assert torch.equal(kp, kp2) and torch.equal(vp, vp2) and lens.cpu().tolist() == (have + 3).tolist()


def test_append_flags_what_it_does_not_write():
    dev = torch.device("cuda", 0)
    Z, L, Hk, D, page = 3, 20, 2, 64, 16
    table = np.asarray([[0, 1], [2, 99], [-5, 3]], np.int32)
    k = torch.randn(Z, L, Hk, D, device=dev).to(torch.bfloat16)
    kp = torch.zeros(5, page, Hk, D, dtype=torch.bfloat16, device=dev)
    vp = torch.zeros_like(kp)
    sa.last_device_status()
    _, lens = sa.cache_append(k, k, kp, vp, _i(table, dev), _i([0, 0, 0], dev), _i([20, 20, 20], dev))
    assert sa.last_device_status() == 10
    assert lens.cpu().tolist() == [20, 20, 20]
    assert torch.equal(kp[0], k[0, :16]) and torch.equal(kp[1, :4], k[0, 16:]) and torch.equal(kp[2], k[1, :16])
    assert torch.equal(kp[3, :4], k[2, 16:]) and not kp[4].any() and not kp[1, 4:].any()
    # more than the table holds: clamped, flagged, the rest written
    kp.zero_()
    _, lens = sa.cache_append(k, k, kp, vp, _i(table, dev), _i([25, -4, 32], dev), _i([20, 5, 0], dev))
    assert sa.last_device_status() == 8
    assert lens.cpu().tolist() == [32, 5, 32]
    assert torch.equal(kp[1, 9:], k[0, :7]) and torch.equal(kp[2, :5], k[1, :5]) and not kp[2, 5:].any()


PAGED = [  # Z, L, H, Hk, D, page, prefix, own lengths, cap, slopes
    (1, 1, 2, 2, 64, 16, 0, [1], 0.0, False),
    (2, 1, 4, 1, 128, 16, 1, [1, 0], 0.0, True),
    (3, 1, 16, 2, 128, 64, 300, [64, 65, 1], 30.0, True),
    (4, 5, 12, 4, 64, 32, 129, [5, 200, 64, 63], 20.0, False),
    (2, 8, 8, 1, 64, 128, 0, [1000, 333], 0.0, True),              # 64 rows a sample
    (3, 20, 6, 2, 128, 256, 64, [20, 700, 90], 0.0, False),         # 60 rows a sample
    (2, 50, 4, 1, 128, 16, 77, [50, 130], 30.0, True),              # 200 rows: several row tiles
    (70, 1, 2, 1, 64, 16, 500, [17 * (i % 9) + 1 for i in range(70)], 0.0, False),
    (130, 2, 4, 2, 128, 16, 40, [2 + i % 50 for i in range(130)], 0.0, True),   # more samples than threads
]


def _paged_inputs(case, dt, dev, seed=0):
    Z, L, H, Hk, D, page, prefix, own, cap, sl = case
    g = np.random.default_rng(seed)
    own = np.asarray(own)
    nq = np.minimum(g.integers(0, L + 1, size=Z), own)
    nq[0] = min(L, own[0])
    table, count = _pages(own, page, spare=2 + -(-prefix // page), seed=seed)
    pre = np.setdiff1d(np.arange(count), table[table >= 0])[:-(-prefix // page)].astype(np.int32)
    gen = torch.Generator().manual_seed(seed + L)
    r = lambda *s: torch.randn(*s, generator=gen).to(dt).to(dev)      # noqa: E731
    kp, vp = r(count, page, Hk, D), r(count, page, Hk, D)
    # places that no query sees hold NaN
    dead = torch.ones(count, page, dtype=torch.bool)
    for z in range(Z):
        at = np.arange(own[z] if nq[z] else 0)
        dead[table[z][at // page], at % page] = False
    at = np.arange(prefix)
    dead[pre[at // page] if prefix else [], at % page if prefix else []] = False
    kp[dead.to(dev)] = float("nan")
    vp[dead.to(dev)] = float("nan")
    q = r(Z, L, H, D) * (2.0 if cap else 1.0)
    for z in range(Z):
        q[z, nq[z]:] = float("nan")
    return q, kp, vp, table, own, nq, pre


def _paged_reference(case, q, kp, vp, table, own, nq, pre, alpha, bias, slopes, fp32):
    Z, L, H, Hk, D, page, prefix, _, cap, _ = case
    ref, bound = torch.zeros(Z, L, H, D, dtype=torch.float64), torch.zeros(Z, L, H, D, dtype=torch.float64)
    ep, eo = (2e-5, 2e-5) if fp32 else (R.HALF_BF16 + 1.1e-3, R.HALF_BF16)
    kp, vp, q = (t.cpu().double() for t in (kp, vp, q))
    for z in range(Z):
        m, n = int(nq[z]), int(own[z])
        if m == 0:
            continue
        at, pa = np.arange(n), np.arange(prefix)
        k = torch.cat([kp[pre[pa // page], pa % page] if prefix else kp[:0, 0], kp[table[z][at // page], at % page]])
        v = torch.cat([vp[pre[pa // page], pa % page] if prefix else vp[:0, 0], vp[table[z][at // page], at % page]])
        k, v = (t.repeat_interleave(H // Hk, 1).transpose(0, 1) for t in (k, v))      # [H, keys, D]
        y = alpha * (q[z, :m].transpose(0, 1) @ k.mT)
        if cap:
            y = cap * torch.tanh(y / cap)
        i, j = prefix + n - m + torch.arange(m)[:, None], torch.arange(prefix + n)[None]
        if slopes is not None:
            y = y - slopes.cpu().double()[:, None, None] * (i - j).abs()
        P = torch.sigmoid(y + float(bias[z])) * (j <= i)
        ref[z, :m] = (P @ v).transpose(0, 1)
        bound[z, :m] = eo * ref[z, :m].abs() + ep * (P @ v.abs()).transpose(0, 1)
    return ref, bound


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("case", PAGED)
def test_paged(dev, case, dt):
    Z, L, H, Hk, D, page, prefix, _, cap, sl = case
    old = sa.get_sigmoid_mode()
    q, kp, vp, table, own, nq, pre = _paged_inputs(case, dt, dev)
    slopes = torch.linspace(0.3, 0.001, H, device=dev) if sl else None
    bias = (-math.log(prefix + max(own)) / 2 + 0.1 * np.arange(Z) / Z).astype(np.float32)
    alpha = D ** -0.5
    more = dict(prefix_table=_i(pre, dev), prefix_len=_i([prefix], dev)) if prefix else {}
    call = lambda: sa.fwd_paged(q, kp, vp, _i(table, dev), _i(own, dev), _i(nq, dev), alpha,      # noqa: E731
                                torch.as_tensor(bias, device=dev), cap=cap, slopes=slopes,
                                out=torch.full_like(q, float("nan")), **more)
    ref, bound = _paged_reference(case, q, kp, vp, table, own, nq, pre, alpha, bias, slopes, dt == torch.float32)
    try:
        sa.set_sigmoid_mode(sa.SIGMOID_EXP)
        got = call()
    finally:
        sa.set_sigmoid_mode(old)
    R.assert_within(got, ref, bound, "O")
    for z in range(Z):
        assert not got[z, nq[z]:].any()
    a, b = call(), call()
    assert torch.equal(a, b)
    # the hardware-tanh form: the framework's bar for it, 5e-3 of the sum
    assert float((a.cpu().double() - ref).abs().sum()) <= 5e-3 * float(ref.abs().sum()) + 1e-30


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("prefix", [0, 100, 640, 2049])
@pytest.mark.parametrize("heads,page", [((4, 2), 16), ((12, 2), 32), ((12, 1), 64), ((24, 3), 128), ((130, 1), 256)])
def test_paged_counts_visible_keys_exactly(dev, D, prefix, heads, page):
    """q = 0 makes sigma 1/2 (within the 3.4e-4 of the polynomial, which P's rounding to bf16 takes away): marked values are
    counted, and one wrong place shows."""
    (H, Hk), Z, L = heads, 5, 3
    own, nq = np.asarray([3, 64, 130, 0, 511]), np.asarray([3, 1, 2, 0, 3])
    table, count = _pages(own, page, spare=1 + -(-prefix // page))
    pre = np.setdiff1d(np.arange(count), table[table >= 0])[:-(-prefix // page)].astype(np.int32)
    g = np.random.default_rng(D + prefix)
    mark = (g.random((count, page, Hk)) < min(0.1, 100 / (prefix + 511))).astype(np.float32)
    vp = torch.zeros(count, page, Hk, D)
    vp[..., 5] = torch.as_tensor(2 * mark)
    vp = vp.to(dev, torch.bfloat16)
    kp = torch.randn(count, page, Hk, D, device=dev).to(torch.bfloat16)
    q = torch.zeros(Z, L, H, D, device=dev, dtype=torch.bfloat16)
    more = dict(prefix_table=_i(pre, dev), prefix_len=_i([prefix], dev)) if prefix else {}
    o = sa.fwd_paged(q, kp, vp, _i(table, dev), _i(own, dev), _i(nq, dev), 1.0, 0.0, **more).cpu()
    pa = np.arange(prefix)
    ahead = mark[pre[pa // page], pa % page].sum(0) if prefix else np.zeros(Hk)
    for z in range(Z):
        for l in range(L):
            at = np.arange(own[z] - nq[z] + l + 1) if l < nq[z] else np.arange(0)
            want = (mark[table[z][at // page], at % page].sum(0) + ahead) if l < nq[z] else np.zeros(Hk)
            for h in range(H):
                assert float(o[z, l, h, 5]) == want[h * Hk // H]
    assert not o[..., :5].any() and not o[..., 6:].any()


def test_paged_replays_with_new_lengths_and_tables(dev):
    """Lengths, tables and the prefix's length are read on the device."""
    Z, L, H, Hk, D, page = 3, 2, 8, 2, 128, 16
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(dev)      # noqa: E731
    kp, vp, q = r(60, page, Hk, D), r(60, page, Hk, D), r(Z, L, H, D)
    table, pre = _i(np.arange(45).reshape(3, 15), dev), _i(np.arange(45, 60), dev)
    own, nq, plen = _i([200, 3, 100], dev), _i([2, 1, 2], dev), _i([240], dev)
    ws = torch.empty(sa.fwd_paged_workspace_bytes(Z, L, H, Hk, D, q.dtype), dtype=torch.uint8, device=dev)
    out = torch.empty_like(q)
    call = lambda o, w: sa.fwd_paged(q, kp, vp, table, own, nq, 0.09, -4.0, prefix_table=pre, prefix_len=plen,      # noqa: E731
                                     cap=20.0, out=o, workspace=w)
    call(out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws)
    for lens, news, ahead in (([240, 1, 0], [2, 1, 0], 0), ([7, 64, 129], [1, 2, 2], 65), ([1, 1, 1], [1, 1, 1], 239)):
        own.copy_(_i(lens, dev))
        nq.copy_(_i(news, dev))
        plen.copy_(_i([ahead], dev))
        table.copy_(table.flip(0))
        ws.fill_(255)
        graph.replay()
        got = out.clone()
        assert torch.equal(got, call(torch.empty_like(q), None))


def test_paged_flags_bad_pages_and_lengths():
    dev = torch.device("cuda", 0)
    Z, L, H, Hk, D, page = 2, 1, 2, 1, 64, 16
    q = torch.randn(Z, L, H, D, device=dev).to(torch.bfloat16)
    kp = torch.randn(4, page, Hk, D, device=dev).to(torch.bfloat16)
    vp = torch.randn_like(kp)
    for dt in (torch.bfloat16, torch.float32):
        args = [t.to(dt) for t in (q, kp, vp)]
        sa.last_device_status()
        good = sa.fwd_paged(*args, _i([[0, 1], [2, 3]], dev), _i([16, 32], dev), _i([1, 1], dev), 0.1, -1.0)
        assert sa.last_device_status() == 0
        bad = sa.fwd_paged(*args, _i([[0, 1], [2, 4]], dev), _i([32, 32], dev), _i([1, 1], dev), 0.1, -1.0)
        assert sa.last_device_status() == 10
        part = sa.fwd_paged(*args, _i([[0, -1], [2, 3]], dev), _i([32, 16], dev), _i([1, 1], dev), 0.1, -1.0)
        assert sa.last_device_status() == 10
        assert torch.equal(part[0], good[0])          # the page that is not there weighs nothing
        assert torch.isfinite(bad).all()
        sa.fwd_paged(*args, _i([[0, 1], [2, 3]], dev), _i([16, 33], dev), _i([1, 1], dev), 0.1, -1.0)
        assert sa.last_device_status() == 8
        sa.fwd_paged(*args, _i([[0, 1], [2, 3]], dev), _i([0, 32], dev), _i([1, 1], dev), 0.1, -1.0)
        assert sa.last_device_status() == 8           # a query that is not in the cache


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_train_form_then_cache_then_decode(dev, dt):
    """The three operators together: a causal batch computed at once equals the same batch answered piece by piece from a
    cache whose prefix all samples share.  Both sides round P, the result and, once each, the rotated rows the same way, and
    differ by the order of fp32 sums: within the bound of one rounding of P and one of the result each."""
    Z, H, Hk, D, page, prefix, own = 3, 8, 2, 64, 16, 150, 40
    T = prefix + own
    g = torch.Generator().manual_seed(8)
    r = lambda *s: torch.randn(*s, generator=g).to(dt).to(dev)      # noqa: E731
    q, k, v = r(Z, T, H, D), r(Z, T, Hk, D), r(Z, T, Hk, D)
    for t in (q, k, v):
        t[1:, :prefix] = t[0, :prefix]
    inv = torch.as_tensor(10000.0 ** (-np.arange(32) / 32), dtype=torch.float32, device=dev)
    slopes = torch.linspace(0.1, 0.01, H, device=dev)
    alpha, bias, cap = 0.125, -5.0, 30.0
    pages = 10 + 3 * 4
    kp, vp = torch.full((pages, page, Hk, D), float("nan"), dtype=dt, device=dev), None
    vp = kp.clone()
    pre = _i(np.arange(10), dev)
    table = _i(10 + np.arange(12).reshape(3, 4), dev)
    zero, plen = _i([0], dev), _i([prefix], dev)
    qr = torch.empty_like(q)
    # the prefix, once
    first, _ = sa.cache_append(k[:1, :prefix].contiguous(), v[:1, :prefix].contiguous(), kp, vp, pre.view(1, -1), zero, plen,
                               inv_freq=inv, q=q[:1, :prefix].contiguous())
    qr[:, :prefix] = first
    lens, outs = _i([0] * Z, dev), []
    for a, b in ((0, 25), (25, 26), (26, 32), (32, 33), (33, 40)):
        cut = lambda t: t[:, prefix + a:prefix + b].contiguous()      # noqa: E731,B023
        new = _i([b - a] * Z, dev)
        qs, lens = sa.cache_append(cut(k), cut(v), kp, vp, table, lens, new, inv_freq=inv, q=cut(q), prefix_len=plen)
        qr[:, prefix + a:prefix + b] = qs
        outs.append(sa.fwd_paged(qs, kp, vp, table, lens, new, alpha, bias, prefix_table=pre, prefix_len=plen, cap=cap,
                                 slopes=slopes))
    got = torch.cat(outs, 1)
    flat = lambda c, t: c[t.long()].flatten(-4, -3)      # noqa: E731
    kr = torch.cat([flat(kp, pre)[None, :prefix].expand(Z, -1, -1, -1), flat(kp, table)[:, :own]], 1).contiguous()
    seq = _i([T] * Z, dev)
    spans = sa.mask_spans(seq, T, causal=True)
    o = sa.fwd_span(qr, kr, v, seq, alpha, bias, spans=spans, cap=cap, slopes=slopes)
    want = o[:, prefix:].double().cpu()
    sees = R.visible(spans, [T] * Z, T)
    _, bound = R.reference(qr, kr, v, None, sees, alpha, [bias] * Z, cap, slopes, dt == torch.float32)
    off = (got.double().cpu() - want).abs()
    assert (off <= 2 * bound["O"][:, prefix:]).all()
