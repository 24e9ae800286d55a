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


@pytest.mark.parametrize("D", [64, 128])
def test_more_key_heads_than_blocks(dev, D):
    """500 key heads, above the tile kernel's grid: each block takes one head after the other."""
    Z, L, H, page = 2, 2, 500, 16
    own, nq = np.asarray([70, 33]), np.asarray([2, 1])
    table = np.arange(10).reshape(2, 5)
    g = np.random.default_rng(4)
    mark = (g.random((10, page, H)) < 0.3).astype(np.float32)
    vp = torch.zeros(10, page, H, D)
    vp[..., 5] = torch.as_tensor(2 * mark)
    kp = torch.randn(10, page, H, D, generator=torch.Generator().manual_seed(1)).to(dev, torch.bfloat16)
    q = torch.zeros(Z, L, H, D, device=dev, dtype=torch.bfloat16)
    o = sa.fwd_paged(q, kp, vp.to(dev, torch.bfloat16), _i(table, dev), _i(own, dev), _i(nq, dev), 1.0, 0.0).float().cpu().numpy()
    for z in range(Z):
        for l in range(L):
            at = np.arange(own[z] - nq[z] + l + 1 if l < nq[z] else 0)
            want = mark[table[z][at // page], at % page].sum(0) if len(at) else np.zeros(H)
            assert (o[z, l, :, 5] == want).all()


def test_the_most_samples(dev):
    """PAGED_MAX_Z samples of one to three tokens, their pages shared by many: marked values are counted."""
    Z, H, D, page = sa.PAGED_MAX_Z, 2, 64, 16
    own = 1 + np.arange(Z) % 3
    table = (np.arange(Z) % 7)[:, None]
    mark = np.asarray([[(p + s) % 2 for s in range(page)] for p in range(7)], np.float32)
    vp = torch.zeros(7, page, 1, D)
    vp[..., 0, 3] = torch.as_tensor(2 * mark)
    kp = torch.randn(7, page, 1, D, generator=torch.Generator().manual_seed(1)).to(dev, torch.bfloat16)
    q = torch.zeros(Z, 1, H, D, device=dev, dtype=torch.bfloat16)
    o = sa.fwd_paged(q, kp, vp.to(dev, torch.bfloat16), _i(table, dev), _i(own, dev), _i(np.ones(Z), dev), 1.0, 0.0).float().cpu().numpy()
    want = np.asarray([mark[table[z, 0], :own[z]].sum() for z in range(Z)])
    assert (o[:, 0, 0, 3] == want).all() and (o[:, 0, 1, 3] == want).all()


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_infinite_keys(dev, rows, cap):
    """Live keys of infinite entries, in the prefix and among a sample's own: sigma is 1 or 0 by the score's sign."""
    Z, H, D, page, prefix = 2, 2, 64, 16, 200
    own = np.asarray([90, 64])
    nq = np.asarray([rows, rows])
    g = torch.Generator().manual_seed(rows)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(dev)      # noqa: E731
    table, pre = np.arange(12).reshape(2, 6), np.arange(12, 25)
    kp, vp, q = r(25, page, 1, D), r(25, page, 1, D), r(Z, rows, H, D)
    kp[0, 3, 0, 0] = kp[7, 1, 0, 1] = float("inf")
    kp[14, 9, 0, 2] = float("-inf")
    o = sa.fwd_paged(q, kp, vp, _i(table, dev), _i(own, dev), _i(nq, dev), 0.125, -4.0, cap=cap, prefix_table=_i(pre, dev),
                     prefix_len=_i([prefix], dev)).cpu().double()
    assert torch.isfinite(o).all()
    kc, vc, qc = (t.cpu().double()[..., :] for t in (kp, vp, q))
    for z in range(Z):
        n, m = int(own[z]), rows
        k = torch.cat([kc[pre].flatten(0, 1)[:prefix], kc[table[z]].flatten(0, 1)[:n]])[:, 0]
        v = torch.cat([vc[pre].flatten(0, 1)[:prefix], vc[table[z]].flatten(0, 1)[:n]])[:, 0]
        y = 0.125 * (qc[z].transpose(0, 1) @ k.T)
        y = cap * torch.tanh(y / cap) if cap else y
        sees = torch.arange(prefix + n)[None] <= prefix + n - m + torch.arange(m)[:, None]
        want = ((torch.sigmoid(y - 4.0) * sees) @ v).transpose(0, 1)
        C.assert_close(o[z].numpy(), want.numpy(), "bf16", f"sample {z}")


def test_a_decoding_loop_in_a_graph(dev):
    """One captured step of append (lengths in place) and attention, replayed over page borders, equals the same steps called."""
    Z, H, Hk, D, page, prefix = 3, 8, 2, 128, 16, 50
    g = torch.Generator().manual_seed(12)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(dev)      # noqa: E731
    have = np.asarray([0, 15, 30])
    table, pre = _i(np.arange(15).reshape(3, 5), dev), _i(np.arange(15, 19), dev)
    inv = torch.logspace(0, -4, D // 2, device=dev)
    kp, vp = r(19, page, Hk, D), r(19, page, Hk, D)
    one, plen = _i([1] * Z, dev), _i([prefix], dev)
    steps = [(r(Z, 1, Hk, D), r(Z, 1, Hk, D), r(Z, 1, H, D)) for _ in range(25)]

    def step(k, v, q, kp, vp, lens, out, ws):
        sa.cache_append(k, v, kp, vp, table, lens, one, inv_freq=inv, q=q, prefix_len=plen, q_out=q, lens_out=lens)
        return sa.fwd_paged(q, kp, vp, table, lens, one, D ** -0.5, -5.0, prefix_table=pre, prefix_len=plen, cap=15.0, out=out,
                            workspace=ws)

    want, kw, vw, lens = [], kp.clone(), vp.clone(), _i(have, dev)
    for k, v, q in steps:
        want.append(step(k, v, q.clone(), kw, vw, lens, None, None))
    bufs = [torch.empty_like(t) for t in steps[0]]
    out, lens2 = torch.empty_like(bufs[2]), _i(have, dev)
    ws = torch.empty(sa.fwd_paged_workspace_bytes(Z, 1, H, Hk, D, out.dtype), dtype=torch.uint8, device=dev)
    spare = kp.clone(), vp.clone()
    step(*(t.zero_() for t in bufs), *spare, lens2.clone(), out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*bufs, kp, vp, lens2, out, ws)
    for at, new in enumerate(steps):
        for b, t in zip(bufs, new):
            b.copy_(t)
        graph.replay()
        assert torch.equal(out, want[at]), f"step {at}"
    assert torch.equal(kp, kw) and torch.equal(vp, vw) and torch.equal(lens2, lens)
    assert lens.tolist() == (have + 25).tolist()


def test_two_threads_on_two_streams(dev):
    """Calls made at the same time from two threads, each on its own stream, equal the same calls alone."""
    import threading
    Z, H, Hk, D, page = 8, 8, 2, 128, 16
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(dev)      # noqa: E731
    kp, vp, table = r(40, page, Hk, D), r(40, page, Hk, D), _i(np.arange(40).reshape(8, 5), dev)
    own, one = _i(1 + 9 * np.arange(8), dev), _i([1] * 8, dev)
    qs = [r(Z, 1, H, D) for _ in range(2)]
    ts = [r(2, 500, H, D) for _ in range(2)]
    seq = _i([500, 130], dev)

    def work(w):
        return (sa.fwd_paged(qs[w], kp, vp, table, own, one, 0.1, -3.0), sa.fwd_span(ts[w], ts[w], ts[w], seq, 0.1, -3.0),
                *sa.bwd_span(ts[w], ts[w], ts[w], ts[1 - w], seq, 0.1, -3.0))

    want = [work(w) for w in range(2)]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def run(w):
        try:
            with torch.cuda.stream(torch.cuda.Stream(dev)):
                got[w] = [work(w) for _ in range(30)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:          # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(w,)) for w in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for w in range(2):
        for outs in got[w]:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[w]))
    assert math.isfinite(float(want[0][0].float().sum()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [1, 40])
def test_the_output_may_be_the_queries(dev, dtype, rows):
    """O over q gives the same as O beside it: with few rows and with the prefix kernel.  O half over q is refused."""
    Z, H, Hk, D, page, prefix = 3, 4, 2, 64, 16, 70
    g = torch.Generator().manual_seed(rows)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).to(dev)      # noqa: E731
    kp, vp = r(20, page, Hk, D), r(20, page, Hk, D)
    buf = r(Z * rows * H * D + 64)
    q = buf[:-64].view(Z, rows, H, D)
    args = (kp, vp, _i(np.arange(15).reshape(3, 5), dev), _i([80, 41, 66], dev), _i([rows, 1, rows // 2 + 1], dev), 0.125, -2.0)
    more = dict(prefix_table=_i(np.arange(15, 20), dev), prefix_len=_i([prefix], dev))
    want = sa.fwd_paged(q, *args, **more)
    with pytest.raises(ValueError, match="out"):
        sa.fwd_paged(q, *args, out=buf[64:].view(Z, rows, H, D), **more)
    assert torch.equal(sa.fwd_paged(q, *args, out=q, **more), want) and torch.equal(q, want)


def _reference(q, keys, values, prefix, n, m, alpha, bias, cap, slopes):
    """O and its bound (tests/_span_ref.py) of one sample's last m tokens: keys and values [prefix + n, Hk, D] in 64 bits."""
    H, G = q.shape[1], q.shape[1] // keys.shape[1]
    k, v = (t.repeat_interleave(G, 1).transpose(0, 1) for t in (keys, values))
    y = alpha * (q[:m].transpose(0, 1) @ k.mT)
    y = cap * torch.tanh(y / cap) if cap else y
    i, j = prefix + n - m + torch.arange(m, device=q.device)[:, None], torch.arange(prefix + n, device=q.device)[None]
    if slopes is not None:
        y = y - slopes.to(q.device).double().view(H, 1, 1) * (i - j).abs()
    P = torch.sigmoid(y + bias) * (j <= i)
    o = (P @ v).transpose(0, 1)
    return o, R.HALF_BF16 * o.abs() + (R.HALF_BF16 + 1.1e-3) * (P @ v.abs()).transpose(0, 1)


@pytest.mark.parametrize("heads,D,page,prefix,cap,sl", [((4, 1), 128, 64, 333, 0.0, False), ((6, 6), 64, 16, 0, 30.0, True),
                                                        ((8, 2), 64, 32, 1000, 20.0, False)])
def test_prompts(dev, exp_mode, heads, D, page, prefix, cap, sl):
    """Hundreds of new tokens a sample, behind cached ones and behind a prefix: many row tiles, ragged at both ends."""
    (H, Hk), Z, L = heads, 3, 300
    own, nq = np.asarray([300, 777, 431]), np.asarray([300, 257, 1])
    need = -(-own // page)
    g = torch.Generator().manual_seed(prefix)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(dev)      # noqa: E731
    ahead = -(-prefix // page)
    pool = np.random.default_rng(1).permutation(ahead + need.sum())
    table = np.full((Z, need.max()), -1)
    at = ahead
    for z in range(Z):
        table[z, :need[z]] = pool[at:at + need[z]]
        at += need[z]
    kp, vp, q = r(len(pool), page, Hk, D), r(len(pool), page, Hk, D), r(Z, L, H, D)
    slopes = torch.linspace(0.2, 0.001, H, device=dev) if sl else None
    more = dict(prefix_table=_i(pool[:ahead], dev), prefix_len=_i([prefix], dev)) if prefix else {}
    o = sa.fwd_paged(q, kp, vp, _i(table, dev), _i(own, dev), _i(nq, dev), D ** -0.5, -4.0, cap=cap, slopes=slopes, **more)
    for z in range(Z):
        n, m = int(own[z]), int(nq[z])
        rows = lambda t: torch.cat([t[pool[:ahead]].flatten(0, 1)[:prefix], t[table[z, :need[z]]].flatten(0, 1)[:n]]).double()  # noqa: E731,B023
        want, bound = _reference(q[z].double(), rows(kp), rows(vp), prefix, n, m, D ** -0.5, -4.0, cap, slopes)
        off = (o[z, :m].double() - want).abs()
        assert (off <= bound).all(), f"sample {z}: {float((off / bound).max()):.3g} of the bound"
        assert not o[z, m:].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [1, 40])
def test_bad_pages_of_the_prefix_weigh_nothing(dtype, rows):
    """Page numbers outside the cache in the prefix's table are flagged and count as keys of weight zero; a prefix length outside its
    table is flagged and clamped."""
    dev = torch.device("cuda", 0)
    Z, H, D, page = 2, 4, 64, 16
    g = torch.Generator().manual_seed(rows)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).to(dev)      # noqa: E731
    kp, vp, q = r(8, page, 1, D), r(8, page, 1, D), r(Z, rows, H, D)
    kp[7], vp[7] = 0.0, 0.0                                       # keys that weigh nothing, as values
    call = lambda pre, n: sa.fwd_paged(q, kp, vp, _i([[0, 1, 2], [3, 4, 4]], dev), _i([40, 40], dev), _i([rows, rows], dev), 0.1, -1.0,      # noqa: E731
                                       prefix_table=_i(pre, dev), prefix_len=_i([n], dev))
    sa.last_device_status()
    good, short, none = call([5, 7, 6, 7], 64), call([5, 7, 6, 7], 40), call([5, 7, 6, 7], 0)
    assert sa.last_device_status() == 0
    for bad in (8, -1, 2 ** 31 - 1, -2 ** 31):
        got = call([5, bad, 6, bad], 64)
        assert sa.last_device_status() == 10
        assert torch.equal(got, good)
    call([5, 7, 6, -3], 40)                                      # a page that no place reaches is not read
    assert sa.last_device_status() == 0
    for n, want in ((65, good), (2 ** 31 - 1, good), (-1, none), (-2 ** 31, none)):
        got = call([5, 7, 6, 7], n)
        assert sa.last_device_status() == 8
        assert torch.equal(got, want)
    assert not torch.equal(good, short)


def test_nothing_to_answer(dev):
    """No queries at all: zeros, whatever the cache and the queries hold."""
    Z, L, H, D, page = 3, 40, 4, 64, 16
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device=dev)      # noqa: E731
    for own in ([0, 0, 0], [30, 0, 5]):
        for prefix in (0, 40):
            o = sa.fwd_paged(nan(Z, L, H, D), nan(9, page, 2, D), nan(9, page, 2, D), _i([[0, 1], [2, 3], [4, 5]], dev), _i(own, dev),
                             _i([0, 0, 0], dev), 1.0, 0.0, prefix_table=_i([6, 7, 8], dev), prefix_len=_i([prefix], dev), out=nan(Z, L, H, D))
            assert not o.any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pages_beyond_two_to_the_31_entries(dev, dtype):
    """A cache of more than 2^31 entries: what is appended to its last pages, and read from them, equals the same in a small one."""
    Z, H, Hk, D, page = 2, 16, 16, 128, 16
    big = 2 ** 31 // (page * Hk * D) + 40
    kp, vp = (torch.zeros(big, page, Hk, D, dtype=dtype, device=dev) for _ in range(2))
    assert kp.numel() > 2 ** 31
    ks, vs = (torch.zeros(12, page, Hk, D, dtype=dtype, device=dev) for _ in range(2))
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).to(dev)      # noqa: E731
    k, v, q = r(Z, 60, Hk, D), r(Z, 60, Hk, D), r(Z, 60, H, D)
    inv = torch.logspace(0, -4, D // 2, device=dev)
    table = np.arange(8).reshape(2, 4)
    pre = np.arange(8, 12)
    outs = []
    for pages_k, pages_v, first in ((ks, vs, 0), (kp, vp, big - 12)):
        t = _i(first + table, dev)
        pages_k[first + 8:first + 12], pages_v[first + 8:first + 12] = k[0, 0, 0] * 0.5, v[0, 0, 0]
        qr, lens = sa.cache_append(k, v, pages_k, pages_v, t, _i([0, 3], dev), _i([60, 41], dev), inv_freq=inv, q=q)
        for last in (1, 40):
            outs.append([sa.fwd_paged(qr[:, :last].contiguous(), pages_k, pages_v, t, lens, _i([last, last], dev), 0.1, -2.0,
                                      prefix_table=_i(first + pre, dev), prefix_len=_i([50], dev))])
        outs[-1] += [qr, pages_k[first:first + 12].clone(), pages_v[first:first + 12].clone()]
        assert not first or not (pages_k[:first].any() or pages_v[:first].any())
    for a, b in zip(outs[:2], outs[2:]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
