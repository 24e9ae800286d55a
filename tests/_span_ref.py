"""Masked sigmoid attention in 64 bits, from its definition, with the error bounds the GPU tests hold the kernels to.

Bounds, per output element, for the EXP sigma form (bf16 path):

* P is evaluated with a relative error of at most 1e-3: 3.4e-4 of the polynomial for 1/(1+u), and the error of the fp32
  argument x (the product's accumulation, at most D 2^-24 sum|q k| alpha, and a few roundings of |x| 2^-24), which moves P by
  at most P dx; with the shapes here dx < 3e-4.  Its derivative g carries twice the polynomial's error: 2e-3.
* P and dS are rounded to bf16 before their second product: half a step, 2^-8.
* sums are kept in fp32 (n 2^-24, below 1e-4 for the lengths here), and the result is rounded to bf16: 2^-8 of itself.

So |O - ref| <= 2^-8 |ref| + (2^-8 + 1e-3 + 1e-4) sum_j P_ij |v_j|, and likewise for dV; for dQ and dK the terms are
dS_ij = g_ij dP_ij with (2^-8 + 2e-3 + 1e-4) |dS| and the fp32 error of dP, D 2^-24 sum|dO v| g.
fp32 path: every constant above becomes 2e-5 (expf, tanhf and divisions of a few ulp, sums of up to n terms)."""
import numpy as np
import torch

HALF_BF16 = 2.0 ** -8


def visible(spans, n, L):
    """[Z, L, L] truth values from spans [Z, L, 2] (None: all) and lengths [Z]."""
    i = torch.arange(L)
    n = torch.as_tensor(np.asarray(n, np.int64))
    ok = (i[None, None, :] < n[:, None, None]) & (i[None, :, None] < n[:, None, None])
    if spans is not None:
        s = spans.long().cpu()
        ok &= (i >= s[..., 0, None]) & (i < s[..., 1, None])
    return ok


def reference(q, k, v, do, sees, alpha, bias, cap, slopes, fp32=False):
    """(outputs, bounds): dicts of O, dQ, dK, dV in 64 bits on the CPU.  bias: [Z]."""
    dt = torch.float64
    q, k, v = (t.detach().cpu().to(dt).transpose(1, 2) for t in (q, k, v))       # [Z, heads, L, D]
    do = None if do is None else do.detach().cpu().to(dt).transpose(1, 2)
    Z, H, L, D = q.shape
    Hk = k.shape[1]
    G = H // Hk
    ke, ve = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    y = alpha * (q @ ke.mT)
    f = torch.ones_like(y)
    if cap:
        t = torch.tanh(y / cap)
        y, f = cap * t, 1 - t * t
    i = torch.arange(L)
    if slopes is not None:
        y = y - slopes.detach().cpu().to(dt).view(1, H, 1, 1) * (i[:, None] - i[None]).abs().to(dt)
    x = y + torch.as_tensor(np.asarray(bias, np.float64)).view(Z, 1, 1, 1)
    m = sees[:, None]
    P = torch.where(m, torch.sigmoid(x), torch.zeros(()).to(dt))
    live = sees.any(-1)[:, None, :, None]
    ve0 = torch.where(sees.any(1)[:, None, :, None], ve, torch.zeros(()).to(dt))   # values no row sees may be NaN
    ke0 = torch.where(sees.any(1)[:, None, :, None], ke, torch.zeros(()).to(dt))
    P = torch.nan_to_num(P)
    ep, eg, eo = (2e-5, 2e-5, 2e-5) if fp32 else (HALF_BF16 + 1.1e-3, HALF_BF16 + 2.1e-3, HALF_BF16)
    out = {"O": P @ ve0}
    bound = {"O": eo * out["O"].abs() + ep * (P @ ve0.abs())}
    if do is not None:
        q0 = torch.where(live, q, torch.zeros(()).to(dt))
        do0 = torch.where(live, do, torch.zeros(()).to(dt))
        g = torch.where(m, torch.sigmoid(x) * torch.sigmoid(-x) * f, torch.zeros(()).to(dt)).nan_to_num()
        dS = alpha * g * (do0 @ ve0.mT)
        E = eg * dS.abs() + alpha * g * (D * 2.0 ** -24) * (do0.abs() @ ve0.abs().mT)
        fold = lambda t: t.view(Z, Hk, G, L, -1).sum(2)      # noqa: E731
        out |= {"dQ": dS @ ke0, "dK": fold(dS.mT @ q0), "dV": fold(P.mT @ do0)}
        bound |= {"dQ": eo * out["dQ"].abs() + E @ ke0.abs(), "dK": eo * out["dK"].abs() + fold(E.mT @ q0.abs()),
                  "dV": eo * out["dV"].abs() + ep * fold(P.mT @ do0.abs())}
    back = lambda d: {a: b.transpose(1, 2).contiguous() for a, b in d.items()}     # noqa: E731
    return back(out), back(bound)


def assert_within(got, ref, bound, what):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = (got - ref).abs()
    over = off > bound + 1e-30
    assert not over.any(), (f"{what}: {int(over.sum())} of {over.numel()} out of bounds, worst "
                            f"{float((off / (bound + 1e-30)).max()):.3g} of the bound")


def make_spans(kind, n, L, seed=0):
    """int32 [Z, L, 2] CPU spans of the kinds the tests use, rows of padding left as they come out."""
    g = np.random.default_rng(seed)
    i = np.arange(L)
    out = np.zeros((len(n), L, 2), np.int64)
    for z, m in enumerate(n):
        lo, hi = np.zeros(L, np.int64), np.full(L, L)
        if kind in ("causal", "docs_causal"):
            hi = i + 1
        if kind == "prefix":
            hi = np.maximum(i + 1, g.integers(0, max(1, m) + 1))
        if kind == "window":
            lo, hi = i - 37, i + 11
        if kind.startswith("docs"):
            cut = np.flatnonzero(g.random(L) < 0.02)
            at = np.searchsorted(cut, i, side="right")
            lo = np.concatenate([[0], cut])[at]
            hi = np.minimum(hi, np.concatenate([cut, [L]])[at])
        if kind == "holes":         # causal, every third run of 50 rows sees nothing, one row outside everything
            hi = np.where((i // 50) % 3 == 1, 0, i + 1)
            lo = np.where(i % 7 == 3, i + 5, 0)
        if kind == "scatter":       # anything: empty, reversed, negative and far beyond the end
            lo = g.integers(-L - 3, 2 * L, size=L)
            hi = g.integers(-L - 3, 2 * L, size=L)
            lo[g.random(L) < 0.3] = -2 ** 31
            hi[g.random(L) < 0.3] = 2 ** 31 - 1
        out[z, :, 0], out[z, :, 1] = lo, hi
    return torch.as_tensor(out.astype(np.int32))
