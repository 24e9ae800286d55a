"""Host-side model check of the barrier protocols of the masked attention (span_fwd_sm100.cuh, span_bwd_sm100.cuh) and of the
paged attention (paged_sm100.cuh), in the model of tests/test_barrier_protocols.py: random interleavings of every role, checked
for parity aliasing, miscounted phases, data flow and progress.  The prefix kernel of the paged attention issues as the forward
with two tiles, one part and equal ranges does."""
import pytest

from tests.test_barrier_protocols import Model, ProtocolError


def _producer(n, S, ring):
    """Loads 0 .. n - 1 into `ring` of S slots."""
    for r in range(n):
        if r >= S:
            yield ("wait", f"{ring}_empty{r % S}", r // S - 1)
        yield ("tma", f"{ring}_full{r % S}", r // S, f"{ring}{r % S}", r)


def _ring_bars(ring, S):
    return {f"{ring}_{k}{s}": 1 for k in ("full", "empty") for s in range(S)}


# ------------------------------------------------------------------ forward

def _fwd_mma(j0, j1, J0, J1, KS, VS, NP, early_s=False):
    NT = len(j0)
    steps = J1 - J0
    seen = [0] * NT

    def s(t, c, j):
        yield ("mma", [(f"k{(j - J0) % KS}", j - J0)], [(f"s{t}{c}", ("S", j))])
        yield ("commit", f"s_full{t}{c}", j - j0[t])

    yield ("wait", "k_full0", 0)
    for u in range(NT * NP):
        if j0[u % NT] == J0 < j1[u % NT]:
            yield from s(u % NT, u // NT, J0)
    yield ("commit", "k_empty0", 0)
    for r in range(steps):
        j, sv, sk, more = J0 + r, r % VS, (r + 1) % KS, r + 1 < steps
        yield ("wait", f"v_full{sv}", r // VS)
        have = False
        for u in range(NT * NP):
            t, c = u % NT, u // NT
            if j0[t] <= j < j1[t]:
                if not early_s:
                    yield ("wait", f"p_full{t}{c}", j - j0[t])
                yield ("mma", [(f"s{t}{c}", ("P", j)), (f"v{sv}", r)], [(f"o{t}", j)])
                seen[t] = j
            if u == NT * NP - 1:
                yield ("commit", f"v_empty{sv}", r // VS)
            if more and j0[t] <= j + 1 < j1[t]:
                if not have:
                    yield ("wait", f"k_full{sk}", (r + 1) // KS)
                have = True
                yield from s(t, c, j + 1)
        if more:
            if not have:
                yield ("wait", f"k_full{sk}", (r + 1) // KS)
            yield ("commit", f"k_empty{sk}", (r + 1) // KS)
    yield ("commit", "drain", 0)


def _fwd_sigma(t, part, j0, j1, split):
    """A warpgroup of tile t, whose half of the scores part `part` hands over.  A block that shares its tiles leaves sums for an
    empty one too, where the other's tiles were."""
    for j in range(j0, j1):
        yield ("wait", f"s_full{t}{part}", j - j0)
        yield ("use", f"s{t}{part}", ("S", j))
        yield ("arrive", f"p_full{t}{part}", j - j0)
    if j1 > j0 or split:
        yield ("wait", "drain", 0)
    if j1 > j0:
        yield ("use", f"o{t}", j1 - 1)


class TurnModel(Model):
    """A score buffer named in `turns` changes kind with its barrier's last arrival: {barrier: (buffer, kind)}."""

    turns = {}

    def run(self, *a):
        for name, (key, kind) in self.turns.items():
            if name not in self.bars:
                continue
            bar = self.bars[name]
            arrive = bar.arrive

            def done(who, nm, phase, bar=bar, arrive=arrive, key=key, kind=kind):
                arrive(who, nm, phase)
                if bar.arrived == 0:
                    self.buf[key] = (kind, self.buf[key][1])
            bar.arrive = done
        return super().run(*a)


class FwdModel(TurnModel):
    # P lies over S, part by part
    turns = {f"p_full{t}{c}": (f"s{t}{c}", "P") for t in range(2) for c in range(2)}


def _fwd(j0, j1, KS, VS, NP, seed, bounds=None, **mistake):
    NT = len(j0)
    J0, J1 = bounds or (min(a for a, b in zip(j0, j1) if b > 0), max(j1))
    steps = J1 - J0
    bars = {**_ring_bars("k", KS), **_ring_bars("v", VS), "drain": 1}
    for t in range(NT):
        for c in range(NP):
            bars[f"s_full{t}{c}"] = 1
            bars[f"p_full{t}{c}"] = 2 // NP
    roles = {"K": _producer(steps, KS, "k"), "V": _producer(steps, VS, "v"), "mma": _fwd_mma(j0, j1, J0, J1, KS, VS, NP, **mistake)}
    for t in range(NT):
        for c in range(2):
            roles[f"wg{t}{c}"] = _fwd_sigma(t, c * NP // 2, j0[t], j1[t], bounds is not None)
    FwdModel(bars, roles, seed).run()


RANGES = [((0, 0), (1, 1)), ((0, 0), (7, 8)), ((0, 2), (3, 9)), ((4, 0), (9, 6)), ((0, 5), (2, 8)), ((6, 1), (9, 3)),
          ((0, 0), (0, 5)), ((2, 0), (6, 0))]


@pytest.mark.parametrize("NP", [1, 2])
@pytest.mark.parametrize("ranges", RANGES)
def test_forward_two_tiles(ranges, NP):
    for seed in range(60):
        _fwd(*ranges, 2, 3, NP, seed)


@pytest.mark.parametrize("NP", [1, 2])
@pytest.mark.parametrize("split", [2, 3, 4])
@pytest.mark.parametrize("ranges", RANGES)
def test_forward_shared_by_a_cluster(ranges, split, NP):
    """Each block's part of the key tiles, gaps between the two hulls among them."""
    (j0, j1) = ranges
    J0, J1 = min(a for a, b in zip(j0, j1) if b > 0), max(j1)
    for rank in range(split):
        a, b = J0 + (J1 - J0) * rank // split, J0 + (J1 - J0) * (rank + 1) // split
        if a == b:
            continue
        mine = [(max(x, a), min(y, b)) for x, y in zip(j0, j1)]
        mine = [(x, y) if x < y else (0, 0) for x, y in mine]
        for seed in range(15):
            _fwd([x for x, _ in mine], [y for _, y in mine], 2, 3, NP, seed, bounds=(a, b))


@pytest.mark.parametrize("steps", [1, 2, 3, 7])
def test_forward_one_tile(steps):
    for seed in range(60):
        _fwd((3,), (3 + steps,), 2, 3, 2, seed)


def test_forward_without_waiting_for_p_is_caught():
    with pytest.raises(ProtocolError):
        for seed in range(200):
            _fwd((0, 0), (5, 5), 2, 3, 2, seed, early_s=True)


# ------------------------------------------------------------------ dQ

def _dq_mma(tiles, SX, SY, NP, early_y=False):
    def x(r):
        return f"x{r // NP % SX}", r // NP

    def y(r):
        return f"y{r // NP % SY}", r // NP

    n = tiles * NP
    yield ("wait", "x_full0", 0)
    yield ("wait", "y_full0", 0)
    yield ("mma", [x(0)], [("s", 0)])
    yield ("commit", "s_full", 0)
    yield ("mma", [y(0)], [("dp0", ("dP", 0))])
    yield ("commit", "dp_full0", 0)
    if NP == 1 or early_y:
        yield ("commit", "y_empty0", 0)
    for r in range(n):
        if r + 1 < n:
            t = (r + 1) // NP
            opens, closes = (r + 1) % NP == 0, (r + 1) % NP == NP - 1
            if opens:
                yield ("wait", f"x_full{t % SX}", t // SX)
            yield ("wait", "s_free", r)
            yield ("mma", [x(r + 1)], [("s", r + 1)])
            yield ("commit", "s_full", r + 1)
            if opens:
                yield ("wait", f"y_full{t % SY}", t // SY)
            b = (r + 1) & 1
            yield ("mma", [y(r + 1)], [(f"dp{b}", ("dP", r + 1))])
            yield ("commit", f"dp_full{b}", (r + 1) >> 1)
            if closes and not (early_y and t == 0):
                yield ("commit", f"y_empty{t % SY}", t // SY)
        yield ("wait", f"ds_ready{r & 1}", r >> 1)
        yield ("mma", [(f"dp{r & 1}", ("dS", r)), x(r)], [("dq", r)])
        if r % NP == NP - 1:
            yield ("commit", f"x_empty{r // NP % SX}", r // NP // SX)
    yield ("commit", "drain", 0)


def _dq_sigma(n):
    for r in range(n):
        yield ("wait", "s_full", r)
        yield ("use", "s", r)
        yield ("arrive", "s_free", r)
        yield ("wait", f"dp_full{r & 1}", r >> 1)
        yield ("use", f"dp{r & 1}", ("dP", r))
        yield ("arrive", f"ds_ready{r & 1}", r >> 1)
    yield ("wait", "drain", 0)
    yield ("use", "dq", n - 1)


class DqModel(TurnModel):
    turns = {"ds_ready0": ("dp0", "dS"), "ds_ready1": ("dp1", "dS")}


def _dq(tiles, SX, SY, NP, NG, seed, **mistake):
    bars = {**_ring_bars("x", SX), **_ring_bars("y", SY), "s_full": 1, "dp_full0": 1, "dp_full1": 1, "s_free": NG,
            "ds_ready0": NG, "ds_ready1": NG, "drain": 1}
    roles = {"X": _producer(tiles, SX, "x"), "Y": _producer(tiles, SY, "y"), "mma": _dq_mma(tiles, SX, SY, NP, **mistake)}
    for g in range(NG):
        roles[f"wg{g}"] = _dq_sigma(tiles * NP)
    DqModel(bars, roles, seed).run()


@pytest.mark.parametrize("shape", [(3, 2, 1, 2), (2, 2, 2, 2)])     # D = 128; D = 64 in halves
@pytest.mark.parametrize("tiles", [1, 2, 3, 7])
def test_dq(shape, tiles):
    for seed in range(60):
        _dq(tiles, *shape, seed)


def test_dq_releasing_a_half_read_tile_is_caught():
    with pytest.raises(ProtocolError):
        for seed in range(300):
            _dq(5, 2, 2, 2, 2, seed, early_y=True)


# ------------------------------------------------------------------ dK/dV

def _dkdv_mma(tiles, SX, SY, NP, order=True):
    """Steps of 1 / NP of a tile; both rings' slots are released when their tile's last step has been issued (dO's at once where
    a step is a tile)."""
    yield ("wait", "x_full0", 0)
    yield ("wait", "y_full0", 0)
    yield ("mma", [("x0", 0)], [("s", 0)])
    yield ("commit", "s_full", 0)
    yield ("mma", [("y0", 0)], [("dp", ("dP", 0)), ("ds", ("dP", 0))])
    yield ("commit", "dp_full", 0)
    for r in range(tiles * NP):
        nxt, t, t1 = r + 1, r // NP, (r + 1) // NP
        more, opens, closes = nxt < tiles * NP, nxt % NP == 0, r % NP == NP - 1
        if more:
            if opens:
                yield ("wait", f"x_full{t1 % SX}", t1 // SX)
            yield ("wait", "s_free", r)
            yield ("mma", [(f"x{t1 % SX}", t1)], [("s", nxt)])
            yield ("commit", "s_full", nxt)
        yield ("wait", "p_ready", r)
        yield ("mma", [("dp", ("P", r)), (f"y{t % SY}", t)], [("dv", r)])
        if NP == 1:
            yield ("commit", f"y_empty{t % SY}", t // SY)
        if order:
            yield ("wait", "ds_ready", r)
        yield ("mma", [("ds", ("dS", r)), (f"x{t % SX}", t)], [("dk", r)])
        if closes:
            if NP > 1:
                yield ("commit", f"y_empty{t % SY}", t // SY)
            yield ("commit", f"x_empty{t % SX}", t // SX)
        if more:
            if opens:
                yield ("wait", f"y_full{t1 % SY}", t1 // SY)
            yield ("mma", [(f"y{t1 % SY}", t1)], [("dp", ("dP", nxt)), ("ds", ("dP", nxt))])
            yield ("commit", "dp_full", nxt)
    yield ("commit", "drain", 0)


def _both_rings(n, SX, SY):
    """One thread that loads a tile of each ring in turn."""
    x, y = _producer(n, SX, "x"), _producer(n, SY, "y")
    for _ in range(n):
        for ring in (x, y):
            for step in ring:
                yield step
                if step[0] == "tma":
                    break


def _dkdv_sigma(n, empty):
    """empty: tiles in which no query of the warpgroup's columns sees a key (P and dS are written as zeros together)."""
    for r in range(n):
        yield ("wait", "s_full", r)
        if r not in empty:
            yield ("use", "s", r)
        yield ("arrive", "s_free", r)
        yield ("wait", "dp_full", r)
        if r not in empty:
            yield ("use", "dp", ("dP", r))
        yield ("arrive", "p_ready", r)
        yield ("arrive", "ds_ready", r)
    yield ("wait", "drain", 0)
    yield ("use", "dk", n - 1)
    yield ("use", "dv", n - 1)


class DkdvModel(TurnModel):
    # P^T lies over one half of each warpgroup's dP^T columns, dS^T over the other
    turns = {"p_ready": ("dp", "P"), "ds_ready": ("ds", "dS")}


def _dkdv(tiles, SX, SY, NP, NG, seed, **mistake):
    bars = {**_ring_bars("x", SX), **_ring_bars("y", SY), "s_full": 1, "dp_full": 1, "s_free": NG, "p_ready": NG,
            "ds_ready": NG, "drain": 1}
    roles = {"mma": _dkdv_mma(tiles, SX, SY, NP, **mistake)}
    roles.update({"XY": _both_rings(tiles, SX, SY)} if NP > 1 else
                 {"X": _producer(tiles, SX, "x"), "Y": _producer(tiles, SY, "y")})
    for g in range(NG):
        roles[f"wg{g}"] = _dkdv_sigma(tiles * NP, {r for r in range(tiles * NP) if (r + g + seed) % 3 == 0})
    DkdvModel(bars, roles, seed).run()


@pytest.mark.parametrize("shape", [(3, 2, 1, 2), (2, 2, 2, 2)])     # D = 128; D = 64 in halves
@pytest.mark.parametrize("tiles", [1, 2, 3, 9])
def test_dkdv(shape, tiles):
    for seed in range(60):
        _dkdv(tiles, *shape, seed)


def test_dkdv_without_waiting_for_ds_is_caught():
    with pytest.raises(ProtocolError):
        for seed in range(200):
            _dkdv(5, 3, 2, 1, 2, seed, order=False)


# ------------------------------------------------------------------ paged tile kernel

def _paged_consumer(n, S, lead):
    for t in range(n):
        yield ("wait", f"k_full{t % S}", t // S)
        yield ("use", f"k{t % S}", t)
        yield ("arrive", f"k_empty{t % S}", t // S)
        if lead and t == lead:
            yield ("arrive", f"k_empty{t % S}", None)


@pytest.mark.parametrize("S", [3, 4])
@pytest.mark.parametrize("n", [1, 2, 5, 17])
def test_paged_ring(S, n):
    for seed in range(60):
        bars = {**{f"k_full{s}": 1 for s in range(S)}, **{f"k_empty{s}": 4 for s in range(S)}}
        roles = {"producer": _producer(n, S, "k"), **{f"warp{w}": _paged_consumer(n, S, 0) for w in range(4)}}
        Model(bars, roles, seed).run()


def test_paged_ring_counts_its_arrivals():
    with pytest.raises(ProtocolError):
        for seed in range(100):
            bars = {**{f"k_full{s}": 1 for s in range(3)}, **{f"k_empty{s}": 4 for s in range(3)}}
            roles = {"producer": _producer(12, 3, "k"), **{f"warp{w}": _paged_consumer(12, 3, 2 if w == 0 else 0)
                                                          for w in range(4)}}
            Model(bars, roles, seed).run()
