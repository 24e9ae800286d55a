"""The masked attention's and the cache's refusals and host state beyond the usual cases, without a GPU."""
import ctypes
import os

import pytest
import torch

from tests.test_span_cpu import sa  # noqa: F401  (the built package)

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "padding_aware_sigmoid_b200", "csrc")


@pytest.mark.parametrize("cast", [lambda m: m.bfloat16(), lambda m: m.half(), lambda m: m.double(), lambda m: m.to(torch.bfloat16),
                                  lambda m: m.bfloat16().float(), lambda m: m.to("meta").to_empty(device="cpu")])
def test_casts_leave_the_slopes_as_they_are(sa, cast):  # noqa: F811
    slopes = [0.3, 1 / 3, 1e-5]
    model = torch.nn.Sequential(torch.nn.Linear(2, 2), sa.SigmoidAttention(slopes=slopes))
    cast(model)
    got = model[1].slopes
    assert got.dtype == torch.float32 and got.shape == (3,) and "slopes" in dict(model[1].named_buffers())
    assert got.device.type == "cpu"


def test_casts_round_no_slope(sa):  # noqa: F811
    m = sa.SigmoidAttention(slopes=[0.3, 1 / 3, 1e-5])
    want = m.slopes.clone()
    for cast in (m.bfloat16, m.half, m.double, m.float):
        assert cast() is m and torch.equal(m.slopes, want)
    assert sa.SigmoidAttention(cap=3.0).bfloat16().slopes is None
    p = sa.SigmoidAttention(learnable_bias=True, bias=-1.0).bfloat16()
    assert p.b.dtype == torch.bfloat16


def test_cluster_barriers_meet_whole_warps():
    """barrier.cluster's .aligned form is undefined for a warp whose lanes have parted; rows beyond L part them (split_add).  The
    barrier is written in one place, which brings the warp together first, so no caller can leave that out."""
    src = {f: open(os.path.join(CSRC, f)).read() for f in os.listdir(CSRC)}
    at = [f for f, text in src.items() if "barrier.cluster" in text]
    assert at == ["span_split.cuh"] and src[at[0]].count("barrier.cluster.arrive") == 1
    body = src[at[0]].split("void cluster_meet() {")[1].split("}")[0]
    assert body.index("__syncwarp()") < body.index("barrier.cluster.arrive")


def test_append_refuses_heads_that_do_not_count_in_32_bits(sa):  # noqa: F811
    """H + 2 Hk heads of a token are counted in 32 bits: beyond that the call wrote nothing and answered OK."""
    lib, P = sa.load_library(), ctypes.c_void_p(16)
    call = lambda H, Hk: lib.sigattn_cache_append(P, P, P if H else None, P if H else None, P, P, P, P, P, None, P, 1, 1, H, Hk, 64, 1,      # noqa: E731
                                                  16, 1, None, 0, 0, 0, None)
    assert call(0, 2 ** 30) == 9 and call(0, 65536) == 9 and call(2 ** 31 - 2, 2 ** 30 - 1) == 9
