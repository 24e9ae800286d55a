"""The readme's Python examples run as they stand, and the serving example's keys are rotated to their positions behind the prefix."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

sa = pytest.importorskip("padding_aware_sigmoid_b200")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_examples():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sa.last_device_status()
    dev = torch.device("cuda", 0)
    blocks = re.findall(r"```python\n(.*?)```", open(os.path.join(ROOT, "README.md")).read(), re.S)
    assert len(blocks) == 2
    r = lambda *s: torch.randn(*s, device=dev).to(torch.bfloat16)      # noqa: E731
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)      # noqa: E731
    Z, H, Hk, D, page = 3, 16, 4, 128, 16
    ns = {"k_new": r(Z, 1, Hk, D), "v_new": r(Z, 1, Hk, D), "q_new": r(Z, 1, H, D), "n_new": i(1, 1, 1), "lens": i(0, 17, 31),
          "k_pages": r(12, page, Hk, D), "v_pages": r(12, page, Hk, D), "page_table": torch.arange(6, device=dev, dtype=torch.int32).view(3, 2),
          "shared_pages": i(6, 7, 8, 9, 10, 11), "shared_len": i(90), "inv_freq": torch.logspace(0, -4, D // 2, device=dev)}
    want_k, want_v = ns["k_pages"].clone(), ns["v_pages"].clone()
    q, lens = sa.cache_append(ns["k_new"], ns["v_new"], want_k, want_v, ns["page_table"], ns["lens"], ns["n_new"], ns["inv_freq"],
                              q=ns["q_new"], prefix_len=ns["shared_len"])
    for b in blocks:
        exec(b, ns)
    assert torch.equal(ns["k_pages"], want_k) and torch.equal(ns["v_pages"], want_v)
    assert torch.equal(ns["q_rot"], q) and torch.equal(ns["lens"], lens)
    assert torch.isfinite(ns["o"]).all() and ns["o"].shape == (Z, 1, H, D) and ns["dk"].shape == (2, 4096, 4, 128)
    assert sa.last_device_status() == 0
