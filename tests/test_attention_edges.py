"""moe_q4_attention at the edges of its arguments (needs an MI355X)."""
from __future__ import annotations

import pytest
import torch

from attention_cases import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hist", [([1, 1], [7, 300]), ([40], [20]), ([200, 3], [0, 0])])
@pytest.mark.parametrize("cap", [0.0, 30.0, 1e6])
def test_slopes_near_the_largest_float(lens, hist, d, cap):
    """A distance of 1 costs everything: a row's own value is left."""
    c = Case(lens, hist, 4, 2, d, 16, seed=1)
    o = c.run(cap=cap, slopes=torch.full((4,), 3.3e38, device="cuda"))
    torch.cuda.synchronize()
    t = 0
    for b, n in enumerate(lens):
        own = c.dense[b][1][c.kv[b] - n:].repeat_interleave(2, 1)
        tol = 2.0 ** -7 * own.abs().float()  # the weight's rounding and the last one
        assert bool(((o[t:t + n].float() - own.float()).abs() <= tol).all()), b
        t += n
