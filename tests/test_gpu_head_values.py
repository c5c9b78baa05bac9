"""The head's losses at values where a rounding, or the range of a number format,
decides.
Helpers are those of test_gpu_head.py and test_gpu_head_calls.py."""
import numpy as np
import pytest
import torch

from oracle import head as oh
from tests.test_gpu_head import U, Case, dev, f64, within
from tests.test_gpu_head_calls import Loss

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,n", [("bf16", 40), ("bf16", 300), ("bf16", 2100), ("f32", 40),
                                  ("f32", 400)])
@pytest.mark.parametrize("scale", [1.0, -1.0])
def test_no_cross_entropy_below_zero(dt, n, scale):
    """A sum of exponentials is never below one of its terms. Of a token that is
    certain the two differ by roundings alone, and those may not show as a sign."""
    V, d = 1000, 192
    c = Case(31, n, V, d, dt, scale)
    tok = c.g.integers(0, V, n)
    c.h.copy_(c.table[torch.from_numpy(tok).to(dev())] * (300 * scale))
    c.H = f64(c.h)
    o = Loss(c, tok)
    o.forward()
    assert bool((o.loss >= 0).all()), float(o.loss.min())
    # the errors of the sum and of the one term, as the loss itself is all but zero
    ref, lse = oh.loss(c.H, c.T, tok, scale)
    z = oh.logits(c.H, c.T, scale)
    ez = np.abs(c.H) @ np.abs(c.T).T * (12 * d * U + 3.1 * 2.0 ** -22) + 3 * U * np.abs(z)
    if dt == "f32":
        H, T = np.abs(c.H), np.abs(c.T)
        ez += 2.0 ** -39 * (H.sum(1)[:, None] * T.max() + H.max(1)[:, None] * T.sum(1)[None])
    within("loss", o.loss, ref, c.lse_bound(z, ez, lse) + ez.max(1) + 2 * U * np.abs(z).max(1))
