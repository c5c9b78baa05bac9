"""The head's losses at values where a rounding, or the range of a number format,
decides: certain tokens, teachers at the ends of fp32, extreme temperatures,
largest elements that never meet.
Helpers are those of test_gpu_head.py and test_gpu_head_calls.py."""
import numpy as np
import pytest
import torch

from oracle import head as oh
from tests.test_gpu_head import U, Case, dev, f64, within
from tests.test_gpu_head_calls import Distill, Loss

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


@pytest.mark.parametrize("n", [40, 300])
def test_teachers_at_the_ends_of_fp32(n):
    """Shares depend on the differences of a teacher's logits over the
    temperature: masks of the type's lowest value, rows of nothing else, and
    values that leave fp32's range when divided."""
    V, d, k, tau = 900, 96, 5, 0.25
    low, high = np.finfo(np.float32).min, np.finfo(np.float32).max
    c = Case(32, n, V, d, "bf16")
    ids = np.argsort(c.g.random((n, V)), axis=1)[:, :k]
    teacher = c.g.normal(size=(n, k)).astype(np.float32)
    teacher[0::6, 2:] = low                # masked entries
    teacher[1::6] = low                    # all the same: equal shares
    teacher[2::6] = high
    teacher[3::6, 0] = high                # one takes all
    teacher[4::6] = -np.inf                # none at all
    o = Distill(c, ids, teacher, tau)
    o.forward()
    o.backward()
    ref, lse, zk = oh.distill(c.H, c.T, ids, teacher, tau)
    # shares to 2^-20: differences of at most 20 over tau, exponentials, a sum of 5
    b = tau ** 2 * (c.lse_bound(c.z / tau, c.ez / tau, lse) + c.ez.max(1) / tau
                    + 2.0 ** -20 * (10 + np.abs(c.z).max(1) / tau + np.abs(lse)))
    within("loss", o.loss, ref, b)
    assert bool((o.loss[4::6] == 0).all()) and bool((o.dh[4::6] == 0).all())
    # the gradient of equal shares is not zero
    assert bool((o.dh[1::6] != 0).any(1).all()) and bool((o.dh[2::6] != 0).any(1).all())
    dz = oh.distill_dz(c.z, ids, teacher, f64(o.lse), f64(o.dl), tau)
    rh, _ = oh.grads(dz, c.H, c.T)
    err = np.linalg.norm(f64(o.dh) - rh, axis=1)
    # half a step of bf16, dz's 2^-12 and the exponentials' error, in the 2-norm of a row
    p = np.abs(f64(o.dl))[:, None] * tau * np.exp(c.z / tau - f64(o.lse)[:, None])
    ez = np.expm1(c.ez / tau + 6 * U * np.abs(c.z) / tau + 2.0 ** -18)
    bound = 2.0 ** -8 * np.linalg.norm(rh, axis=1) + np.linalg.norm(
        (p * ez + np.abs(dz) * (2.0 ** -11 + 2.0 ** -18)) @ np.abs(c.T), axis=1) + 1e-30
    assert np.all(err <= bound), (err / bound).max()


def test_extreme_temperatures():
    """tau^2 and its reciprocal may leave fp32's range where the loss does not:
    tau = 2^-65, logits of about 2^-45, a loss of about 2^-110."""
    n, V, d, k = 30, 500, 64, 4
    tau = 2.0 ** -65
    c = Case(33, n, V, d, "bf16", 2.0 ** -45)
    ids = np.argsort(c.g.random((n, V)), axis=1)[:, :k]
    o = Distill(c, ids, np.zeros((n, k), np.float32), tau)
    o.forward()
    ref = oh.distill(c.H, c.T, ids, np.zeros((n, k)), tau, 2.0 ** -45)[0]
    assert np.all(ref > 2.0 ** -126)
    within("loss", o.loss, ref, 1e-4 * ref + tau * (c.ez.max(1) * 2))


@pytest.mark.parametrize("n", [40, 400])
@pytest.mark.parametrize("scale", [1.0, -1.0])
def test_largest_elements_that_never_meet(n, scale):
    """A column of h where T is zero, and one of T where h is, both of 2^90: what
    undoes their placements is no fp32 number, and the logits are zero all the same."""
    V, d = 700, 96
    c = Case(34, n, V, d, "f32", scale)
    c.h.zero_()
    c.table.zero_()
    c.h[:, 5] = 2.0 ** 90
    c.table[:, 7] = 2.0 ** 90
    tok = c.g.integers(0, V, n)
    o = Loss(c, tok)
    o.forward()
    within("lse", o.lse, np.full(n, np.log(V)), np.full(n, 230 * U + 8 * U))
    o.backward()
    # dz = dloss (1 / V - [target]); dh = dz T, dT = dz^T h, each in its own column
    dz = f64(o.dl)[:, None] * (np.full((n, V), 1.0 / V) - np.eye(V)[tok])
    dh, dw = np.zeros((n, d)), np.zeros((V, d))
    dh[:, 7], dw[:, 5] = scale * 2.0 ** 90 * dz.sum(1), scale * 2.0 ** 90 * dz.sum(0)
    # exponents of 2 ln V at most, sums of V (n) terms
    e = 2.0 ** 90 * np.abs(dz) * 300 * U
    within("dh", o.dh, dh, (2.0 ** 90 * np.abs(dz).sum(1) * 2 * (3 * V + 1000) * U)[:, None]
           + e.sum(1)[:, None])
    within("dw", o.dw, dw, (2.0 ** 90 * np.abs(dz).sum(0) * 2 * (3 * n + 1000) * U)[:, None]
           + e.sum(0)[:, None])
