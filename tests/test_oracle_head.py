"""Pins of the head's oracle (oracle/head.py): autograd in float64 and differences."""
import numpy as np
import pytest
import torch

from oracle import head as oh


def inputs(seed, n=7, V=23, d=5, k=4):
    g = np.random.default_rng(seed)
    h, t = g.normal(size=(n, d)), g.normal(size=(V, d))
    tok = g.integers(0, V, n)
    tok[1], tok[3] = -1, V
    ids = np.stack([g.permutation(V)[:k] for _ in range(n)])
    ids[2, 1:] = -1
    ids[4] = V
    ids[5, 3] = ids[5, 0]
    return h, t, tok, ids, g.normal(size=(n, k)) * 2, g.normal(size=n), g.normal(size=n)


@pytest.mark.parametrize("scale", [1.0, -0.7])
def test_loss_against_autograd(scale):
    h, t, tok, _, _, dl, ds = inputs(0)
    H = torch.tensor(h, requires_grad=True)
    T = torch.tensor(t, requires_grad=True)
    z = scale * H @ T.T
    ok = torch.tensor((tok >= 0) & (tok < len(t)))
    want = torch.nn.functional.cross_entropy(z, torch.tensor(np.where(ok, tok, 0)),
                                             reduction="none") * ok
    lse = torch.logsumexp(z, 1)
    (want * torch.tensor(dl) + lse * torch.tensor(ds)).sum().backward()
    got, glse = oh.loss(h, t, tok, scale)
    np.testing.assert_allclose(got, want.detach(), atol=1e-12)
    np.testing.assert_allclose(glse, lse.detach(), atol=1e-12)
    dh, dt = oh.grads(oh.loss_dz(oh.logits(h, t, scale), tok, glse, dl, ds), h, t, scale)
    np.testing.assert_allclose(dh, H.grad, atol=1e-12)
    np.testing.assert_allclose(dt, T.grad, atol=1e-12)


@pytest.mark.parametrize("temperature", [1.0, 2.5])
def test_distill_against_autograd(temperature):
    h, t, _, ids, teacher, dl, _ = inputs(1)
    n, V = len(h), len(t)
    H = torch.tensor(h, requires_grad=True)
    T = torch.tensor(t, requires_grad=True)
    logp = torch.log_softmax(H @ T.T / temperature, 1)
    want = []
    for i in range(n):
        ok = (ids[i] >= 0) & (ids[i] < V)
        if not ok.any():
            want.append(logp[i].sum() * 0)
            continue
        q = torch.softmax(torch.tensor(teacher[i][ok]) / temperature, 0)
        want.append(temperature ** 2 * (q * (q.log() - logp[i][torch.tensor(ids[i][ok])])).sum())
    want = torch.stack(want)
    (want * torch.tensor(dl)).sum().backward()
    got, lse, zk = oh.distill(h, t, ids, teacher, temperature)
    np.testing.assert_allclose(got, want.detach(), atol=1e-11)
    dh, dt = oh.grads(oh.distill_dz(oh.logits(h, t, 1.0), ids, teacher, lse, dl, temperature), h, t)
    np.testing.assert_allclose(dh, H.grad, atol=1e-11)
    np.testing.assert_allclose(dt, T.grad, atol=1e-11)
    assert np.all(zk[4] == 0) and np.all(zk[2, 1:] == 0)


@pytest.mark.parametrize("kind", ["loss", "distill"])
def test_gradients_against_differences(kind):
    h, t, tok, ids, teacher, dl, _ = inputs(2)

    def total(h, t):
        if kind == "loss":
            return (oh.loss(h, t, tok, 0.9)[0] * dl).sum()
        return (oh.distill(h, t, ids, teacher, 1.7, 0.9)[0] * dl).sum()

    z = oh.logits(h, t, 0.9)
    if kind == "loss":
        dz = oh.loss_dz(z, tok, oh.log_sum_exp(z), dl)
    else:
        dz = oh.distill_dz(z, ids, teacher, oh.log_sum_exp(z / 1.7), dl, 1.7)
    dh, dt = oh.grads(dz, h, t, 0.9)
    e = 1e-5
    for x, dx in ((h, dh), (t, dt)):
        for i in np.ndindex(x.shape):
            keep = x[i]
            x[i] = keep + e
            up = total(h, t)
            x[i] = keep - e
            down = total(h, t)
            x[i] = keep
            assert abs((up - down) / (2 * e) - dx[i]) < 1e-7
