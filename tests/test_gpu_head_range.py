"""Gradients of vocabulary rows that no position finds likely: of 1e-8 to 1e-30,
where a batch's other rows have their 1e-3. An optimiser that divides by a
gradient's own size needs them as it needs the others, so every row of dT is
held to its own size here, not to the largest one's.

dz's error, element by element: the exponential's, a rounding to 11 bits (fp32
operands 22), and steps of at most 2^-19 of the largest dz of its vocabulary row,
both in units of their rows' bounds, |a| + |w| rounded down to a power of two.
u = 2^-24 and the products' errors are those of test_gpu_head.py."""
import numpy as np
import pytest
import torch

from oracle import head as oh
from tests.test_gpu_head import HALF, U, Case, f32, f64, to, within
from tests.test_gpu_head_calls import Distill, Loss

pytestmark = pytest.mark.gpu


def unlikely(seed, n, V, d, dt, depth, mixed, pad=0):
    """A case whose vocabulary rows v with v % 3 == 0 lie `depth` and more below
    the others in every row of h; mixed: those with v % 6 == 0 only in the rows
    of its first two thirds."""
    c = Case(seed, n, V, d, dt, pad=pad)
    g = c.g
    H, T = np.array(c.H), np.array(c.T)
    H[:, 0], T[:, 0] = 1.0, 0.0
    rare = np.arange(V) % 3 == 0
    T[rare, 0] = -depth * (1 + g.random(rare.sum()))
    if mixed:
        H[:, 1], T[:, 1] = 0.0, 0.0
        H[n * 2 // 3:, 1] = 1.0
        some = np.arange(V) % 6 == 0
        T[some, 1] = -T[some, 0]
    c.h.copy_(to(H, dt))
    c.table.copy_(to(T, dt))
    c.H, c.T = f64(c.h), f64(c.table)
    c.z = oh.logits(c.H, c.T, 1.0)
    H, T = np.abs(c.H), np.abs(c.T)
    c.ez = H @ T.T * (2 * 6 * d * U + 3.1 * 2.0 ** -22) + 3 * U * np.abs(c.z) + 2.0 ** -39 * (
        H.sum(1)[:, None] * T.max() + H.max(1)[:, None] * T.sum(1)[None])
    return c, rare


def row_bounds(c, dz, p, ez, lse, bound):
    """dT and its bound, each vocabulary row by its own dz; bound: |a| + |w| by row."""
    unit = 2.0 ** np.floor(np.log2(np.where(bound > 0, bound, 1.0)))[:, None]
    one = c.dt == "bf16"
    H = np.abs(c.H)
    edz = p * np.expm1(ez + 6 * U * (np.abs(c.z) + np.abs(lse)[:, None]) + 16 * U)
    edz += 8 * U * (np.abs(dz) + p)
    edz += (np.abs(dz) + edz) * (2.0 ** -11 if one else 2.0 ** -22)
    edz += 2.0 ** -19 * unit * ((np.abs(dz) + edz) / unit).max(0) + 3 * 2.0 ** -126
    mag = np.abs(dz) + edz
    _, ref = oh.grads(dz, c.H, c.T, 1.0)
    b = edz.T @ H + (mag.T @ H) * (2 * (3 * c.n + 1000) * U + (0 if one else 3.1 * 2.0 ** -22))
    # h's copy: half steps of 2^-39 of the largest of its elements times their row's unit
    b += ((mag / unit).sum(0) * 2.0 ** -38 * (H.max(1) * unit[:, 0]).max())[:, None]
    return ref, b + HALF[c.dt] * (np.abs(ref) + b) + 2.0 ** -124


SHAPES = [(300, 900, 128, "bf16"), (700, 1500, 96, "bf16"), (2100, 5003, 128, "bf16"),
          (5, 900, 64, "f32"), (50, 900, 72, "f32"), (64, 9000, 40, "f32"), (300, 900, 72, "f32"),
          (1500, 1300, 129, "f32"), (200, 900, 128, "bf16")]


def weights(g, n):
    return ((1 + g.random(n)) / n * np.where(g.random(n) < 0.5, -1, 1)).astype(np.float32)


@pytest.mark.parametrize("n,V,d,dt", SHAPES)
@pytest.mark.parametrize("depth", [12.0, 30.0])
@pytest.mark.parametrize("mixed", [False, True])
def test_rows_unlikely_everywhere(n, V, d, dt, depth, mixed):
    c, rare = unlikely(41, n, V, d, dt, depth, mixed)
    tok = c.g.choice(np.nonzero(~rare)[0], n)
    tok[::9] = -1
    tok[1] = 3                             # a rare row as a target
    o = Loss(c, tok, zloss=True)
    o.dl, o.ds = f32(weights(c.g, n)), f32(weights(c.g, n) * 0.1)
    o.forward()
    o.backward()
    lse = f64(o.lse)
    dl, ds = f64(o.dl), f64(o.ds)
    dz = oh.loss_dz(c.z, tok, lse, dl, ds)
    p = np.abs(np.where(tok >= 0, dl, 0) + ds)[:, None] * np.exp(c.z - lse[:, None])
    wt = np.where((tok >= 0) & (tok < V), dl, 0)
    ref, b = row_bounds(c, dz, p, c.ez, lse, np.abs(wt + ds) + np.abs(wt))
    own = np.abs(ref).max(1)
    assert own[rare].min() < 2.0 ** -35 * own.max()     # what the test is about
    within("dw", o.dw, ref, b)
    got = f64(o.dw)
    assert np.all(np.abs(got[rare]).max(1) > 0)
    # and dh, as everywhere
    rh, bh, _, _ = c.grad_bounds(dz, p, np.abs(dl) * 2 + np.abs(ds), c.ez, c.z, lse, dt)
    within("dh", o.dh, rh, bh)
    assert o.w2.intact()


@pytest.mark.parametrize("n,V,d,dt", SHAPES)
@pytest.mark.parametrize("mixed", [False, True])
def test_entries_among_unlikely_rows(n, V, d, dt, mixed):
    """Distillation: rare rows named with shares of 1e-6 to 1e-20 and of one half."""
    c, rare = unlikely(42, n, V, d, dt, 20.0, mixed)
    k, tau = 6, 1.0
    ids = np.argsort(c.g.random((n, V)), axis=1)[:, :k]
    few = np.nonzero(rare)[0]
    ids[:, 3:] = few[3:][np.argsort(c.g.random((n, len(few) - 3)), axis=1)[:, :3]]
    teacher = c.g.normal(size=(n, k)).astype(np.float32)
    teacher[:, 3:] -= (14 + 32 * c.g.random((n, 3))).astype(np.float32)
    teacher[::50, 5] = teacher[::50, :3].max(1)
    ids[::7, 4] = ids[::7, 3]              # named twice
    ids[::11] = -1
    o = Distill(c, ids, teacher, tau)
    o.dl = f32(weights(c.g, n))
    o.forward()
    o.backward()
    lse, dl = f64(o.lse), f64(o.dl)
    dz = oh.distill_dz(c.z, ids, teacher, lse, dl, tau)
    q, ok = oh.shares(ids, teacher, V, tau)
    a = np.abs(dl) * (q.sum(1) > 0)
    p = a[:, None] * np.exp(c.z - lse[:, None])
    share = np.zeros_like(p)
    r, j = np.nonzero(ok)
    np.add.at(share, (r, ids[r, j]), a[r] * q[r, j])
    # p and the shares, each with its error: the shares' from logits of at most 64
    ref, b = row_bounds(c, dz, p + share, c.ez + 2.0 ** -16, lse, 2 * a)
    within("dw", o.dw, ref, b)
    rh, bh, _, _ = c.grad_bounds(dz, p + share, 2 * a, c.ez + 2.0 ** -16, c.z, lse, dt)
    within("dh", o.dh, rh, bh)
    assert o.w2.intact()


@pytest.mark.parametrize("n,V,d,dt", [(300, 900, 128, "bf16"), (50, 900, 72, "f32"),
                                      (300, 900, 72, "f32")])
def test_a_graph_with_and_without_unlikely_rows(n, V, d, dt):
    """What one replay lifted is of no account in the next, nor is the workspace."""
    c, rare = unlikely(43, n, V, d, dt, 30.0, True)
    with_rare = c.h.clone()
    without = c.h.clone()
    without[:, 0] = 0
    o = Loss(c, c.g.choice(np.nonzero(~rare)[0], n), zloss=True)

    def step():
        o.forward()
        o.backward()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    seen = []
    for i, h in enumerate((with_rare, without, without, with_rare, without)):
        c.h.copy_(h)
        o.w2.ws.fill_(0xFF if i % 2 else 0)
        step()
        want = o.outputs()
        o.w2.ws.fill_(0x3C if i % 2 else 0xFF)
        for t in (o.loss, o.lse, o.dh, o.dw):
            t.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        got = o.outputs()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, got)), i
        seen.append(got)
    for i, j in ((0, 3), (1, 2), (1, 4)):
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
                   for a, b in zip(seen[i], seen[j]))
    size = f64(seen[0][3])[rare]
    assert 0 < np.abs(size).max(1).min() < 1e-12
    assert o.w1.intact() and o.w2.intact()
