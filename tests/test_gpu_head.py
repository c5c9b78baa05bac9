"""GPU parity of the head's losses and their gradients against the float64
oracle (oracle/head.py).

Bounds count roundings, element by element. u = 2^-24 is half a step of fp32
relative to the value; a matrix instruction may add its terms with up to a
whole step each, so a sum of m products is off by at most 2 m u times the sum
of their magnitudes. fp32 operands, and dz with them, enter as two fp16 halves:
3 d products instead of d, and 3 * 2^-22 of |x||y| for what they leave out (two
halves hold x to 2^-22 of it, and the product of the low ones is dropped); up to
64 tokens' logits as three bf16 planes, 6 d products, of which less is left out. fp16
values are placed with their largest between 2^14 and 2^15, where steps never
get smaller than 2^-24: half of one is 2^-39 of the largest.
"""
import numpy as np
import pytest
import torch

import hashed_head_gram_amd as pg
from oracle import head as oh

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
CODE = {"f32": pg.PG_F32, "bf16": pg.PG_BF16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def dev():
    return torch.device("cuda:0")


def f64(t):
    return t.detach().double().cpu().numpy()


def to(x, dt):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev()).to(DT[dt])


def f32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev())


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(dev())


class Workspace:
    """A workspace full of NaN patterns with a guard behind its end."""

    def __init__(self, size):
        self.all = torch.full((size + 4096,), 0xFF, dtype=torch.uint8, device=dev())
        self.ws = self.all[:size]

    def intact(self):
        return bool((self.all[len(self.ws):] == 0xFF).all())


def products(dt, d):
    """Relative error of a dot product of d terms by the sum of magnitudes."""
    return 2 * d * U if dt == "bf16" else 2 * 6 * d * U + 3.1 * 2.0 ** -22


def within(name, got, ref, bound):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert np.all(np.isfinite(got)), f"{name}: not finite"
    over = np.abs(got - ref) > bound
    at = tuple(x[0] for x in np.nonzero(over)) if over.any() else ()
    assert not over.any(), f"{name}: {over.sum()} over the bound, at {at} {got[at]:.9e} for " \
        f"{ref[at]:.9e}, bound {bound[at]:.3e}"


class Case:
    """Operands, their logits in float64 and the bound of the library's."""

    def __init__(self, seed, n, V, d, dt, scale=1.0, spread=1.0, pad=0):
        g = np.random.default_rng(seed)
        self.n, self.V, self.d, self.dt, self.scale = n, V, d, dt, scale
        whole = torch.full((n, d + pad), 7.0, dtype=DT[dt], device=dev())
        self.h = whole[:, :d]
        self.h.copy_(to(g.normal(size=(n, d)) * spread, dt))
        self.table = to(g.normal(size=(V, d)) / np.sqrt(d), dt)
        self.handle = pg.make_table(CODE[dt], self.table, V)
        self.H, self.T = f64(self.h), f64(self.table)
        self.z = oh.logits(self.H, self.T, scale)
        self.ez = abs(scale) * (np.abs(self.H) @ np.abs(self.T).T) * products(dt, d) \
            + 3 * U * np.abs(self.z)
        if dt == "f32":
            H, T = np.abs(self.H), np.abs(self.T)
            self.ez += abs(scale) * 2.0 ** -39 * (H.sum(1)[:, None] * T.max() +
                                                  H.max(1)[:, None] * T.sum(1)[None])
        self.g = g

    def lse_bound(self, z, ez, lse):
        # the largest of the logits' errors, the exponents' roundings, a sum of
        # positive terms at most 200 deep, exp and log to a few steps
        return ez.max(1) + 4 * U * np.abs(z).max(1) + 220 * U + 4 * U * np.abs(lse)

    def grad_bounds(self, dz, p, bound, ez, z, lse, dw_dt):
        """Bounds of dh and dT: p's error, one rounding of dz (placed by its
        row's bound), the copies' rounding, the two sums."""
        one = self.dt == "bf16"
        rel = np.expm1(ez + 6 * U * (np.abs(z) + np.abs(lse)[:, None]) + 16 * U)
        edz = p * rel + 8 * U * (np.abs(dz) + p)
        edz = edz + (np.abs(dz) + edz) * (2.0 ** -11 if one else 2.0 ** -22)
        # steps below fp16's normal numbers; an exponential, a weight times it and
        # a result below 2^-126, the smallest normal number, may count as zero
        edz = edz + (2.0 ** -39 * bound)[:, None] + 3 * 2.0 ** -126
        s = abs(self.scale)
        V, n = self.V, self.n
        H, T = np.abs(self.H), np.abs(self.T)
        mag = np.abs(dz) + edz
        dh, dt = s * (edz @ T), s * (edz.T @ H)
        # sums over whole slots, splits and pieces; halves: three times as many
        # products, for bf16 and few tokens (dz alone in halves) twice
        k, drop = (2, 0) if one else (3, 3.1 * 2.0 ** -22)
        dh += s * (mag @ T) * (2 * (k * V + 1000) * U + drop)
        dt += s * (mag.T @ H) * (2 * (k * n + 1000) * U + drop)
        # the placed copies of T and h: T by its largest element, h times its
        # row's bound by the largest of those products (bounds are rounded down
        # to powers of two: a factor of 2)
        dh += s * mag.sum(1)[:, None] * 2.0 ** -39 * T.max()
        dt += s * n * 2.0 ** -37 * (bound * H.max(1)).max()
        ref_h, ref_t = oh.grads(dz, self.H, self.T, self.scale)
        dh += HALF[self.dt] * (np.abs(ref_h) + dh)
        dt += HALF[dw_dt] * (np.abs(ref_t) + dt)
        # so may a result and its partial sums
        return ref_h, dh + 2.0 ** -124, ref_t, dt + 2.0 ** -124


def some_targets(g, n, V, ignored=0.1):
    t = g.integers(0, V, n)
    t[g.random(n) < ignored] = -1
    if n > 3:
        t[n // 2] = V                     # just outside
        t[n // 3] = V - 1
    return t


def some_entries(g, n, V, k):
    ids = np.argsort(g.random((n, min(V, 4 * k))), axis=1)[:, :k]
    ids = np.concatenate([ids, np.full((n, k - ids.shape[1]), -1)], 1) if ids.shape[1] < k else ids
    ids = ids * max(1, V // (4 * k)) if V > 4 * k else ids
    ids = np.where(ids >= V, -1, ids)
    teacher = g.normal(size=(n, k)) * 3
    u = g.random(n)
    ids[u < 0.1, k // 2:] = -1
    ids[u < 0.05] = -1
    if n > 4 and k > 2:
        ids[n // 2, k - 1] = ids[n // 2, 0]          # the same id twice
        teacher[n // 3, 1] = -np.inf
        ids[n // 4, 0] = V
    return ids, teacher.astype(np.float32)


SIZES = [  # n, V, d, dtype, scale, spread, pad
    (1, 1, 1, "f32", 1.0, 1.0, 0),
    (1, 2, 16, "bf16", 1.0, 1.0, 0),
    (2, 7, 7, "f32", 1.0, 2.0, 1),
    (31, 100, 63, "bf16", 0.5, 1.0, 3),
    (64, 127, 64, "f32", -1.0, 1.0, 0),
    (127, 1000, 65, "bf16", 1.0, 4.0, 0),
    (128, 1024, 128, "bf16", 1.0, 1.0, 8),
    (129, 129, 192, "f32", 1.0, 1.0, 0),
    (256, 1024, 64, "f32", 1.0, 1.0, 0),
    (257, 2049, 128, "bf16", 1.0, 3.0, 0),
    (300, 5003, 385, "bf16", 1.0, 1.0, 0),
    (33, 50304, 768, "bf16", 1.0, 1.0, 0),
    (32, 20000, 2560, "bf16", 1.0, 1.0, 0),
    (1000, 9001, 129, "f32", 1.0, 2.0, 5),
    (2100, 5003, 128, "bf16", 2.0, 1.0, 8),
    (1500, 6144, 256, "f32", 1.0, 1.0, 0),
    (2500, 300, 320, "bf16", 1.0, 1.0, 0),
    (16, 3000, 16, "bf16", 1.0, 40.0, 0),            # logits of several hundred
    (200, 1000, 128, "bf16", 1.0, 1.0, 0),           # the last rows of the table apart
    (60, 9001, 160, "bf16", 1.0, 1.0, 3),
    (17, 8193, 40, "f32", 1.0, 1.0, 1),
    (200, 777, 97, "bf16", 1.0, 1.0, 0),
    (250, 700, 64, "f32", 1.0, 1.0, 0),
]


@pytest.mark.parametrize("n,V,d,dt,scale,spread,pad", SIZES)
def test_loss(n, V, d, dt, scale, spread, pad):
    c = Case(1, n, V, d, dt, scale, spread, pad)
    tok = some_targets(c.g, n, V)
    w = Workspace(pg.pg_head_loss_workspace_size(n, d, V, CODE[dt]))
    loss, lse = torch.full((n,), 5.0, device=dev()), torch.full((n,), 5.0, device=dev())
    pg.pg_head_loss(c.h, c.handle, i32(tok), loss, lse, w.ws, scale=scale)
    ref, ref_lse = oh.loss(c.H, c.T, tok, scale)
    b = c.lse_bound(c.z, c.ez, ref_lse)
    within("lse", lse, ref_lse, b)
    within("loss", loss, ref, b + c.ez.max(1) + 2 * U * np.abs(c.z).max(1))
    assert w.intact()
    bad = (tok < 0) | (tok >= V)
    assert np.all(f64(loss)[bad] == 0)


@pytest.mark.parametrize("n,V,d,dt,scale,spread,pad", SIZES)
@pytest.mark.parametrize("zloss", [False, True])
def test_loss_backward(n, V, d, dt, scale, spread, pad, zloss):
    c = Case(2, n, V, d, dt, scale, spread, pad)
    tok = some_targets(c.g, n, V)
    lse = oh.log_sum_exp(c.z).astype(np.float32)
    dl = (c.g.normal(size=n) / n).astype(np.float32)
    dl[::5] = 0
    ds = (c.g.normal(size=n) * 1e-2 / n).astype(np.float32) if zloss else None
    w = Workspace(pg.pg_head_loss_backward_workspace_size(n, d, V, CODE[dt]))
    whole = torch.full((n, d + pad), 3.0, dtype=DT[dt], device=dev())
    dw = torch.full((V, d), 3.0, dtype=DT[dt], device=dev())
    pg.pg_head_loss_backward(c.h, c.handle, i32(tok), f32(lse), f32(dl), whole[:, :d], dw, w.ws,
                             dlse=None if ds is None else f32(ds), scale=scale)
    dz = oh.loss_dz(c.z, tok, lse, dl, ds)
    wt = np.where((tok >= 0) & (tok < V), dl, 0)
    a = np.abs(wt + (0 if ds is None else ds))
    p = a[:, None] * np.exp(c.z - lse.astype(np.float64)[:, None])
    rh, bh, rt, bt = c.grad_bounds(dz, p, a + np.abs(wt), c.ez, c.z, lse, dt)
    within("dh", whole[:, :d], rh, bh)
    within("dw", dw, rt, bt)
    assert w.intact() and bool((whole[:, d:] == 3.0).all())


DISTILL = [  # n, V, d, dtype, k, temperature, scale, pad
    (1, 1, 1, "f32", 1, 1.0, 1.0, 0),
    (3, 5, 8, "bf16", 5, 2.0, 1.0, 0),
    (40, 100, 33, "f32", 33, 1.5, 1.0, 2),
    (130, 1000, 128, "bf16", 64, 2.0, 0.5, 0),
    (300, 5003, 129, "bf16", 7, 1.0, 1.0, 3),
    (77, 3001, 64, "f32", 256, 4.0, 1.0, 0),
    (500, 4096, 192, "f32", 100, 0.5, 1.0, 0),
    (2100, 5003, 256, "bf16", 65, 1.0, -1.0, 8),
]


@pytest.mark.parametrize("n,V,d,dt,k,tau,scale,pad", DISTILL)
def test_distill(n, V, d, dt, k, tau, scale, pad):
    c = Case(3, n, V, d, dt, scale, 2.0, pad)
    ids, teacher = some_entries(c.g, n, V, k)
    w = Workspace(pg.pg_head_distill_workspace_size(n, d, V, k, CODE[dt]))
    loss, lse = torch.full((n,), 5.0, device=dev()), torch.full((n,), 5.0, device=dev())
    zk = torch.full((n, k), 5.0, device=dev())
    pg.pg_head_distill(c.h, c.handle, i32(ids), f32(teacher), loss, lse, zk, w.ws,
                       temperature=tau, scale=scale)
    ref, ref_lse, ref_zk = oh.distill(c.H, c.T, ids, teacher, tau, scale)
    ok = (ids >= 0) & (ids < V)
    ek = np.where(ok, np.take_along_axis(c.ez, np.where(ok, ids, 0), 1), 0)
    within("logits", zk, ref_zk, ek)
    b = c.lse_bound(c.z / tau, c.ez / tau, ref_lse)
    within("lse", lse, ref_lse, b)
    q, _ = oh.shares(ids, teacher, V, tau)
    # shares: the teacher's logits over tau and a sum of at most 256
    t = np.where(ok & np.isfinite(teacher), np.abs(teacher) / tau, 0).max(1)
    eq = np.expm1(8 * U * t + 280 * U)
    term = np.abs(np.where(q > 0, np.log(np.where(q > 0, q, 1)), 0)) + np.abs(ref_zk) / tau \
        + np.abs(ref_lse)[:, None]
    within("loss", loss, ref, tau ** 2 * (b + (q * (ek / tau + (eq[:, None] + 300 * U) * (term + 1))
                                               ).sum(1)) + 8 * U * np.abs(ref))
    assert w.intact()


@pytest.mark.parametrize("n,V,d,dt,k,tau,scale,pad", DISTILL)
def test_distill_backward(n, V, d, dt, k, tau, scale, pad):
    c = Case(4, n, V, d, dt, scale, 2.0, pad)
    ids, teacher = some_entries(c.g, n, V, k)
    zt = c.z / tau
    lse = oh.log_sum_exp(zt).astype(np.float32)
    ok = (ids >= 0) & (ids < V)
    zk = np.where(ok, np.take_along_axis(c.z, np.where(ok, ids, 0), 1), 0).astype(np.float32)
    dl = (c.g.normal(size=n) / n).astype(np.float32)
    dl[::7] = 0
    w = Workspace(pg.pg_head_distill_backward_workspace_size(n, d, V, k, CODE[dt]))
    whole = torch.full((n, d + pad), 3.0, dtype=DT[dt], device=dev())
    dw = torch.full((V, d), 3.0, dtype=DT[dt], device=dev())
    pg.pg_head_distill_backward(c.h, c.handle, i32(ids), f32(teacher), f32(lse), f32(zk), f32(dl),
                                whole[:, :d], dw, w.ws, temperature=tau, scale=scale)
    dz = oh.distill_dz(c.z, ids, teacher, lse, dl, tau)
    q, _ = oh.shares(ids, teacher, V, tau)
    a = np.abs(dl) * tau * (q.sum(1) > 0)
    p = a[:, None] * np.exp(zt - lse.astype(np.float64)[:, None])
    # the shares' own error joins p's
    t = np.where(ok & np.isfinite(teacher), np.abs(teacher) / tau, 0).max(1)
    eq = np.expm1(8 * U * t + 280 * U)
    share = np.zeros_like(p)
    r, j = np.nonzero(ok)
    np.add.at(share, (r, ids[r, j]), (a[r] * q[r, j]) * eq[r])
    rh, bh, rt, bt = c.grad_bounds(dz, p, 2 * a, c.ez / tau, zt, lse, dt)
    s = abs(scale)
    bh = bh + 1.01 * s * (share @ np.abs(c.T))
    bt = bt + 1.01 * s * (share.T @ np.abs(c.H))
    within("dh", whole[:, :d], rh, bh)
    within("dw", dw, rt, bt)
    assert w.intact() and bool((whole[:, d:] == 3.0).all())
