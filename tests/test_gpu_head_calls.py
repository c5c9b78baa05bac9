"""The head's losses and gradients as programs call them: padded batches, parts
of the gradients, tied tables, pieces of the vocabulary and of the batch,
captured and repeated calls, other streams, values of very different sizes.
Bounds and helpers are those of test_gpu_head.py."""
import numpy as np
import pytest
import torch

import hashed_head_gram_amd as pg
from oracle import head as oh
from oracle import train as ot
from tests.test_gpu_head import (CODE, DT, HALF, U, Case, Workspace, dev, f32, f64, i32, products,
                                 some_entries, some_targets, to, within)

pytestmark = pytest.mark.gpu

SHAPES = [(40, 300, 96, "bf16"), (40, 300, 96, "f32"), (300, 900, 128, "bf16"),
          (300, 900, 130, "bf16"), (300, 900, 72, "f32")]


class Loss:
    """Cross entropy of a case: buffers and the two calls."""

    def __init__(self, c, tok, zloss=False, dw=None):
        n, V, d, code = c.n, c.V, c.d, CODE[c.dt]
        self.c, self.tok = c, i32(tok)
        self.loss, self.lse = torch.empty(n, device=dev()), torch.empty(n, device=dev())
        self.dl = f32(c.g.normal(size=n) / n)
        self.ds = f32(c.g.normal(size=n) * 1e-2 / n) if zloss else None
        self.dh = torch.empty_like(c.h.contiguous())
        self.dw = torch.empty(V, d, dtype=DT[dw or c.dt], device=dev())
        self.w1 = Workspace(pg.pg_head_loss_workspace_size(n, d, V, code))
        self.w2 = Workspace(pg.pg_head_loss_backward_workspace_size(n, d, V, code))

    def forward(self, **kw):
        pg.pg_head_loss(self.c.h, self.c.handle, self.tok, self.loss, self.lse, self.w1.ws,
                        scale=self.c.scale, **kw)

    def backward(self, dh=True, dw=True, **kw):
        pg.pg_head_loss_backward(self.c.h, self.c.handle, self.tok, self.lse, self.dl,
                                 self.dh if dh else None, self.dw if dw else None, self.w2.ws,
                                 dlse=self.ds, scale=self.c.scale, **kw)

    def outputs(self):
        return [t.clone() for t in (self.loss, self.lse, self.dh, self.dw)]


class Distill(Loss):
    """Distillation of a case."""

    def __init__(self, c, ids, teacher, tau=1.5):
        n, V, d, code, k = c.n, c.V, c.d, CODE[c.dt], ids.shape[1]
        super().__init__(c, np.zeros(n))
        self.ids, self.teacher, self.tau = i32(ids), f32(teacher), tau
        self.zk = torch.empty(n, k, device=dev())
        self.w1 = Workspace(pg.pg_head_distill_workspace_size(n, d, V, k, code))
        self.w2 = Workspace(pg.pg_head_distill_backward_workspace_size(n, d, V, k, code))

    def forward(self, **kw):
        pg.pg_head_distill(self.c.h, self.c.handle, self.ids, self.teacher, self.loss, self.lse,
                           self.zk, self.w1.ws, temperature=self.tau, scale=self.c.scale, **kw)

    def backward(self, dh=True, dw=True, **kw):
        pg.pg_head_distill_backward(self.c.h, self.c.handle, self.ids, self.teacher, self.lse,
                                    self.zk, self.dl, self.dh if dh else None,
                                    self.dw if dw else None, self.w2.ws, temperature=self.tau,
                                    scale=self.c.scale, **kw)

    def outputs(self):
        return super().outputs() + [self.zk.clone()]


def both(c, k=9):
    ids, teacher = some_entries(c.g, c.n, c.V, k)
    return [Loss(c, some_targets(c.g, c.n, c.V)), Distill(c, ids, teacher)]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def grad_bounds(o, dw_dt=None):
    """(dh, its bound, dw, its bound) of a Loss from its own lse."""
    c, tok = o.c, o.tok.cpu().numpy()
    lse, dl = f64(o.lse), f64(o.dl)
    ds = None if o.ds is None else f64(o.ds)
    dz = oh.loss_dz(c.z, tok, lse, dl, ds)
    wt = np.where((tok >= 0) & (tok < c.V), dl, 0)
    a = np.abs(wt + (0 if ds is None else ds))
    p = a[:, None] * np.exp(c.z - lse[:, None])
    return c.grad_bounds(dz, p, a + np.abs(wt), c.ez, c.z, lse, dw_dt or c.dt)


@pytest.mark.parametrize("n,V,d,dt", SHAPES)
def test_rows_without_target_may_hold_anything(n, V, d, dt):
    c = Case(10, n, V, d, dt)
    out = np.arange(n) % 4 == 1
    tok = np.where(out, -100, c.g.integers(0, V, n))
    ids, teacher = some_entries(c.g, n, V, 5)
    ids[out] = -1
    for o in (Loss(c, tok), Distill(c, ids, teacher)):
        results = []
        for junk in (0.0, float("nan"), float("inf"), 1e30):
            c.h[torch.from_numpy(out).to(dev())] = junk
            o.forward()
            o.lse[torch.from_numpy(out).to(dev())] = junk
            o.backward()
            loss, lse, dh, dw = o.outputs()[:4]
            assert bool((loss[torch.from_numpy(out).to(dev())] == 0).all())
            assert bool((dh[torch.from_numpy(out).to(dev())] == 0).all())
            lse[torch.from_numpy(out).to(dev())] = 0
            assert bool(torch.isfinite(dw.float()).all()) and bool(torch.isfinite(dh.float()).all())
            results.append([loss, lse, dh, dw])
        for r in results[1:]:
            assert same(results[0], r)


@pytest.mark.parametrize("n,V,d,dt", SHAPES)
def test_nothing_to_learn(n, V, d, dt):
    c = Case(11, n, V, d, dt)
    for o in (Loss(c, np.full(n, -1)), Distill(c, np.full((n, 3), V), np.zeros((n, 3)))):
        o.forward()
        o.backward()
        assert bool((o.loss == 0).all()) and bool((o.dh == 0).all()) and bool((o.dw == 0).all())
        within("lse", o.lse, oh.log_sum_exp(c.z / getattr(o, "tau", 1.0)),
               c.lse_bound(c.z, c.ez, oh.log_sum_exp(c.z)))


@pytest.mark.parametrize("n,V,d,dt", SHAPES)
def test_a_nan_row_stays_its_own(n, V, d, dt):
    """Forward, and dh, of the other rows; dT is NaN as a sum over the rows."""
    c = Case(12, n, V, d, dt)
    for o in both(c):
        c.h[3] = 0.5
        o.forward()
        o.backward()
        loss, lse, dh, _ = o.outputs()[:4]
        c.h[3, 0] = float("nan")
        o.forward()
        o.backward()
        keep = torch.arange(n, device=dev()) != 3
        assert bool(torch.isnan(o.lse[3]))
        assert same([loss[keep], lse[keep]], [o.loss[keep], o.lse[keep]])
        assert same([dh[keep]], [o.dh[keep]])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_no_rows(dt):
    V, d = 50, 40
    table = to(np.ones((V, d)), dt)
    handle = pg.make_table(CODE[dt], table, V)
    h = torch.empty(0, d, dtype=DT[dt], device=dev())
    e = torch.empty(0, device=dev())
    tok = torch.empty(0, dtype=torch.int32, device=dev())
    pg.pg_head_loss(h, handle, tok, e, e, None)
    dw = torch.full((V, d), 2.0, device=dev())
    pg.pg_head_loss_backward(h, handle, tok, e, e, h, dw, None, accumulate=1)
    assert bool((dw == 2).all())
    pg.pg_head_loss_backward(h, handle, tok, e, e, h, dw, None)
    assert bool((dw == 0).all())
    dw16 = torch.full((V, d), 2.0, dtype=torch.bfloat16, device=dev())
    k = torch.empty(0, 4, device=dev())
    pg.pg_head_distill(h, handle, k.int(), k, e, e, k, None)
    pg.pg_head_distill_backward(h, handle, k.int(), k, e, k, e, None, dw16, None)
    assert bool((dw16 == 0).all())


@pytest.mark.parametrize("n,V,d,dt", SHAPES)
@pytest.mark.parametrize("zloss", [False, True])
def test_parts_of_the_gradients_and_the_other_type(n, V, d, dt, zloss):
    c = Case(13, n, V, d, dt)
    for dw_dt in ("f32", "bf16"):
        o = Loss(c, some_targets(c.g, n, V), zloss, dw_dt)
        o.forward()
        rh, bh, rt, bt = grad_bounds(o, dw_dt)
        o.backward()
        within("dh", o.dh, rh, bh)
        within("dw", o.dw, rt, bt)
        o.dh.fill_(9.0)
        o.dw.fill_(9.0)
        o.backward(dh=False)
        within("dw alone", o.dw, rt, bt)
        assert bool((o.dh == 9).all())
        o.dw.fill_(9.0)
        o.backward(dw=False)
        within("dh alone", o.dh, rh, bh)
        assert bool((o.dw == 9).all())


@pytest.mark.parametrize("n,V,d,dt", SHAPES)
def test_gradient_of_a_tied_table(n, V, d, dt):
    """Embedding, norm, head: the table's gradient collects both of its uses."""
    c = Case(14, n, V, d, dt)
    code = CODE[dt]
    tok = c.g.integers(0, V, n)
    target = some_targets(c.g, n, V)
    x = torch.empty(n, d, dtype=DT[dt], device=dev())
    pg.pg_embed(c.handle, i32(tok), x, scale=3.0)
    gamma = f32(1 + 0.1 * c.g.normal(size=d))
    mean, rstd = torch.empty(n, device=dev()), torch.empty(n, device=dev())
    pg.pg_layer_norm(x, gamma, None, c.h if c.h.is_contiguous() else x, mean=mean, rstd=rstd)
    c.H = f64(c.h)
    c.z = oh.logits(c.H, c.T, 1.0)
    c.ez = np.abs(c.H) @ np.abs(c.T).T * products(dt, d) + 3 * U * np.abs(c.z)
    if dt == "f32":
        H, T = np.abs(c.H), np.abs(c.T)
        c.ez += 2.0 ** -39 * (H.sum(1)[:, None] * T.max() + H.max(1)[:, None] * T.sum(1)[None])
    o = Loss(c, target, dw="f32")
    o.forward()
    dw = o.dw
    rh, bh, rt, bt = grad_bounds(o, "f32")
    o.backward(dw=False)
    within("dh", o.dh, rh, bh)
    dx = torch.empty_like(x)
    dgamma = torch.empty(d, device=dev())
    wn = Workspace(pg.pg_layer_norm_workspace_size(n, d))
    pg.pg_layer_norm_backward(o.dh, x, gamma, mean, rstd, dx, dgamma, None, wn.ws)
    we = Workspace(pg.pg_embed_workspace_size(n, V, d))
    pg.pg_embed_backward_dense(dx, i32(tok), dw, we.ws, scale=3.0)
    first = f64(dw)
    o.backward(dh=False, accumulate=1)
    # one more rounding of the sum
    within("dw", f64(dw) - first, rt, bt + 2 * U * (np.abs(first) + np.abs(rt)))
    e = ot.embed_dense(f64(dx), tok, V, 3.0)
    np.testing.assert_allclose(first, e, rtol=1e-4, atol=1e-4 * np.abs(e).max())


def test_pieces_of_the_vocabulary_and_of_the_batch():
    """Many tokens against a wide table: 2 pieces of columns; more rows than a
    piece of the batch: 2 of those, the last one short; few tokens against many
    rows, several tiles a block; in bf16 and fp32, against float64."""
    g = torch.Generator(device="cuda").manual_seed(3)
    for n, V, d, dt in ((16500, 33001, 128, "bf16"), (33000, 20000, 64, "bf16"),
                        (9000, 33000, 32, "f32"), (33000, 300, 40, "f32"),
                        (33000, 301, 129, "bf16"), (32800, 300, 128, "bf16"),
                        (32800, 300, 40, "f32"), (100, 70001, 1024, "bf16"),
                        (40, 70000, 1024, "bf16"), (40, 40000, 1024, "f32")):
        h = torch.randn(n, d, device="cuda", generator=g).to(DT[dt])
        t = (torch.randn(V, d, device="cuda", generator=g) / d ** 0.5).to(DT[dt])
        tok = torch.randint(-1, V, (n,), device="cuda", generator=g, dtype=torch.int32)
        handle = pg.make_table(CODE[dt], t, V)
        loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        w = Workspace(pg.pg_head_loss_workspace_size(n, d, V, CODE[dt]))
        pg.pg_head_loss(h, handle, tok, loss, lse, w.ws)
        assert w.intact()
        dl = torch.randn(n, device="cuda", generator=g) / n
        dh, dw = torch.empty_like(h), torch.empty_like(t)
        w = Workspace(pg.pg_head_loss_backward_workspace_size(n, d, V, CODE[dt]))
        pg.pg_head_loss_backward(h, handle, tok, lse, dl, dh, dw, w.ws)
        assert w.intact()
        torch.cuda.synchronize()
        T, e = t.double(), products(dt, d)
        wt = torch.where(tok >= 0, dl, 0.0).double()
        rt, bt = torch.zeros_like(T), torch.zeros_like(T)
        # 2 (k m + 1000) u for a sum of m terms, k products each; dT over the tokens
        k = 2 if dt == "bf16" else 3
        sum_h, sum_t = 2 * (k * V + 1000) * U, 2 * (k * n + 1000) * U
        rel = 2.0 ** -11 if dt == "bf16" else 2.0 ** -22
        drop = 0 if dt == "bf16" else 3.1 * 2.0 ** -22
        B = wt.abs().max() * 2
        M = (2 * wt.abs()[:, None] * h.double().abs()).max()
        for a in range(0, n, 2048):
            b = min(n, a + 2048)
            H = h[a:b].double()
            z = H @ T.T.contiguous()
            ez = (H.abs() @ T.abs().T.contiguous()) * e + 3 * U * z.abs()
            if dt == "f32":
                ez += 2.0 ** -39 * (H.abs().sum(1)[:, None] * T.abs().max()
                                    + H.abs().max(1).values[:, None] * T.abs().sum(1)[None])
            ref = torch.logsumexp(z, 1)
            bl = ez.max(1).values + 4 * U * z.abs().max(1).values + 300 * U + 4 * U * ref.abs()
            assert bool(((lse[a:b].double() - ref).abs() <= bl).all())
            at = tok[a:b].long().clamp(min=0)[:, None]
            ce = torch.where(tok[a:b] >= 0, ref - z.gather(1, at)[:, 0], 0.0)
            assert bool(((loss[a:b].double() - ce).abs() <= bl + ez.max(1).values
                         + 2 * U * z.abs().max(1).values).all())
            L = lse[a:b].double()[:, None]
            p = (z - L).exp() * wt[a:b, None]
            ep = p.abs() * torch.expm1(ez + 6 * U * (z.abs() + L.abs()) + 16 * U)
            p.scatter_add_(1, at, -wt[a:b, None])
            ep += 8 * U * (p.abs() + p.abs())
            ep = ep + (p.abs() + ep) * rel + 2.0 ** -39 * B
            mag = p.abs() + ep
            rh = p @ T
            bh = ep @ T.abs() + (mag @ T.abs()) * (sum_h + drop) \
                + mag.sum(1, keepdim=True) * 2.0 ** -39 * T.abs().max()
            bh += HALF[dt] * (rh.abs() + bh) + 1e-30
            bad = (dh[a:b].double() - rh).abs() > bh
            assert not bool(bad.any()), (n, V, d, dt, a, int(bad.sum()))
            rt += p.T.contiguous() @ H
            bt += ep.T.contiguous() @ H.abs() + (mag.T.contiguous() @ H.abs()) * (sum_t + drop)
        bt += n * 2.0 ** -37 * M
        bt += HALF[dt] * (rt.abs() + bt) + 1e-30
        bad = (dw.double() - rt).abs() > bt
        assert not bool(bad.any()), (n, V, d, dt, int(bad.sum()))


@pytest.mark.parametrize("n,V,d,dt", SHAPES + [(2100, 5003, 128, "bf16")])
def test_equal_calls_give_equal_bits(n, V, d, dt):
    c = Case(15, n, V, d, dt)
    for o in both(c, 70):
        o.forward()
        o.backward()
        first = o.outputs()
        for w in (o.w1, o.w2):
            w.ws.fill_(0x3C)
        for t in (o.loss, o.lse, o.dh, o.dw):
            t.fill_(-1)
        o.forward()
        o.backward()
        assert same(first, o.outputs()) and o.w1.intact() and o.w2.intact()


@pytest.mark.parametrize("n,V,d,dt", SHAPES)
def test_captured_calls(n, V, d, dt):
    c = Case(16, n, V, d, dt)
    h0 = c.h.clone()
    for o in both(c):
        def step():
            o.forward()
            o.backward()
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for i in range(4):
            c.h.copy_(h0 * (1 + 0.25 * i))
            step()
            want = o.outputs()
            for t in (o.loss, o.lse, o.dh, o.dw):
                t.fill_(-1)
            junk = torch.randn(1 << 20, device="cuda").sum()     # eager work between replays
            graph.replay()
            torch.cuda.synchronize()
            assert same(want, o.outputs()), i
            del junk
        c.h.copy_(h0)


@pytest.mark.parametrize("n,V,d,dt", SHAPES)
def test_other_streams(n, V, d, dt):
    c = Case(17, n, V, d, dt)
    for o in both(c):
        o.forward()
        o.backward()
        torch.cuda.synchronize()
        want = o.outputs()
        for t in (o.loss, o.lse, o.dh, o.dw):
            t.fill_(-1)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        o.forward(stream=side)
        o.backward(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert same(want, o.outputs())
        with torch.cuda.stream(side):
            o.forward()
            o.backward()
        side.synchronize()
        assert same(want, o.outputs())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,d", [(50, 400, 96), (300, 900, 128)])
def test_values_of_very_different_sizes(n, V, d, dt):
    """Rows of h, of the table, and weights of rows over many powers of two."""
    c = Case(18, n, V, d, dt)
    g = np.random.default_rng(19)
    c.h.copy_(to(c.H * 2.0 ** g.integers(-30, 2, (n, 1)), dt))
    c.table.copy_(to(c.T * 2.0 ** g.integers(-12, 3, (V, 1)), dt))
    c.H, c.T = f64(c.h), f64(c.table)
    c.z = oh.logits(c.H, c.T, 1.0)
    H, T = np.abs(c.H), np.abs(c.T)
    c.ez = H @ T.T * products(dt, d) + 3 * U * np.abs(c.z) + 2.0 ** -39 * (
        H.sum(1)[:, None] * T.max() + H.max(1)[:, None] * T.sum(1)[None])
    o = Loss(c, some_targets(c.g, n, V))
    o.dl = f32(f64(o.dl) * 2.0 ** g.integers(-40, 20, n))
    o.forward()
    ref, lse = oh.loss(c.H, c.T, o.tok.cpu().numpy())
    b = c.lse_bound(c.z, c.ez, lse)
    within("lse", o.lse, lse, b)
    within("loss", o.loss, ref, b + c.ez.max(1) + 2 * U * np.abs(c.z).max(1))
    o.backward()
    rh, bh, rt, bt = grad_bounds(o)
    within("dh", o.dh, rh, bh)
    within("dw", o.dw, rt, bt)


@pytest.mark.parametrize("at", [0, 0.5, 1])
@pytest.mark.parametrize("n", [1, 30, 64])
@pytest.mark.parametrize("V,d", [(1001, 40), (9001, 77)])
def test_one_element_far_larger_than_the_rest(V, d, n, at):
    """The table's copies are placed by its largest element, wherever it stands."""
    c = Case(25, n, V, d, "f32")
    row, col = int(at * (V - 1)), int(at * (d - 1))
    c.h[:, col] = 0                                   # the logits do not see it
    c.table[row, col] = -2.0 ** 20
    c.H, c.T = f64(c.h), f64(c.table)
    H, T = np.abs(c.H), np.abs(c.T)
    c.z = oh.logits(c.H, c.T, 1.0)
    c.ez = H @ T.T * products("f32", d) + 3 * U * np.abs(c.z) + 2.0 ** -39 * (
        H.sum(1)[:, None] * T.max() + H.max(1)[:, None] * T.sum(1)[None])
    o = Loss(c, some_targets(c.g, n, V), zloss=True)
    o.lse.copy_(f32(oh.log_sum_exp(c.z)))
    for _ in range(2):
        o.backward()
        rh, bh, rt, bt = grad_bounds(o)
        within("dh", o.dh, rh, bh)
        within("dw", o.dw, rt, bt)
        c.table[row, col] = 2.0 ** 3                  # nothing of the call before stays
        c.T = f64(c.table)
    assert o.w2.intact()


@pytest.mark.parametrize("n", [30, 400])
def test_scale_undoes_large_operands(n):
    """Logits of order one from very large and very small operands; h . T itself
    has to lie in fp32's range (2^130, say, is no fp32 value, scaled or not)."""
    V, d = 700, 96
    c = Case(24, n, V, d, "f32")
    h0, t0 = c.h.clone(), c.table.clone()
    tok = some_targets(c.g, n, V)
    o = Loss(c, tok)
    o.forward()
    o.backward()
    want = o.outputs()
    # powers of two throughout: the same bits, but for the gradients' exponents
    for eh, et in ((40, 70), (-60, -50), (70, -75)):
        c.h.copy_(h0 * 2.0 ** eh)
        c.table.copy_(t0 * 2.0 ** et)
        c.scale = 2.0 ** -(eh + et)
        o.forward()
        # one more rounding of the scaled logits where they are single dot products
        for got, ref in zip((o.loss, o.lse), want[:2]):
            within("loss", got, f64(ref), 1e-5 * np.ones(n))


@pytest.mark.parametrize("n", [20, 300])
def test_flat_and_certain(n):
    """scale 0 makes every token as likely; large logits a certain one."""
    V, d = 1000, 128
    c = Case(20, n, V, d, "bf16", 0.0)
    tok = c.g.integers(0, V, n)
    o = Loss(c, tok)
    o.forward()
    within("lse", o.lse, np.full(n, np.log(V)), np.full(n, 230 * U + 8 * U))
    c = Case(21, n, V, d, "bf16")
    tok = c.g.integers(0, V, n)
    c.h.copy_(c.table[torch.from_numpy(tok).to(dev())] * 1000)
    o = Loss(c, tok)
    o.forward()
    o.backward()
    c.H = f64(c.h)
    c.z = oh.logits(c.H, c.T, 1.0)
    c.ez = np.abs(c.H) @ np.abs(c.T).T * products("bf16", d) + 3 * U * np.abs(c.z)
    ref, lse = oh.loss(c.H, c.T, tok)
    b = c.lse_bound(c.z, c.ez, lse)
    within("loss", o.loss, ref, 2 * b + c.ez.max(1))
    rh, bh, rt, bt = grad_bounds(o)
    within("dh", o.dh, rh, bh)
    within("dw", o.dw, rt, bt)


def test_unaligned_operands():
    """h, dh and dw that start on odd elements."""
    n, V, d = 300, 900, 128
    c = Case(22, n, V, d, "bf16")
    for shift in (1, 3):
        o = Loss(c, some_targets(c.g, n, V))
        room = torch.empty(n * d + 8, dtype=torch.bfloat16, device=dev())
        h = room[shift:shift + n * d].view(n, d)
        h.copy_(c.h)
        out = torch.full((n * d + 8,), 3.0, dtype=torch.bfloat16, device=dev())
        o.dh = out[shift:shift + n * d].view(n, d)
        wide = torch.full((V * d + 8,), 3.0, dtype=torch.bfloat16, device=dev())
        o.dw = wide[shift:shift + V * d].view(V, d)
        keep, c.h = c.h, h
        o.forward()
        o.backward()
        c.h = keep
        rh, bh, rt, bt = grad_bounds(o)
        within("dh", o.dh, rh, bh)
        within("dw", o.dw, rt, bt)
        assert bool((out[:shift] == 3).all()) and bool((out[shift + n * d:] == 3).all())
        assert bool((wide[:shift] == 3).all()) and bool((wide[shift + V * d:] == 3).all())


def test_binding_refuses_what_does_not_fit():
    n, V, d = 8, 30, 16
    c = Case(23, n, V, d, "bf16")
    o = Loss(c, some_targets(c.g, n, V))
    one = torch.zeros(n, device=dev())
    ok = dict(h=c.h, table=c.handle, targets=o.tok, loss=one, lse=one, workspace=o.w1.ws)
    for bad in (dict(targets=o.tok[:-1]), dict(targets=o.tok.long()), dict(loss=one.double()),
                dict(lse=one[::2]), dict(lse=None), dict(h=c.h.half()), dict(h=c.h[:, ::2]),
                dict(table=pg.make_table(pg.PG_BF16, c.table[:, :8].contiguous(), V)),
                dict(table=pg.make_table(pg.PG_BF16, c.table.float(), V)),
                dict(workspace=one), dict(loss=one.cpu())):
        with pytest.raises(ValueError):
            pg.pg_head_loss(**{**ok, **bad})
    with pytest.raises(pg.PagegramError):
        pg.pg_head_loss(**{**ok, "workspace": None})
    with pytest.raises(pg.PagegramError) as err:
        pg.pg_head_loss(**{**ok, "h": c.h.float()})
    assert err.value.status == pg.PG_EUNSUPPORTED
    back = dict(h=c.h, table=c.handle, targets=o.tok, lse=one, dloss=one, dh=o.dh, dw=o.dw,
                workspace=o.w2.ws)
    for bad in (dict(dh=o.dh.float()), dict(dh=o.dh[:-1]), dict(dw=o.dw[:-1]), dict(dw=o.dw.half()),
                dict(dlse=one[:-1]), dict(dloss=None)):
        with pytest.raises(ValueError):
            pg.pg_head_loss_backward(**{**back, **bad})
    for bad in (dict(dh=None, dw=None), dict(accumulate=1), dict(accumulate=2**32)):
        with pytest.raises(pg.PagegramError):
            pg.pg_head_loss_backward(**{**back, **bad})
    ids, t = torch.zeros(n, 3, dtype=torch.int32, device=dev()), torch.zeros(n, 3, device=dev())
    dis = dict(h=c.h, table=c.handle, ids=ids, teacher=t, loss=one, lse=one, logits=t.clone(),
               workspace=torch.empty(pg.pg_head_distill_workspace_size(n, d, V, 3, pg.PG_BF16),
                                     dtype=torch.uint8, device=dev()))
    for bad in (dict(ids=ids[:, :2]), dict(teacher=t[:, :2].contiguous()), dict(logits=t[:-1]),
                dict(ids=None), dict(ids=ids.long())):
        with pytest.raises(ValueError):
            pg.pg_head_distill(**{**dis, **bad})
    with pytest.raises(pg.PagegramError):
        pg.pg_head_distill(**{**dis, "temperature": 0.0})
