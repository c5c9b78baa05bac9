"""The head's losses on the paths that only large or particular sizes take: copied
pieces of the table, pieces of the batch and of the vocabulary with every argument
that reaches them, more column tiles than entries are sorted by, and fp32 batches
beyond the few-token kernels. The limits (csrc/head_rows.h): fragments up to 320
rows forward (fp32), 128 (bf16 rows that cannot be read in place) and 64 backward;
copies of T by 256 MB, dz by 2^29 elements over both halves and 32,768 rows.

References are float64 on the GPU, row by row of the batch; bounds as in
test_gpu_head.py and test_gpu_head_range.py."""
import numpy as np
import pytest
import torch

import hashed_head_gram_amd as pg
from tests import test_gpu_head as basic
from tests import test_gpu_head_calls as calls
from tests.test_gpu_head import CODE, DT, HALF, U, Workspace, products

pytestmark = pytest.mark.gpu


class Big:
    """Operands on the GPU and their logits' error, a chunk of rows at a time."""

    def __init__(self, seed, n, V, d, dt, scale=1.0, pad=0, rare=0.0):
        self.g = g = torch.Generator(device="cuda").manual_seed(seed)
        self.n, self.V, self.d, self.dt, self.scale = n, V, d, dt, scale
        whole = torch.full((n, d + pad), 7.0, dtype=DT[dt], device="cuda")
        self.h = whole[:, :d]
        self.h.copy_(torch.randn(n, d, device="cuda", generator=g))
        t = torch.randn(V, d, device="cuda", generator=g) / d ** 0.5
        if rare:                           # every fifth row far below the others
            self.h[:, 0] = 1.0
            t[:, 0] = 0.0
            t[::5, 0] = -rare * (1 + torch.rand(len(t[::5]), device="cuda", generator=g))
        self.table = t.to(DT[dt])
        self.handle = pg.make_table(CODE[dt], self.table, V)
        self.T = self.table.double()
        self.Tt = self.T.T.contiguous()

    def chunks(self):
        step = max(1, int(4e7) // self.V)
        return [(a, min(self.n, a + step)) for a in range(0, self.n, step)]

    def logits(self, a, b):
        H = self.h[a:b].double()
        z = self.scale * (H @ self.Tt)
        ez = abs(self.scale) * (H.abs() @ self.Tt.abs()) * products(self.dt, self.d) \
            + 3 * U * z.abs()
        if self.dt == "f32":
            T = self.T.abs()
            ez += abs(self.scale) * 2.0 ** -39 * (H.abs().sum(1)[:, None] * T.max()
                                                  + H.abs().max(1).values[:, None] * T.sum(1)[None])
        return H, z, ez

    def check_forward(self, lse, inv_tau, ids, zk=None, loss=None):
        """lse, the logits at ids, and the cross entropy of one id a row."""
        for a, b in self.chunks():
            _, z, ez = self.logits(a, b)
            ref = torch.logsumexp(z * inv_tau, 1)
            # a sum of positive terms, its parts joined over the vocabulary: 400 deep at most
            bl = (ez.max(1).values + 4 * U * z.abs().max(1).values) * inv_tau + 420 * U \
                + 4 * U * ref.abs()
            assert bool(((lse[a:b].double() - ref).abs() <= bl).all()), ("lse", a)
            there = (ids[a:b] >= 0) & (ids[a:b] < self.V)
            at = torch.where(there, ids[a:b], 0).long()
            want, e = z.gather(1, at), ez.gather(1, at)
            if zk is not None:
                off = (zk[a:b].double() - torch.where(there, want, 0.0)).abs()
                assert bool((off <= torch.where(there, e, 0.0)).all()), ("logits", a)
            if loss is not None:
                ce = torch.where(there[:, 0], ref - want[:, 0], 0.0)
                bound = bl + ez.max(1).values + 2 * U * z.abs().max(1).values
                assert bool(((loss[a:b].double() - ce).abs() <= bound).all()), ("loss", a)

    def check_grads(self, a_n, w_n, lse, inv_tau, ids, share, dh, dw, first=None, slack=0.0):
        """dz = a exp(z / tau - lse) - w sum of share; slack: the shares' relative error."""
        one = self.dt == "bf16"
        a_n, w_n, L = a_n.double(), w_n.double(), lse.double()
        bound = a_n.abs() + w_n.abs()
        unit = torch.where(bound > 0, 2.0 ** torch.floor(torch.log2(bound.clamp(min=1e-300))), 1.0)
        there = (ids >= 0) & (ids < self.V)
        at = torch.where(there, ids, 0).long()
        val = torch.where(there, share.double(), 0.0) * w_n[:, None]

        def dz_of(a, b):
            H, z, ez = self.logits(a, b)
            l = L[a:b, None]
            p = torch.exp(z * inv_tau - l) * a_n[a:b, None]
            size = p.abs().scatter_add_(1, at[a:b], val[a:b].abs())
            p.scatter_add_(1, at[a:b], -val[a:b])
            e = size * torch.expm1(ez * inv_tau + slack + 6 * U * (z.abs() * inv_tau + l.abs())
                                   + 16 * U) + 8 * U * (p.abs() + size)
            e += (p.abs() + e) * (2.0 ** -11 if one else 2.0 ** -22)
            return H, p, e

        top = torch.zeros(self.V, dtype=torch.float64, device="cuda")
        for a, b in self.chunks():
            _, dz, e = dz_of(a, b)
            top = torch.maximum(top, ((dz.abs() + e) / unit[a:b, None]).max(0).values)
        k, drop = (2, 0) if one else (3, 3.1 * 2.0 ** -22)
        s, T = abs(self.scale), self.T
        ref_t, b_t = torch.zeros_like(T), torch.zeros_like(T)
        Hmax = (self.h.double().abs().max(1).values * unit).max()
        for a, b in self.chunks():
            H, dz, e = dz_of(a, b)
            # steps of 2^-19 of a vocabulary row's largest, in units of the row's bound,
            # but no more than 2^-39 of the bound where a column is not lifted
            e = e + 2.0 ** -19 * unit[a:b, None] * top[None] + 3 * 2.0 ** -126
            eh = torch.minimum(e, e - 2.0 ** -19 * unit[a:b, None] * top[None]
                               + 2.0 ** -38 * unit[a:b, None])
            mag = dz.abs() + e
            rh = self.scale * (dz @ T)
            bh = s * (eh @ T.abs() + (mag @ T.abs()) * (2 * (k * self.V + 1000) * U + drop))
            # T's copy: steps of 2^-39 of its largest, of each lifted row too
            bh += s * (mag.sum(1) + unit[a:b] * 2.0 ** -13 * self.V)[:, None] * 2.0 ** -38 * T.abs().max()
            bh += HALF[self.dt] * (rh.abs() + bh) + 1e-30
            off = (dh[a:b].double() - rh).abs() > bh
            assert not bool(off.any()), ("dh", a, int(off.sum()))
            ref_t += self.scale * (dz.T.contiguous() @ H)
            b_t += s * (e.T.contiguous() @ H.abs()
                        + (mag.T.contiguous() @ H.abs()) * (2 * (k * self.n + 1000) * U + drop))
            # h's copy: steps of 2^-39 of the largest of its elements times their row's unit
            b_t += s * ((mag / unit[a:b, None]).sum(0) * 2.0 ** -38 * Hmax)[:, None]
        if first is not None:
            ref_t += first.double()
            b_t += 2 * U * (first.double().abs() + ref_t.abs())
        b_t += (2.0 ** -24 if dw.dtype == torch.float32 else 2.0 ** -8) * (ref_t.abs() + b_t) + 1e-37
        off = (dw.double() - ref_t).abs() > b_t
        assert not bool(off.any()), ("dw", int(off.sum()), off.nonzero()[0].tolist())


def signs(c, n):
    """Weights within a factor of two, of either sign."""
    w = (1 + torch.rand(n, device="cuda", generator=c.g)) / n
    return torch.where(torch.rand(n, device="cuda", generator=c.g) < 0.5, -w, w)


def entries(c, k):
    """ids with some in the first and the last rows of the table, some named twice,
    short lists and rows without any, and the teacher's logits."""
    n, V = c.n, c.V
    ids = torch.randint(0, V, (n, k), device="cuda", generator=c.g, dtype=torch.int32)
    ids[::3, 0] = torch.arange(len(ids[::3]), device="cuda", dtype=torch.int32) % min(V, 300)
    ids[1::3, 0] = V - 1 - torch.arange(len(ids[1::3]), device="cuda", dtype=torch.int32) % min(V, 300)
    if k > 1:
        ids[::7, k - 1] = ids[::7, 0]
        ids[::11, k // 2:] = -1
    ids[::13] = V
    return ids, torch.randn(n, k, device="cuda", generator=c.g) * 2


def shares(ids, teacher, V, tau):
    there = (ids >= 0) & (ids < V)
    t = torch.where(there, teacher.double() / tau, -np.inf)
    return torch.softmax(t, 1).nan_to_num(0.0), there.any(1)


@pytest.mark.parametrize("n,V,d,dt", [
    (130, 140001, 1000, "bf16"),           # pieces of 131,072 rows, the last one ragged
    (330, 140001, 500, "f32"),
    (130, 400003, 500, "bf16"),            # of 262,144
    (130, 2100007, 32, "bf16"),            # more column tiles than entries are sorted by
])
def test_copied_pieces_of_the_table(n, V, d, dt):
    c = Big(51, n, V, d, dt)
    ids, teacher = entries(c, 9)
    ids[0, 1:5] = torch.tensor([131071, 131072, 131070, 131073])    # on both sides of a border
    for x in (262143, 262144, 1048575, 1048576, 2097151, 2097152):
        if x < V:
            ids[x % n, 2] = x
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    w = Workspace(pg.pg_head_loss_workspace_size(n, d, V, CODE[dt]))
    tok = ids[:, 2].contiguous()
    pg.pg_head_loss(c.h, c.handle, tok, loss, lse, w.ws)
    c.check_forward(lse, 1.0, tok[:, None], loss=loss)
    assert w.intact()
    zk = torch.full(ids.shape, 9.0, device="cuda")
    w = Workspace(pg.pg_head_distill_workspace_size(n, d, V, 9, CODE[dt]))
    pg.pg_head_distill(c.h, c.handle, ids, teacher, loss, lse, zk, w.ws, temperature=2.0)
    c.check_forward(lse, 0.5, ids, zk=zk)
    assert w.intact()
    # the loss from what was just checked
    q, some = shares(ids, teacher, V, 2.0)
    want = 4 * (torch.special.xlogy(q, q) - q * zk.double() / 2).sum(1) + 4 * lse.double() * some
    size = 4 * (1 + (q * (zk.double().abs() + 10)).sum(1) + lse.double().abs())
    assert bool(((loss.double() - want).abs() <= size * 2.0 ** -18).all())


@pytest.mark.parametrize("n,V,d,dt,k,pad,rare", [
    (33000, 20000, 64, "bf16", 3, 0, 0.0),     # two pieces of rows, two of the vocabulary
    (33000, 20001, 136, "bf16", 2, 8, 30.0),   # read in place, strided, rows that are lifted
    (33000, 9001, 40, "f32", 2, 1, 30.0),
    (16500, 40001, 128, "bf16", 5, 0, 0.0),    # vocabulary alone
    (40, 2200001, 16, "f32", 3, 0, 20.0),      # few tokens, two pieces
    (300, 1800001, 32, "bf16", 3, 3, 20.0),
])
def test_pieces_with_every_argument(n, V, d, dt, k, pad, rare):
    c = Big(52, n, V, d, dt, pad=pad, rare=rare)
    code = CODE[dt]
    # cross entropy with a gradient of lse, fp32 dT added to
    ids, teacher = entries(c, k)
    tok = ids[:, 0].contiguous()
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    w = Workspace(pg.pg_head_loss_workspace_size(n, d, V, code))
    pg.pg_head_loss(c.h, c.handle, tok, loss, lse, w.ws)
    c.check_forward(lse, 1.0, tok[:, None], loss=loss)
    dl, ds = signs(c, n), signs(c, n)
    ok = (tok >= 0) & (tok < V)
    w_n = torch.where(ok, dl, 0.0)
    a_n = w_n + ds
    whole = torch.full((n, d + pad), 3.0, dtype=DT[dt], device="cuda")
    first = torch.randn(V, d, device="cuda", generator=c.g) * 1e-6
    dw = first.clone()
    w = Workspace(pg.pg_head_loss_backward_workspace_size(n, d, V, code))
    pg.pg_head_loss_backward(c.h, c.handle, tok, lse, dl, whole[:, :d], dw, w.ws, dlse=ds,
                             accumulate=1)
    c.check_grads(a_n, w_n, lse, 1.0, tok[:, None], torch.ones(n, 1, device="cuda"), whole[:, :d],
                  dw, first=first)
    assert w.intact() and bool((whole[:, d:] == 3.0).all())
    # distillation, dT of bf16 and of fp32
    tau = 2.0
    zk = torch.empty(n, k, device="cuda")
    w = Workspace(pg.pg_head_distill_workspace_size(n, d, V, k, code))
    pg.pg_head_distill(c.h, c.handle, ids, teacher, loss, lse, zk, w.ws, temperature=tau)
    c.check_forward(lse, 1 / tau, ids, zk=zk)
    q, some = shares(ids, teacher, V, tau)
    w_n = torch.where(some, dl, 0.0) * tau
    for kind in (torch.bfloat16, torch.float32):
        dw = torch.full((V, d), 5.0, dtype=kind, device="cuda")
        w = Workspace(pg.pg_head_distill_backward_workspace_size(n, d, V, k, code))
        pg.pg_head_distill_backward(c.h, c.handle, ids, teacher, lse, zk, dl, whole[:, :d], dw, w.ws,
                                    temperature=tau)
        # shares of logits of at most 10: 2^-18
        c.check_grads(w_n, w_n, lse, 1 / tau, ids, q, whole[:, :d], dw, slack=2.0 ** -18)
        assert w.intact() and bool((whole[:, d:] == 3.0).all())


# fp32 beyond the few-token kernels, plain and with rows that are not whole vectors
TILED = [(400, 900, 72, "f32"), (330, 700, 129, "f32")]


@pytest.mark.parametrize("n,V,d,dt", TILED)
@pytest.mark.parametrize("test", [
    calls.test_rows_without_target_may_hold_anything, calls.test_nothing_to_learn,
    calls.test_a_nan_row_stays_its_own, calls.test_gradient_of_a_tied_table,
    calls.test_equal_calls_give_equal_bits, calls.test_captured_calls, calls.test_other_streams],
    ids=lambda t: t.__name__[5:])
def test_tiled_fp32_as_programs_call_it(test, n, V, d, dt):
    test(n, V, d, dt)


@pytest.mark.parametrize("n,V,d,dt", TILED)
def test_tiled_fp32_parts_of_the_gradients(n, V, d, dt):
    calls.test_parts_of_the_gradients_and_the_other_type(n, V, d, dt, True)


@pytest.mark.parametrize("n,V,d,dt", TILED)
@pytest.mark.parametrize("scale", [-1.0, -0.3])
def test_tiled_fp32_of_a_negative_scale(n, V, d, dt, scale):
    basic.test_loss(n, V, d, dt, scale, 1.0, 3)
    basic.test_loss_backward(n, V, d, dt, scale, 1.0, 3, True)
    basic.test_distill(n, V, d, dt, 9, 1.5, scale, 1)
    basic.test_distill_backward(n, V, d, dt, 9, 1.5, scale, 1)


@pytest.mark.parametrize("n,V,d", [(400, 900, 72), (700, 1300, 128)])
def test_tiled_fp32_values_of_very_different_sizes(n, V, d):
    calls.test_values_of_very_different_sizes(n, V, d, "f32")


@pytest.mark.parametrize("n,V,d,dt", [(40, 300, 96, "bf16"), (300, 900, 128, "bf16"),
                                      (50, 900, 72, "f32"), (400, 900, 72, "f32")])
def test_graphs_that_share_a_workspace(n, V, d, dt):
    """Two captured calls with one workspace, replayed in any order; and two calls at
    once on streams of their own, each with its own."""
    made = []
    for seed in (61, 62):
        c = basic.Case(seed, n, V, d, dt)
        made += calls.both(c)
    size = max(max(len(o.w1.ws), len(o.w2.ws)) for o in made)
    shared = Workspace(size)
    want, graphs = [], []
    for o in made:
        o.forward()
        o.backward()
        want.append(o.outputs())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(3):
        for s, o in zip(streams, made):
            s.wait_stream(torch.cuda.current_stream())
            o.forward(stream=s)
            o.backward(stream=s)
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        assert all(calls.same(x, o.outputs()) for x, o in zip(want, made))
    for o in made:
        o.w1.ws, o.w2.ws = shared.ws[:len(o.w1.ws)], shared.ws[:len(o.w2.ws)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o.forward()
            o.backward()
        graphs.append(g)
    for order in ((0, 1, 2, 3), (3, 1, 0, 2), (2, 2, 0, 1)):
        for i in order:
            for t in (made[i].loss, made[i].lse, made[i].dh, made[i].dw):
                t.fill_(-1)
            graphs[i].replay()
        torch.cuda.synchronize()
        junk = torch.randn(1 << 18, device="cuda").sum()
        assert all(calls.same(want[i], made[i].outputs()) for i in order)
        del junk
    assert shared.intact()


@pytest.mark.parametrize("n,V,d,dt", [(64, 3001, 64, "f32"), (63, 9001, 40, "f32"),
                                      (64, 3001, 128, "bf16"), (20, 8193, 33, "f32")])
def test_few_tokens_with_the_most_entries(n, V, d, dt):
    basic.test_distill(n, V, d, dt, 256, 2.0, 1.0, 0)
    basic.test_distill_backward(n, V, d, dt, 256, 2.0, 1.0, 0)
