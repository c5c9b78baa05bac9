"""The head's losses at the ends of their sizes: the widest rows, tables past 2^32
bytes and 2^31 elements, rows of h and dh that lie 32 MB apart. Bounds are those of
test_gpu_head.py."""
import numpy as np
import pytest
import torch

import hashed_head_gram_amd as pg
from tests import test_gpu_head as basic
from tests.test_gpu_head import CODE, DT, HALF, U, Workspace, products

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 40, 130, 400])
@pytest.mark.parametrize("d", [16384, 16383])
def test_widest_rows(n, d, dt):
    basic.test_loss(n, 300, d, dt, 1.0, 1.0, 0)
    basic.test_loss_backward(n, 300, d, dt, 1.0, 1.0, 0, True)
    basic.test_distill_backward(n, 300, d, dt, 3, 1.0, 1.0, 1)


@pytest.mark.parametrize("n,V,d,dt", [(40, 1100000, 2048, "bf16"), (130, 1100000, 2048, "bf16"),
                                      (300, 1100000, 2048, "bf16"), (40, 600000, 2048, "f32"),
                                      (400, 600000, 2048, "f32")])
def test_table_past_32_bit_offsets(n, V, d, dt):
    """All rows of T but the first and the last 500 are zeros, so float64 has only
    those and one more, which stands for the others."""
    g = torch.Generator(device="cuda").manual_seed(71)
    m = 500
    code = CODE[dt]
    assert V * d * (2 if dt == "bf16" else 4) > 2 ** 32
    table = torch.zeros(V, d, dtype=DT[dt], device="cuda")
    for part in (table[:m], table[-m:]):
        part.copy_(torch.randn(m, d, device="cuda", generator=g) / d ** 0.5 * 3)
    handle = pg.make_table(code, table, V)
    h = torch.randn(n, d, device="cuda", generator=g).to(DT[dt])
    tok = torch.randint(V - m, V, (n,), device="cuda", generator=g, dtype=torch.int32)
    tok[::3] -= V - m
    tok[1] = V // 2
    T = torch.cat([table[:m], table[-m:], table[m:m + 1]]).double()
    count = torch.ones(2 * m + 1, dtype=torch.float64, device="cuda")
    count[-1] = V - 2 * m
    at = torch.where(tok < m, tok, torch.where(tok >= V - m, tok - (V - 2 * m), 2 * m)).long()[:, None]
    H = h.double()
    z = H @ T.T.contiguous()
    ez = (H.abs() @ T.T.abs().contiguous()) * products(dt, d) + 3 * U * z.abs()
    if dt == "f32":
        ez += 2.0 ** -39 * (H.abs().sum(1)[:, None] * T.abs().max()
                            + H.abs().max(1).values[:, None] * T.abs().sum(1)[None])
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    w = Workspace(pg.pg_head_loss_workspace_size(n, d, V, code))
    pg.pg_head_loss(h, handle, tok, loss, lse, w.ws)
    assert w.intact()
    ref = torch.logsumexp(z + count.log(), 1)
    bl = ez.max(1).values + 4 * U * z.abs().max(1).values + 420 * U + 4 * U * ref.abs()
    assert bool(((lse.double() - ref).abs() <= bl).all())
    off = (loss.double() - (ref - z.gather(1, at)[:, 0])).abs()
    assert bool((off <= bl + ez.max(1).values + 2 * U * z.abs().max(1).values).all())

    dl = (1 + torch.rand(n, device="cuda", generator=g)) / n
    dh, dw = torch.empty_like(h), torch.empty_like(table)
    del w
    w = Workspace(pg.pg_head_loss_backward_workspace_size(n, d, V, code))
    pg.pg_head_loss_backward(h, handle, tok, lse, dl, dh, dw, w.ws)
    assert w.intact()
    one = dt == "bf16"
    L, a = lse.double()[:, None], dl.double()[:, None]
    p = torch.exp(z - L) * a
    e = p * torch.expm1(ez + 6 * U * (z.abs() + L.abs()) + 16 * U)
    hit = torch.zeros_like(p).scatter_(1, at, a.expand(n, 1))
    # dT: a row of the zeros apart from the named one has no target
    dz = p - hit
    dz[:, -1] = p[:, -1]
    size = p + hit
    e = e + 8 * U * (dz.abs() + size) + (dz.abs() + e) * (2.0 ** -11 if one else 2.0 ** -22)
    # weights within a factor of two: rows' bounds within four
    e = e + 2.0 ** -19 * 4 * (dz.abs() + e).max(0).values + 3 * 2.0 ** -126
    k, drop = (2, 0) if one else (3, 3.1 * 2.0 ** -22)
    mag = dz.abs() + e
    want = dz.T.contiguous() @ H
    b = e.T.contiguous() @ H.abs() + (mag.T.contiguous() @ H.abs()) * (2 * (k * n + 1000) * U + drop) \
        + mag.sum(0)[:, None] * 2.0 ** -36 * H.abs().max()
    b += HALF[dt] * (want.abs() + b) + 1e-30
    got = torch.cat([dw[:m], dw[-m:], dw[m:m + 1]]).double()
    bad = (got - want).abs() > b
    assert not bool(bad.any()), ("dw", int(bad.sum()), bad.nonzero()[0].tolist())
    # every row of the zeros has the same gradient, but for the one named
    same = (dw[m:V - m] == dw[m]).all(1)
    same[V // 2 - m] = True
    assert bool(same.all()), same.logical_not().nonzero()[0].tolist()
    assert not bool((dw[V // 2] == dw[m]).all())
    # dh: zeros add nothing, however many
    dzh = p - hit
    dzh[:, -1] = 0
    e[:, -1] = 0
    want = dzh @ T
    mag = dzh.abs() + e
    b = e @ T.abs() + (mag @ T.abs()) * (2 * (k * V + 1000) * U + drop) \
        + mag.sum(1, keepdim=True) * 2.0 ** -38 * T.abs().max()
    b += HALF[dt] * (want.abs() + b) + 1e-30
    bad = (dh.double() - want).abs() > b
    assert not bool(bad.any()), ("dh", int(bad.sum()))


@pytest.mark.parametrize("n,dt", [(5, "bf16"), (70, "bf16"), (300, "bf16"), (40, "f32"), (330, "f32")])
def test_rows_far_apart(n, dt):
    """Strides beyond 2^24 elements: h is copied, not read in place; dh goes out at
    the same stride, and nothing between its rows changes."""
    V, d, ld = 700, 128, (1 << 24) + 8
    c = basic.Case(72, n, V, d, dt)
    room = torch.zeros((n - 1) * ld + d, dtype=DT[dt], device="cuda")
    far = room.as_strided((n, d), (ld, 1))
    far.copy_(c.h)
    tok = torch.from_numpy(basic.some_targets(c.g, n, V)).int().cuda()
    code = CODE[dt]
    dl = torch.rand(n, device="cuda") / n
    out = []
    for h in (c.h, far):
        loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        w = Workspace(pg.pg_head_loss_workspace_size(n, d, V, code))
        pg.pg_head_loss(h, c.handle, tok, loss, lse, w.ws)
        dh = torch.full_like(c.h, 3.0)
        if h is far:
            back = torch.full_like(room, 3.0)
            dh = back.as_strided((n, d), (ld, 1))
        dw = torch.empty_like(c.table)
        v = Workspace(pg.pg_head_loss_backward_workspace_size(n, d, V, code))
        pg.pg_head_loss_backward(h, c.handle, tok, lse, dl, dh, dw, v.ws)
        assert w.intact() and v.intact()
        out.append([loss, lse, dh.clone(), dw])
    for x, y in zip(*out):
        assert torch.equal(x, y)
    dh.fill_(3.0)
    assert bool((back == 3.0).all())
