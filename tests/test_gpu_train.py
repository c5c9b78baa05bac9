"""GPU parity of the training-step operators (token embedding and its table
gradient, layer norm forward and backward, the orthogonalised update) against
the float64 oracle (oracle/train.py).

Bounds count roundings: u = 2^-24 for an fp32 operation, half a step of the
result's type at the end (bf16 2^-8, fp32 2^-24, relative). A sum of k terms
in any order is off by at most k u times the sum of their magnitudes; a sum
through a tree of depth h by h u.
"""
import numpy as np
import pytest
import torch

import hashed_head_gram_amd as pg
from oracle import train as ot

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
PGDT = {"f32": pg.PG_F32, "bf16": pg.PG_BF16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
COEF = (3.4445, -4.7750, 2.0315)


def dev():
    return torch.device("cuda:0")


def to(x, dt):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(dev()).to(DT[dt])


def f64(t):
    return t.detach().double().cpu().numpy()


def strided(n, d, dt, pad, fill, shift=0):
    """[n, d] view of rows d + pad wide, starting `shift` elements in, and the
    whole buffer it lies in."""
    whole = torch.full((n * (d + pad) + shift + 64,), fill, dtype=DT[dt], device=dev())
    return whole[shift:shift + n * (d + pad)].view(n, d + pad)[:, :d], whole


def untouched(view, whole, fill):
    """Every element of whole outside view still holds fill."""
    keep = view.clone()
    view.fill_(fill)
    ok = bool((whole == fill).all())
    view.copy_(keep)
    return ok


def within(got, ref, bound):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    over = np.abs(got - ref) - bound
    assert np.all(np.isfinite(got)) and np.all(over <= 0), \
        f"off by {np.max(np.abs(got - ref)):.3e}, {np.sum(over > 0)} over"


# ---------------------------------------------------------------------------
# Token embedding

EMBED = [  # n, V, d, table, out, pad, shift
    (1, 1, 1, "f32", "f32", 0, 0), (3, 7, 7, "bf16", "bf16", 1, 1), (5, 9, 8, "f32", "bf16", 0, 0),
    (33, 50, 64, "bf16", "f32", 3, 1), (257, 1000, 385, "f32", "f32", 0, 1),
    (64, 300, 513, "bf16", "bf16", 5, 3), (1000, 2000, 768, "bf16", "bf16", 0, 0),
    (40, 500, 2560, "f32", "bf16", 8, 0), (9, 20, 16384, "bf16", "bf16", 0, 0),
]


@pytest.mark.parametrize("n,V,d,table,out,pad,shift", EMBED)
def test_embed(n, V, d, table, out, pad, shift):
    rng = np.random.default_rng(n + d)
    T = to(rng.standard_normal((V, d)), table)
    tok = rng.integers(0, V, n)
    if n > 2:
        tok[1], tok[n // 2], tok[-1] = -1, V, 2**31 - 1
    tokens = torch.from_numpy(tok.astype(np.int32)).to(dev())
    y, whole = strided(n, d, out, pad, 7.0, shift)
    status = torch.zeros(1, dtype=torch.int32, device=dev())
    scale = float(np.float32(0.37))
    pg.pg_embed(pg.make_table(PGDT[table], T, V), tokens, y, scale=scale, dev_status=status)
    ref = ot.embed(f64(T), tok, scale)
    within(y, ref, np.abs(ref) * (HALF[out] + U32))
    assert untouched(y, whole, 7.0)
    assert status.item() == (1 if n > 2 else 0)


def test_embed_empty_and_non_finite():
    T = torch.tensor([[1.0, float("inf")], [float("nan"), -2.0]], device=dev())
    tab = pg.make_table(pg.PG_F32, T, 2)
    y = torch.empty(0, 2, device=dev())
    pg.pg_embed(tab, torch.empty(0, dtype=torch.int32, device=dev()), y)
    y = torch.empty(2, 2, dtype=torch.bfloat16, device=dev())
    pg.pg_embed(tab, torch.tensor([1, 0], dtype=torch.int32, device=dev()), y)
    assert torch.isnan(y[0, 0]) and y[0, 1] == -2 and y[1, 0] == 1 and y[1, 1] == float("inf")


def zipf(rng, n, V):
    p = np.arange(1, V + 1) ** -1.1
    return rng.permutation(V)[rng.choice(V, n, p=p / p.sum())]


TOKENS = {
    "zipf": zipf,
    "one_row": lambda rng, n, V: np.full(n, V - 1),
    "two_rows": lambda rng, n, V: (np.arange(n) % 2) * (V - 1),
    "distinct": lambda rng, n, V: rng.permutation(V)[:n],
    "runs": lambda rng, n, V: np.minimum(np.arange(n) // 65, V - 1),
    "none": lambda rng, n, V: np.where(np.arange(n) % 2, -5, V),
    "some": lambda rng, n, V: rng.integers(-V, 2 * V, n),
}
ROWS = [  # n, V, d, dtype, pad, shift, tokens
    (1, 1, 1, "f32", 0, 0, "one_row"), (1, 500, 64, "bf16", 0, 0, "distinct"),
    (7, 3, 7, "bf16", 1, 1, "some"), (64, 511, 385, "f32", 0, 1, "zipf"),
    (65, 512, 8, "f32", 0, 0, "one_row"), (300, 600, 513, "bf16", 3, 1, "runs"),
    (2049, 5000, 65, "f32", 0, 0, "zipf"), (4097, 262143, 24, "bf16", 0, 0, "zipf"),
    (2500, 262144, 16, "f32", 0, 0, "distinct"), (5000, 40, 520, "bf16", 0, 0, "two_rows"),
    (5000, 3, 130, "f32", 0, 0, "one_row"), (1000, 10, 40, "bf16", 0, 0, "none"),
    (9000, 700, 1025, "bf16", 7, 0, "some"), (20000, 128000, 2560, "bf16", 0, 0, "zipf"),
    (70000, 100, 33, "f32", 0, 0, "zipf"), (3, 5, 16384, "f32", 0, 0, "two_rows"),
    # both sides of each way to sort
    (1024, 900, 16, "f32", 0, 0, "zipf"), (1025, 900, 100, "bf16", 0, 0, "some"),
    (2048, 70000, 200, "f32", 0, 0, "zipf"), (4096, 70000, 96, "f32", 0, 0, "zipf"), (16384, 50304, 256, "bf16", 0, 0, "zipf"),
    (65536, 300, 9, "f32", 0, 0, "some"), (65537, 128000, 20, "bf16", 0, 0, "zipf"),
    (1 << 18, 512, 8, "bf16", 0, 0, "zipf"), ((1 << 18) + 1, 5000, 8, "f32", 0, 0, "some"),
    (300000, 300000, 5, "f32", 0, 0, "distinct"), (270000, 2, 12, "bf16", 0, 0, "two_rows"),
]


def rows_inputs(n, V, d, dtype, pad, shift, tokens):
    rng = np.random.default_rng(n * 7 + d)
    tok = TOKENS[tokens](rng, n, V).astype(np.int32)
    dout, _ = strided(n, d, dtype, pad, float("nan"), shift)
    dout.copy_(to(rng.standard_normal((n, d)), dtype))
    return tok, torch.from_numpy(tok).to(dev()), dout


@pytest.mark.parametrize("n,V,d,dtype,pad,shift,tokens", ROWS)
def test_embed_backward(n, V, d, dtype, pad, shift, tokens):
    print(f"[embed_backward] {n} {V} {d} {dtype} {tokens}", flush=True)
    tok, tokens_d, dout = rows_inputs(n, V, d, dtype, pad, shift, tokens)
    cap = min(n, V)
    ws = torch.full((pg.pg_embed_workspace_size(n, V, d),), 0xA5, dtype=torch.uint8, device=dev())
    urows = torch.full((cap + 1,), -9, dtype=torch.int64, device=dev())
    ugrad = torch.full((cap + 1, d), 3.5, device=dev())
    nu = torch.full((1,), -1, dtype=torch.int64, device=dev())
    scale = float(np.float32(1.3))
    pg.pg_embed_backward(dout, tokens_d, V, urows, ugrad, nu, ws, scale=scale)
    ref_rows, ref, cnt, mag = ot.embed_rows(f64(dout), tok, V, scale)
    k = nu.item()
    assert k == len(ref_rows)
    assert np.array_equal(urows[:k].cpu().numpy(), ref_rows)
    within(ugrad[:k], ref, (cnt[:, None] + 1) * U32 * mag)
    assert bool((urows[k:] == -9).all()) and bool((ugrad[k:] == 3.5).all())
    # equal calls give equal bits, whatever the workspace held
    again = torch.full_like(ugrad, 3.5)
    ws.zero_()
    pg.pg_embed_backward(dout, tokens_d, V, urows, again, nu, ws, scale=scale)
    assert torch.equal(again, ugrad)


@pytest.mark.parametrize("n,V,d,dtype,pad,shift,tokens",
                         [r for r in ROWS if r[1] * r[2] <= 20_000_000])
def test_embed_backward_dense(n, V, d, dtype, pad, shift, tokens):
    print(f"[embed_backward_dense] {n} {V} {d} {dtype} {tokens}", flush=True)
    tok, tokens_d, dout = rows_inputs(n, V, d, dtype, pad, shift, tokens)
    ws = torch.full((pg.pg_embed_workspace_size(n, V, d),), 0xA5, dtype=torch.uint8, device=dev())
    scale = float(np.float32(0.7))
    whole = torch.full((V * d + 8,), float("nan"), device=dev())
    pg.pg_embed_backward_dense(dout, tokens_d, whole[:V * d].view(V, d), ws, scale=scale)
    urows, grad, cnt, mag = ot.embed_rows(f64(dout), tok, V, scale)
    ref, bound = np.zeros((V, d)), np.zeros((V, d))
    ref[urows], bound[urows] = grad, (cnt[:, None] + 1) * U32 * mag
    within(whole[:V * d].view(V, d), ref, bound)
    assert bool(torch.isnan(whole[V * d:]).all())
    base = to(np.random.default_rng(5).standard_normal((V, d)), "f32")
    acc = base.clone()
    pg.pg_embed_backward_dense(dout, tokens_d, acc, ws, scale=scale, accumulate=1)
    total = f64(base) + ref
    within(acc, total, np.where(bound > 0, bound + U32 * np.abs(total) + U32 * bound, 0.0))
    left = np.setdiff1d(np.arange(V), urows)
    assert torch.equal(acc[left], base[left])


def test_embed_backward_empty():
    e = torch.empty(0, 4, device=dev())
    tok = torch.empty(0, dtype=torch.int32, device=dev())
    nu = torch.full((1,), 5, dtype=torch.int64, device=dev())
    ws = torch.empty(pg.pg_embed_workspace_size(0, 9, 4), dtype=torch.uint8, device=dev())
    pg.pg_embed_backward(e, tok, 9, tok.long(), e, nu, ws)
    assert nu.item() == 0
    dt = torch.full((9, 4), 2.0, device=dev())
    pg.pg_embed_backward_dense(e, tok, dt, ws, accumulate=1)
    assert bool((dt == 2).all())
    pg.pg_embed_backward_dense(e, tok, dt, ws)
    assert bool((dt == 0).all())


def test_embed_backward_non_finite_stays_in_its_row():
    n, V, d = 200, 10, 9
    tok = torch.arange(n, dtype=torch.int32, device=dev()) % V
    dout = torch.ones(n, d, device=dev())
    dout[13, 4] = float("nan")          # row 3
    dout[25, 0] = float("inf")          # row 5
    ws = torch.empty(pg.pg_embed_workspace_size(n, V, d), dtype=torch.uint8, device=dev())
    dt = torch.empty(V, d, device=dev())
    pg.pg_embed_backward_dense(dout, tok, dt, ws)
    want = torch.full((V, d), 20.0, device=dev())
    want[3, 4], want[5, 0] = float("nan"), float("inf")
    assert torch.equal(torch.nan_to_num(dt, nan=-1.0), torch.nan_to_num(want, nan=-1.0))


def test_embed_backward_of_the_largest_vocabulary():
    V, n, d = 2**31 - 2, 5000, 9
    rng = np.random.default_rng(4)
    tok = rng.integers(0, V, n).astype(np.int32)
    tok[::7] = tok[0]
    tok[1], tok[2], tok[3] = V - 1, -1, 2**31 - 1
    dout = to(rng.standard_normal((n, d)), "f32")
    urows = torch.zeros(n, dtype=torch.int64, device=dev())
    ugrad = torch.zeros(n, d, device=dev())
    nu = torch.zeros(1, dtype=torch.int64, device=dev())
    ws = torch.empty(pg.pg_embed_workspace_size(n, V, d), dtype=torch.uint8, device=dev())
    pg.pg_embed_backward(dout, torch.from_numpy(tok).to(dev()), V, urows, ugrad, nu, ws)
    ref_rows, ref, cnt, mag = ot.embed_rows(f64(dout), tok, V, 1.0)
    k = nu.item()
    assert np.array_equal(urows[:k].cpu().numpy(), ref_rows)
    within(ugrad[:k], ref, (cnt[:, None] + 1) * U32 * mag)


def test_rows_beyond_32_bit_offsets():
    """Row strides of 2^30 elements, and a table of 2.4 G elements."""
    g = torch.Generator(device=dev()).manual_seed(3)
    n, d, ld = 3, 520, 1 << 30
    buf = torch.empty(n * ld, dtype=torch.bfloat16, device=dev())
    wide = buf.view(n, ld)[:, :d]
    near = torch.randn(n, d, device=dev(), generator=g).bfloat16()
    wide.copy_(near)
    gamma = torch.ones(d, device=dev())
    y, mean, rstd = torch.empty_like(near), torch.empty(n, device=dev()), torch.empty(n, device=dev())
    pg.pg_layer_norm(near, gamma, None, y, mean=mean, rstd=rstd)
    pg.pg_layer_norm(wide, gamma, None, wide)
    assert torch.equal(wide, y)
    ws = torch.empty(pg.pg_layer_norm_workspace_size(n, d), dtype=torch.uint8, device=dev())
    dx, dg = torch.empty_like(near), torch.empty(d, device=dev())
    pg.pg_layer_norm_backward(near, near, gamma, mean, rstd, dx, dg, None, ws)
    wide.copy_(near)
    pg.pg_layer_norm_backward(wide, near, gamma, mean, rstd, wide, dg, None, ws)
    assert torch.equal(wide, dx)
    V, d = 1_200_000, 2048
    del buf, wide
    table = torch.zeros(V, d, dtype=torch.bfloat16, device=dev())
    tok = torch.tensor([V - 1, 0, V - 2, V - 1], dtype=torch.int32, device=dev())
    rows = torch.randn(4, d, device=dev(), generator=g).bfloat16()
    table[tok.long()] = rows
    out = torch.empty(4, d, dtype=torch.bfloat16, device=dev())
    pg.pg_embed(pg.make_table(pg.PG_BF16, table, V), tok, out)
    assert torch.equal(out, table[tok.long()])
    del table
    dt = torch.full((V, d), 3.0, device=dev())
    ws = torch.empty(pg.pg_embed_workspace_size(4, V, d), dtype=torch.uint8, device=dev())
    pg.pg_embed_backward_dense(rows, tok, dt, ws)
    assert torch.equal(dt[V - 1], rows[0].float() + rows[3].float())
    assert torch.equal(dt[0], rows[1].float()) and torch.equal(dt[V - 2], rows[2].float())
    assert int(torch.count_nonzero(dt)) <= 3 * d


# ---------------------------------------------------------------------------
# Layer norm

# widths at both sides of every row geometry, odd ones, strided and shifted
NORM = [(1, 1, "f32", 0, 0), (5, 2, "bf16", 0, 0), (3, 7, "bf16", 1, 1), (100, 64, "bf16", 0, 0),
        (33, 65, "f32", 0, 1), (17, 128, "f32", 0, 0), (9, 129, "bf16", 3, 1),
        (70, 256, "bf16", 0, 0), (70, 257, "f32", 0, 0), (129, 512, "bf16", 8, 0),
        (65, 513, "bf16", 0, 1), (37, 768, "bf16", 0, 0), (31, 1024, "f32", 0, 0),
        (600, 1001, "f32", 0, 1), (40, 1536, "bf16", 0, 0), (21, 1537, "f32", 1, 0),
        (33, 2048, "bf16", 0, 0), (50, 2560, "bf16", 0, 0), (50, 2560, "f32", 0, 0),
        (11, 2561, "bf16", 0, 1), (6, 4096, "f32", 0, 0), (5, 4100, "bf16", 0, 0),
        (4, 8192, "bf16", 0, 0), (3, 8199, "f32", 0, 1), (3, 16384, "bf16", 0, 0),
        (5000, 72, "bf16", 0, 0), (5003, 384, "f32", 0, 0), (600, 5001, "f32", 0, 1),
        (600, 12001, "f32", 0, 0), (520, 12001, "bf16", 1, 0)]
DEPTH = 66     # deepest row sum: 40 terms a lane, 6 lane steps, 16 waves, the division


def norm_inputs(n, d, dt, pad, shift):
    rng = np.random.default_rng(n * 3 + d)
    x, _ = strided(n, d, dt, pad, float("nan"), shift)
    x.copy_(to(rng.standard_normal((n, d)) * 2 + rng.standard_normal((n, 1)), dt))
    gamma = to(1 + 0.3 * rng.standard_normal(d), "f32")
    beta = to(rng.standard_normal(d), "f32")
    return rng, x, gamma, beta


@pytest.mark.parametrize("n,d,dt,pad,shift", NORM)
def test_layer_norm(n, d, dt, pad, shift):
    print(f"[layer_norm] {n} {d} {dt}", flush=True)
    _, x, gamma, beta = norm_inputs(n, d, dt, pad, shift)
    eps = float(np.float32(1e-5))
    y, whole = strided(n, d, dt, pad, 7.0, shift)
    mean = torch.empty(n, device=dev())
    rstd = torch.empty(n, device=dev())
    pg.pg_layer_norm(x, gamma, beta, y, eps=eps, mean=mean, rstd=rstd)
    X, g, b = f64(x), f64(gamma), f64(beta)
    ref, mu, rs = ot.layer_norm(X, g, b, eps)
    t = X - mu[:, None]
    dmu = DEPTH * U32 * np.abs(X).mean(1)
    dt_ = U32 * np.abs(t) + dmu[:, None]
    var = (t * t).mean(1)
    dvar = (2 * np.abs(t) * dt_ + dt_ ** 2).mean(1) + DEPTH * U32 * var
    drs = dvar / (2 * (var + eps)) + 4 * U32          # relative; second order in dvar below
    drs = drs + drs ** 2 * 2
    within(mean, mu, dmu + U32 * np.abs(mu))
    within(rstd, rs, rs * drs)
    raw = np.abs(t * rs[:, None] * g)
    err = np.abs(g) * rs[:, None] * dt_ + raw * (drs[:, None] + 4 * U32) + U32 * np.abs(ref)
    within(y, ref, err + HALF[dt] * (np.abs(ref) + err))
    assert untouched(y, whole, 7.0)
    # without beta and statistics, in place: the same rows
    y2 = torch.empty(n, d, dtype=DT[dt], device=dev())
    pg.pg_layer_norm(x, gamma, None, y2, eps=eps)
    z = x.clone()
    pg.pg_layer_norm(z, gamma, None, z, eps=eps)
    assert torch.equal(y2, z)
    e2 = err + U32 * np.abs(ref - b)
    within(y2, ref - b, e2 + HALF[dt] * (np.abs(ref - b) + e2))


@pytest.mark.parametrize("n,d,dt,pad,shift", NORM)
@pytest.mark.parametrize("add", [False, True])
def test_layer_norm_backward(n, d, dt, pad, shift, add):
    print(f"[layer_norm_backward] {n} {d} {dt} {add}", flush=True)
    rng, x, gamma, _ = norm_inputs(n, d, dt, pad, shift)
    _, mu64, rs64 = ot.layer_norm(f64(x), f64(gamma), None, 1e-5)
    mean, rstd = to(mu64, "f32"), to(rs64, "f32")
    dy, _ = strided(n, d, dt, pad, float("nan"), shift)
    dy.copy_(to(rng.standard_normal((n, d)), dt))
    res = to(rng.standard_normal((n, d)), dt) if add else None
    dx, whole = strided(n, d, dt, pad, 7.0, shift)
    dg = torch.full((d,), 9.0, device=dev())
    db = torch.full((d,), 9.0, device=dev())
    ws = torch.full((pg.pg_layer_norm_workspace_size(n, d),), 0xA5, dtype=torch.uint8,
                    device=dev())
    pg.pg_layer_norm_backward(dy, x, gamma, mean, rstd, dx, dg, db, ws, add=res)
    DY, g = f64(dy), f64(gamma)
    mu, rs = f64(mean)[:, None], f64(rstd)[:, None]
    ref, rdg, rdb = ot.layer_norm_backward(DY, f64(x), g, mu[:, 0], rs[:, 0],
                                           None if res is None else f64(res))
    xh = (f64(x) - mu) * rs
    gd = DY * g
    m1, m2 = gd.mean(1, keepdims=True), (gd * xh).mean(1, keepdims=True)
    dm1 = (DEPTH + 2) * U32 * np.abs(gd).mean(1, keepdims=True)
    dm2 = (DEPTH + 5) * U32 * np.abs(gd * xh).mean(1, keepdims=True)
    err = rs * (dm1 + np.abs(xh) * dm2 + 6 * U32 * (np.abs(gd) + np.abs(m1) + np.abs(xh * m2))) \
        + U32 * np.abs(ref)
    within(dx, ref, err + HALF[dt] * (np.abs(ref) + err))
    # rows a group visits, the groups of a block, the two levels of the join
    depth = 128 + n / 1024
    within(dg, rdg, (depth + 3) * U32 * np.abs(DY * xh).sum(0))
    within(db, rdb, depth * U32 * np.abs(DY).sum(0))
    assert untouched(dx, whole, 7.0)
    # dx in dy's place, and in add's; no dbeta
    for place in ("dy", "add") if add else ("dy",):
        src = dict(dy=dy.clone(), add=None if res is None else res.clone())
        pg.pg_layer_norm_backward(src["dy"], x, gamma, mean, rstd, src[place], db, None, ws,
                                  add=src["add"])
        assert torch.equal(src[place], dx) and torch.equal(db, dg)


def test_layer_norm_backward_against_differences():
    n, d, h = 6, 130, 2.0 ** -6
    rng, x, gamma, beta = norm_inputs(n, d, "f32", 0, 0)
    w = to(rng.standard_normal((n, d)), "f32")
    y = torch.empty_like(x)
    mean, rstd, dg, db = (torch.empty(k, device=dev()) for k in (n, n, d, d))
    ws = torch.empty(pg.pg_layer_norm_workspace_size(n, d), dtype=torch.uint8, device=dev())
    pg.pg_layer_norm(x, gamma, beta, y, mean=mean, rstd=rstd)
    dx = torch.empty_like(x)
    pg.pg_layer_norm_backward(w, x, gamma, mean, rstd, dx, dg, db, ws)

    def loss(x, g, b):
        pg.pg_layer_norm(x, g, b, y)
        return float((w.double() * y.double()).sum())

    # along random directions v: (f(x + h v) - f(x - h v)) / 2h against <grad, v>.
    # The third-order term is below h^2 times a few hundred; rounding of y
    # below 2 n d 2^-23 max|y w| / h
    slack = 2 * n * d * 2.0 ** -23 * 16 / h + 300 * h * h
    for k in range(3):
        v = to(rng.standard_normal((n, d)) / np.sqrt(n * d), "f32")
        num = (loss(x + h * v, gamma, beta) - loss(x - h * v, gamma, beta)) / (2 * h)
        assert abs(num - float((dx.double() * v.double()).sum())) < slack
        u = to(rng.standard_normal(d) / np.sqrt(d), "f32")
        num = (loss(x, gamma + h * u, beta) - loss(x, gamma - h * u, beta)) / (2 * h)
        assert abs(num - float((dg.double() * u.double()).sum())) < slack
        num = (loss(x, gamma, beta + h * u) - loss(x, gamma, beta - h * u)) / (2 * h)
        assert abs(num - float((db.double() * u.double()).sum())) < slack


def test_layer_norm_empty_constant_and_non_finite():
    d = 40
    gamma = torch.ones(d, device=dev())
    e = torch.empty(0, d, device=dev())
    s = torch.empty(0, device=dev())
    ws = torch.empty(0, dtype=torch.uint8, device=dev())
    dg, db = torch.full((d,), 3.0, device=dev()), torch.full((d,), 3.0, device=dev())
    pg.pg_layer_norm(e, gamma, None, e)
    pg.pg_layer_norm_backward(e, e, gamma, s, s, e, dg, db, ws)
    assert bool((dg == 0).all()) and bool((db == 0).all())
    x = torch.zeros(4, d, device=dev())
    x[1] = 5.0                                 # constant rows: zeros out
    x[2, 7] = float("nan")
    x[3, 1] = float("inf")
    y = torch.empty_like(x)
    pg.pg_layer_norm(x, gamma, None, y)
    assert bool((y[:2] == 0).all()) and bool(torch.isnan(y[2:]).all())


# ---------------------------------------------------------------------------
# Orthogonalised update

ORTHO = [(1, 1, 1, "f32"), (2, 1, 9, "f32"), (1, 5, 3, "bf16"), (3, 16, 16, "f32"),
         (1, 64, 128, "f32"), (2, 100, 37, "bf16"), (1, 129, 130, "f32"), (1, 257, 128, "bf16"),
         (2, 200, 333, "f32"), (1, 520, 390, "f32"), (1, 640, 1000, "bf16"), (5, 96, 160, "f32"),
         (1, 24, 700, "f32"), (1, 1500, 130, "f32"),
         (3, 64, 256, "f32"), (2, 63, 255, "bf16"), (1, 65, 256, "f32"), (2, 64, 257, "f32"),
         (7, 2, 2, "f32"), (300, 40, 64, "bf16"), (4, 65, 64, "f32"), (2, 129, 33, "f32"),
         # enough matrices for the larger tiles
         (200, 256, 256, "bf16"), (64, 256, 200, "f32"), (50, 300, 384, "bf16"),
         (65, 250, 500, "f32")]


def spectrum(rng, n, r, c):
    k = min(r, c)
    u, v = rng.standard_normal((n, r, k)), rng.standard_normal((n, k, c))
    s = np.arange(1, k + 1) ** -0.7
    G = (u * s) @ v
    return G + 0.02 * np.sqrt((G * G).mean()) * rng.standard_normal((n, r, c))


def ortho(G, **kw):
    n = int(np.prod(G.shape[:-2]))
    ws = torch.full((pg.pg_orthogonalize_workspace_size(n, *G.shape[-2:]),), 0xFF,
                    dtype=torch.uint8, device=dev())
    out = torch.full(G.shape, 9.0, dtype=torch.bfloat16, device=dev())
    pg.pg_orthogonalize(G, out, ws, **kw)
    return out


def check_ortho(got, G, steps=5, coef=COEF, eps=1e-7, scale=1.0):
    """Half a bf16 step of each value, and twice what the documented fp16
    storage alone moves the oracle: in the 2-norm, and for single values
    eight times its root mean square."""
    for g, o in zip(f64(G), f64(got)):
        ref = ot.newton_schulz(g, steps, coef, eps, scale)
        noise = ot.newton_schulz_half(g, steps, coef, eps, scale) - ref
        far = np.linalg.norm(o - ref)
        limit = 2.0 ** -8 * np.linalg.norm(ref) + 2 * np.linalg.norm(noise)
        assert far <= limit, f"{far / np.linalg.norm(ref):.2e} of {limit / np.linalg.norm(ref):.2e}"
        rms = np.sqrt((noise * noise).mean())
        within(o, ref, 2.0 ** -8 * np.abs(ref) + 2 * np.abs(noise).max() + 8 * rms + 1e-7)


@pytest.mark.parametrize("n,r,c,dt", ORTHO)
def test_orthogonalize(n, r, c, dt):
    print(f"[orthogonalize] {n} {r} {c} {dt}", flush=True)
    G = to(spectrum(np.random.default_rng(r + c), n, r, c) * 1e-3, dt)
    out = ortho(G)
    some = sorted({0, n // 2, n - 1}) if n > 5 else range(n)
    check_ortho(out[list(some)], G[list(some)])
    assert bool(torch.isfinite(out).all()) and torch.equal(ortho(G), out)


@pytest.mark.parametrize("shape", [(40, 70), (200, 150)])
def test_orthogonalize_arguments(shape):
    G = to(spectrum(np.random.default_rng(2), 2, *shape), "f32")
    check_ortho(ortho(G, steps=1), G, steps=1)
    check_ortho(ortho(G, steps=9, coef=(1.875, -1.25, 0.375), eps=0.5, scale=-0.2), G, 9,
                (1.875, -1.25, 0.375), 0.5, -0.2)
    check_ortho(ortho(G, steps=12, coef=(1.5, -0.5, 0.0)), G, 12, (1.5, -0.5, 0.0))
    # the norm is taken in a range that fp32 squares would leave
    for s in (2.0 ** 110, 2.0 ** -100):
        assert torch.equal(ortho(G * s, eps=0.0), ortho(G, eps=0.0))


@pytest.mark.parametrize("shape", [(40, 70), (200, 150)])
def test_orthogonalize_zero_and_non_finite_matrices(shape):
    G = to(spectrum(np.random.default_rng(2), 4, *shape), "f32")
    G[0] = 0
    G[1, 5, 6] = float("nan")
    G[3, 2, 3] = float("inf")
    out = ortho(G)
    assert bool((out[0] == 0).all())
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(out[3]).all())
    check_ortho(out[2:3], G[2:3])          # its neighbours do not reach it
    assert bool((ortho(G[:1], eps=0.0) == 0).all())


# ---------------------------------------------------------------------------
# Streams, graphs, and the operators together


def test_refusals_of_the_binding():
    x = torch.zeros(4, 8, device=dev())
    tok = torch.zeros(4, dtype=torch.int32, device=dev())
    one = torch.ones(8, device=dev())
    s = torch.zeros(4, device=dev())
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=dev())
    tab = pg.make_table(pg.PG_F32, x, 4)
    calls = [
        lambda: pg.pg_embed(tab, tok.long(), x), lambda: pg.pg_embed(tab, tok[:3], x),
        lambda: pg.pg_embed(tab, tok, x.half()), lambda: pg.pg_embed(tab, tok.cpu(), x),
        lambda: pg.pg_embed(tab, tok, x.t()[:, :4]),
        lambda: pg.pg_embed(tab, tok, torch.zeros(4, 7, device=dev())),
        lambda: pg.pg_embed(pg.make_table(pg.PG_BF16, x, 4), tok, x),
        lambda: pg.pg_embed_backward(x, tok, 4, tok, x, tok.long(), ws),
        lambda: pg.pg_embed_backward(x, tok, 4, tok.long(), x[:2], tok.long(), ws),
        lambda: pg.pg_embed_backward_dense(x, tok, x.t(), ws),
        lambda: pg.pg_layer_norm(x, one[:7], one, x), lambda: pg.pg_layer_norm(x, one, one, x[:3]),
        lambda: pg.pg_layer_norm(x, one.double(), one, x),
        lambda: pg.pg_layer_norm(x.t(), one[:4], None, x.t()),
        lambda: pg.pg_layer_norm(x, one, one, x, mean=s[:3]),
        lambda: pg.pg_layer_norm_backward(x, x.bfloat16(), one, s, s, x, one, one, ws),
        lambda: pg.pg_layer_norm_backward(x, x, one, s, s, x.clone(), one, one, ws.float()),
        lambda: pg.pg_orthogonalize(x, x, ws),
        lambda: pg.pg_orthogonalize(x.t(), x.t().bfloat16(), ws),
        lambda: pg.pg_orthogonalize(x, x[:2].bfloat16(), ws),
        lambda: pg.pg_orthogonalize(one, one.bfloat16(), ws),
    ]
    for k, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was taken")
    # broadcast rows: a row stride of zero
    wide = torch.zeros(1, 8, device=dev()).expand(4, 8)
    with pytest.raises(pg.PagegramError):
        pg.pg_layer_norm_backward(wide, x, one, s, s, x.clone(), one.clone(), None, ws)


class Step:
    """A training step around the memory: embed -> memory -> norm, back through
    all of it, and the update of W."""

    def __init__(self, seed, B=2, T=100, V=300, d=128, K=4, r=32):
        g = torch.Generator(device=dev()).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, device=dev(), generator=g)  # noqa: E731
        self.B, self.T, self.V, self.d = B, T, V, d
        self.N, self.E = B * T, 2 * K * r
        self.lay = pg.make_layout("pagegram", K, r, S=4, pages=[31, 29], hash_seed=7, pad_id=V)
        R = pg.pg_layout_rows(self.lay)
        self.mem = rnd(R, r).bfloat16()
        self.table = pg.make_table(pg.PG_BF16, self.mem, R)
        self.fuse = pg.make_fuse(pg.PG_GATE_SCALAR, pg.PG_BF16, d, g=0.5)
        self.tokens = torch.randint(0, V, (B, T), device=dev(), generator=g).int()
        self.cmap = torch.arange(V, device=dev(), dtype=torch.int32)
        self.emb = rnd(V, d)
        self.W = (0.05 * rnd(d, self.E)).bfloat16()
        self.gamma, self.beta = 1 + 0.1 * rnd(d), rnd(d)
        self.dz, self.dres = rnd(self.N, d).bfloat16(), rnd(self.N, d).bfloat16()
        N, E, L = self.N, self.E, self.N * 2 * K
        e = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device=dev())  # noqa: E731
        self.x, self.h, self.z, self.dx = (e(N, d, dt=torch.bfloat16) for _ in range(4))
        self.e = e(N, E, dt=torch.bfloat16)
        self.rows, self.signs = e(N, 2, K, dt=torch.int64), e(N, 2, K, 1, dt=torch.int64)
        self.mean, self.rstd, self.dgamma, self.dbeta = e(N), e(N), e(d), e(d)
        self.dW, self.de = e(d, E), e(N, E)
        self.murows, self.mugrad = e(L, dt=torch.int64), e(L, r)
        self.mn, self.en = e(1, dt=torch.int64), e(1, dt=torch.int64)
        cap = min(N, V)
        self.eurows, self.eugrad = e(cap, dt=torch.int64), e(cap, d)
        self.demb = e(V, d)
        self.upd = e(d, E, dt=torch.bfloat16)
        size = max(pg.pg_workspace_size(self.lay, self.fuse, B, T),
                   pg.pg_backward_workspace_size(self.lay, self.fuse, B, T),
                   pg.pg_embed_workspace_size(N, V, d), pg.pg_layer_norm_workspace_size(N, d),
                   pg.pg_orthogonalize_workspace_size(1, d, E))
        self.ws = e(size, dt=torch.uint8)

    def run(self):
        tok = self.tokens.view(-1)
        pg.pg_embed(pg.make_table(pg.PG_F32, self.emb, self.V), tok, self.x, scale=2.0)
        pg.pg_index(self.lay, self.tokens, self.cmap, self.rows, self.signs)
        pg.pg_gather(self.lay, self.table, self.rows, self.signs, pg.PG_BF16, self.e)
        pg.pg_project_gate(self.fuse, self.e, self.B, self.T, self.W, self.x, self.h, self.ws)
        pg.pg_layer_norm(self.h, self.gamma, self.beta, self.z, mean=self.mean, rstd=self.rstd)
        pg.pg_layer_norm_backward(self.dz, self.h, self.gamma, self.mean, self.rstd, self.dx,
                                  self.dgamma, self.dbeta, self.ws, add=self.dres)
        pg.pg_backward_scalar(self.lay, self.fuse, self.rows, self.signs, self.e, self.dx, self.W,
                              self.B, self.T, self.dW, self.de, self.murows, self.mugrad, self.mn,
                              self.ws)
        pg.pg_embed_backward(self.dx, tok, self.V, self.eurows, self.eugrad, self.en, self.ws,
                             scale=2.0)
        pg.pg_embed_backward_dense(self.dx, tok, self.demb, self.ws, scale=2.0)
        pg.pg_orthogonalize(self.dW, self.upd, self.ws)

    def results(self):
        return [t.clone() for t in (self.x, self.h, self.z, self.mean, self.rstd, self.dx,
                                    self.dgamma, self.dbeta, self.dW, self.eurows, self.eugrad,
                                    self.en, self.demb, self.upd)]


def test_training_step_together():
    """Each operator's result from what the one before it left, and the table
    gradient through the row-wise optimiser of the memory."""
    s = Step(1)
    s.run()
    tok = s.tokens.view(-1).cpu().numpy()
    ref = ot.embed(f64(s.emb), tok, 2.0)
    within(s.x, ref, np.abs(ref) * (HALF["bf16"] + U32))
    ref, mu, rs = ot.layer_norm(f64(s.h), f64(s.gamma), f64(s.beta), 1e-5)
    within(s.z, ref, 2.0 ** -8 * np.abs(ref) + 1e-5)
    dx, dg, db = ot.layer_norm_backward(f64(s.dz), f64(s.h), f64(s.gamma), mu, rs, f64(s.dres))
    within(s.dx, dx, 2.0 ** -8 * np.abs(dx) + 1e-4)
    urows, grad, cnt, mag = ot.embed_rows(f64(s.dx), tok, s.V, 2.0)
    k = s.en.item()
    assert np.array_equal(s.eurows[:k].cpu().numpy(), urows)
    within(s.eugrad[:k], grad, (cnt[:, None] + 1) * U32 * mag)
    assert torch.equal(s.demb[s.eurows[:k]], s.eugrad[:k])
    check_ortho(s.upd[None], s.dW[None])
    # the embedding's touched rows feed pg_row_rms_step: a flat layout of V
    # rows (one order, one head, one slot)
    flat = pg.make_layout("pagegram", 1, s.d, S=1, pages=[s.V], n_min=1, n_max=1)
    assert pg.pg_layout_rows(flat) == s.V
    theta, vhat = s.emb.clone(), torch.zeros(s.V, device=dev())
    last = torch.zeros(s.V, dtype=torch.int64, device=dev())
    pg.pg_row_rms_step(flat, s.eurows, s.eugrad, s.en, len(s.eurows), theta, vhat, last, 1,
                       lr=0.01)
    from oracle import backward as ob
    want, v64, _ = ob.rms_step_sparse(f64(s.emb), np.zeros(s.V), np.zeros(s.V, np.int64), urows,
                                      f64(s.eugrad[:k]), 1, 0.01, 0.95, 0.0, 1e-8)
    assert np.max(np.abs(f64(theta) - want)) < 1e-5


def test_explicit_stream():
    """stream= overrides the current stream (a torch stream or its handle)."""
    x = torch.randn(7, 40, device=dev())
    gamma = torch.rand(40, device=dev())
    want = torch.empty_like(x)
    pg.pg_layer_norm(x, gamma, None, want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for how in (s, s.cuda_stream):
        y = torch.zeros_like(x)
        torch.cuda.synchronize()
        pg.pg_layer_norm(x, gamma, None, y, stream=how)
        s.synchronize()
        assert torch.equal(y, want)


def test_training_step_captured_and_on_another_stream():
    """The captured step replays to the eager result, with eager work on the
    same buffers in between; a second step runs on its own stream meanwhile."""
    a, b = Step(2), Step(3, B=1, T=77, d=192)
    a.run()
    b.run()
    want_a, want_b = a.results(), b.results()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a.run()
    for k in range(3):
        for t in (a.upd, a.demb, a.eugrad, a.dx, a.z, a.dgamma, a.ws):
            t.zero_()
        graph.replay()
        with torch.cuda.stream(stream):
            for t in (b.upd, b.demb, b.dx, b.ws):
                t.zero_()
            b.run()
        torch.cuda.synchronize()
        for got, want in ((a.results(), want_a), (b.results(), want_b)):
            for i, (x, y) in enumerate(zip(got, want)):
                assert torch.equal(x, y), (k, i)
        a.run()                                     # eager, between replays
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(a.results(), want_a)):
            assert torch.equal(x, y), (k, i)
