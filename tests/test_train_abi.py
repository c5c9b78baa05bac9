"""Refusals of the training-step entry points, all without a GPU: the C ABI's
checks run before anything is enqueued, and the binding refuses tensors that
do not fit before it calls the library."""
import ctypes

import pytest
import torch

import hashed_head_gram_amd as pg

FAKE = 1 << 40          # aligned, never dereferenced by these calls
BIG = 1 << 50
E, U, R = pg.PG_EINVAL, pg.PG_EUNSUPPORTED, pg.PG_ERANGE
COEF = (3.4445, -4.7750, 2.0315)


def check(fn, good, bad):
    """Each (change, status) of bad turns the good arguments into an error."""
    f = getattr(pg.lib(), fn)
    for change, status in bad:
        args = {**good, **change}
        assert f(*args.values()) == status, (fn, change)


def table(dtype=pg.PG_BF16, data=FAKE, n=100):
    return ctypes.byref(pg.make_table(dtype, data, n))


def test_embed_refusals():
    good = dict(table=table(), d=64, scale=1.0, tokens=FAKE, n=5, dtype=pg.PG_F32, out=FAKE,
                ld=64, status=None, stream=None)
    check("pg_embed", good, [
        (dict(table=None), E), (dict(table=table(data=None)), E),
        (dict(table=table(data=FAKE + 8)), E), (dict(table=table(pg.PG_NF4)), U),
        (dict(table=table(9)), E), (dict(table=table(n=0)), E), (dict(table=table(n=-1)), E),
        (dict(table=table(n=2**31 - 1)), R), (dict(d=0), E), (dict(d=-1), E), (dict(d=16385), U),
        (dict(tokens=None), E), (dict(tokens=FAKE + 2), E), (dict(n=-1), E), (dict(n=1 << 26), R),
        (dict(dtype=pg.PG_NF4), E), (dict(dtype=7), E), (dict(out=None), E),
        (dict(out=FAKE + 2), E), (dict(ld=63), E), (dict(status=FAKE + 1), E)])
    check("pg_embed", {**good, "tokens": None, "out": None}, [(dict(n=0), pg.PG_OK)])


def test_embed_backward_refusals():
    need = pg.pg_embed_workspace_size(5, 100, 64)
    assert need > 0
    good = dict(dout=FAKE, dtype=pg.PG_BF16, ld=64, tokens=FAKE, n=5, V=100, d=64, scale=1.0,
                urows=FAKE, ugrad=FAKE, n_unique=FAKE, ws=FAKE, bytes=need, stream=None)
    common = [(dict(dout=None), E), (dict(dout=FAKE + 1), E), (dict(dtype=pg.PG_NF4), E),
              (dict(ld=63), E), (dict(tokens=None), E), (dict(n=-1), E), (dict(n=1 << 26), R),
              (dict(V=0), E), (dict(V=2**31 - 1), R), (dict(d=0), E), (dict(d=16385), U),
              (dict(ws=None), E), (dict(ws=FAKE + 128), E), (dict(bytes=need - 1), E)]
    check("pg_embed_backward", good, common + [
        (dict(urows=None), E), (dict(urows=FAKE + 4), E), (dict(ugrad=None), E),
        (dict(ugrad=FAKE + 2), E), (dict(n_unique=None), E), (dict(n_unique=FAKE + 4), E)])
    dense = dict(dout=FAKE, dtype=pg.PG_BF16, ld=64, tokens=FAKE, n=5, V=100, d=64, scale=1.0,
                 dtable=FAKE, accumulate=0, ws=FAKE, bytes=need, stream=None)
    check("pg_embed_backward_dense", dense, common + [
        (dict(dtable=None), E), (dict(dtable=FAKE + 2), E), (dict(accumulate=2), E)])
    check("pg_embed_backward_dense", {**dense, "dtable": None},
          [(dict(n=0, accumulate=1), pg.PG_OK), (dict(n=0), E)])
    for bad, status in (((-1, 5, 5), E), ((5, 0, 5), E), ((5, 5, 0), E), ((5, 5, 16385), U),
                        ((1 << 26, 5, 5), R), ((5, 2**31, 5), R)):
        with pytest.raises(pg.PagegramError) as err:
            pg.pg_embed_workspace_size(*bad)
        assert err.value.status == status


def test_layer_norm_refusals():
    good = dict(x=FAKE, dtype=pg.PG_BF16, n=5, d=64, ldx=64, gamma=FAKE, beta=FAKE, eps=1e-5,
                y=FAKE + 4096, ldy=64, mean=FAKE, rstd=FAKE, stream=None)
    check("pg_layer_norm", good, [
        (dict(x=None), E), (dict(x=FAKE + 1), E), (dict(dtype=pg.PG_NF4), E), (dict(n=-1), E),
        (dict(n=(1 << 31) + 1), R), (dict(d=0), E), (dict(d=16385), U), (dict(ldx=63), E),
        (dict(gamma=None), E), (dict(gamma=FAKE + 2), E), (dict(beta=FAKE + 2), E),
        (dict(eps=-1.0), E), (dict(eps=float("nan")), E), (dict(y=None), E), (dict(ldy=63), E),
        (dict(y=FAKE, ldx=64, ldy=65), E), (dict(mean=FAKE + 2), E), (dict(rstd=FAKE + 2), E)])
    check("pg_layer_norm", {**good, "x": None, "y": None, "gamma": None}, [(dict(n=0), pg.PG_OK)])
    need = pg.pg_layer_norm_workspace_size(5, 64)
    back = dict(dy=FAKE, lddy=64, x=FAKE + 4096, ldx=64, dtype=pg.PG_F32, n=5, d=64, gamma=FAKE,
                mean=FAKE, rstd=FAKE, add=FAKE + 8192, ldadd=64, dx=FAKE + 12288, lddx=64,
                dgamma=FAKE, dbeta=FAKE, ws=FAKE, bytes=need, stream=None)
    check("pg_layer_norm_backward", back, [
        (dict(dy=None), E), (dict(dy=FAKE + 2), E), (dict(lddy=63), E), (dict(x=None), E),
        (dict(ldx=63), E), (dict(dtype=5), E), (dict(n=-1), E), (dict(d=0), E),
        (dict(d=16385), U), (dict(gamma=None), E), (dict(mean=None), E), (dict(rstd=None), E),
        (dict(add=FAKE + 8194), E), (dict(ldadd=63), E), (dict(dx=None), E),
        (dict(dx=FAKE + 4096), E), (dict(dx=FAKE, lddx=65), E),
        (dict(dx=FAKE + 8192, lddx=65), E), (dict(lddx=63), E), (dict(dgamma=None), E),
        (dict(dbeta=FAKE + 2), E), (dict(ws=None), E), (dict(ws=FAKE + 128), E),
        (dict(bytes=need - 1), E)])
    for bad, status in (((-1, 5), E), ((5, 0), E), ((5, 16385), U)):
        with pytest.raises(pg.PagegramError) as err:
            pg.pg_layer_norm_workspace_size(*bad)
        assert err.value.status == status


def test_orthogonalize_refusals():
    need = pg.pg_orthogonalize_workspace_size(2, 30, 50)
    a, b, c = COEF
    good = dict(G=FAKE, dtype=pg.PG_F32, n=2, rows=30, cols=50, steps=5, a=a, b=b, c=c, eps=1e-7,
                scale=1.0, out=FAKE, ws=FAKE, bytes=need, stream=None)
    nan, inf = float("nan"), float("inf")
    check("pg_orthogonalize", good, [
        (dict(G=None), E), (dict(G=FAKE + 2), E), (dict(dtype=pg.PG_NF4), E), (dict(n=-1), E),
        (dict(n=65536), R), (dict(rows=0), E), (dict(cols=0), E), (dict(rows=16385), U),
        (dict(cols=16385), U), (dict(steps=0), E), (dict(steps=65), E), (dict(eps=-1e-9), E),
        (dict(eps=nan), E), (dict(out=None), E), (dict(out=FAKE + 1), E), (dict(ws=None), E),
        (dict(ws=FAKE + 128), E), (dict(bytes=need - 1), E),
        # iterates that would leave the range the fp16 copies hold
        (dict(a=10.0, b=0.0, c=0.0), U), (dict(a=nan), U), (dict(b=inf), U), (dict(c=nan), U),
        (dict(b=-150.0, c=149.0), U), (dict(a=-4.0, b=0.0, c=0.0), U)])
    # other admissible polynomials, and no matrices at all
    for coef in ((1.5, -0.5, 0.0), (1.875, -1.25, 0.375), (2.0, -1.5, 0.5)):
        check("pg_orthogonalize", {**good, **dict(zip("abc", coef))}, [(dict(n=0), pg.PG_OK)])
    for bad, status in (((-1, 5, 5), E), ((1, 0, 5), E), ((1, 5, 16385), U), ((65536, 5, 5), R),
                        ((65, 16384, 16384), R)):
        with pytest.raises(pg.PagegramError) as err:
            pg.pg_orthogonalize_workspace_size(*bad)
        assert err.value.status == status


def test_binding_refuses_tensors_off_the_gpu():
    x = torch.zeros(4, 8)
    tok = torch.zeros(4, dtype=torch.int32)
    ws = torch.zeros(0, dtype=torch.uint8)
    one = torch.zeros(8)
    with pytest.raises(ValueError, match="not on a GPU"):
        pg.pg_embed(pg.make_table(pg.PG_F32, x, 4), tok, x)
    with pytest.raises(ValueError, match="not on a GPU"):
        pg.pg_embed_backward(x, tok, 4, tok.long(), x, tok.long(), ws)
    with pytest.raises(ValueError, match="not on a GPU"):
        pg.pg_embed_backward_dense(x, tok, x, ws)
    with pytest.raises(ValueError, match="not on a GPU"):
        pg.pg_layer_norm(x, one, one, x)
    with pytest.raises(ValueError, match="not on a GPU"):
        pg.pg_layer_norm_backward(x, x, one, tok, tok, x, one, one, ws)
    with pytest.raises(ValueError, match="not on a GPU"):
        pg.pg_orthogonalize(x, x, ws)
