"""Refusals of the head's entry points and their workspace sizes, all without a
GPU: the C ABI's checks run before anything is enqueued, and the binding refuses
tensors that do not fit before it calls the library."""
import ctypes

import pytest
import torch

import hashed_head_gram_amd as pg

FAKE = 1 << 40          # aligned, never dereferenced by these calls
E, U, R = pg.PG_EINVAL, pg.PG_EUNSUPPORTED, pg.PG_ERANGE
NAN, INF = float("nan"), float("inf")
B, F = pg.PG_BF16, pg.PG_F32


def check(fn, good, bad):
    """Each (change, status) of bad turns the good arguments into an error."""
    f = getattr(pg.lib(), fn)
    for change, status in bad:
        args = {**good, **change}
        assert f(*args.values()) == status, (fn, change)


def table(dtype=B, data=FAKE, n=100):
    return ctypes.byref(pg.make_table(dtype, data, n))


COMMON = [
    (dict(h=None), E), (dict(h=FAKE + 1), E), (dict(dtype=pg.PG_NF4), E), (dict(dtype=F), U),
    (dict(n=-1), E), (dict(n=1 << 26), R), (dict(d=0), E), (dict(d=-1), E), (dict(d=16385, ld=16385), U),
    (dict(ld=63), E), (dict(table=None), E), (dict(table=table(data=None)), E),
    (dict(table=table(data=FAKE + 8)), E), (dict(table=table(pg.PG_NF4)), U),
    (dict(table=table(9)), E), (dict(table=table(F)), U), (dict(table=table(n=0)), E),
    (dict(table=table(n=-5)), E), (dict(table=table(n=2**31 - 1)), R),
    (dict(n=(1 << 26) - 1, table=table(n=2**31 - 2)), R),
    (dict(scale=NAN), E), (dict(scale=INF), E), (dict(lse=None), E),
    (dict(lse=FAKE + 2), E), (dict(ws=None), E), (dict(ws=FAKE + 128), E)]
GRADS = [
    (dict(dh=None, dw=None), E), (dict(dh=FAKE + 1), E), (dict(ld_dh=63), E), (dict(dw=FAKE + 1), E),
    (dict(dw_dtype=pg.PG_NF4), E), (dict(dw_dtype=F, dw=FAKE + 2), E), (dict(accumulate=2), E),
    (dict(accumulate=-1), E), (dict(accumulate=1), U), (dict(dloss=None), E),
    (dict(dloss=FAKE + 2), E)]
TAU = [(dict(tau=0.0), E), (dict(tau=-1.0), E), (dict(tau=NAN), E), (dict(tau=INF), E),
       (dict(tau=1e-45), E), (dict(k=0), E), (dict(k=-1), E), (dict(k=257), U)]


def test_loss_refusals():
    need = pg.pg_head_loss_workspace_size(5, 64, 100, B)
    good = dict(h=FAKE, dtype=B, n=5, d=64, ld=64, table=table(), scale=1.0, targets=FAKE,
                loss=FAKE, lse=FAKE, ws=FAKE, bytes=need, stream=None)
    check("pg_head_loss", good, COMMON + [
        (dict(scale=3e38), E),
        (dict(targets=None), E), (dict(targets=FAKE + 2), E), (dict(loss=None), E),
        (dict(loss=FAKE + 1), E), (dict(bytes=need - 1), E)])
    none = dict(h=None, n=0, targets=None, loss=None, lse=None, ws=None, bytes=0)
    check("pg_head_loss", {**good, **none}, [({}, pg.PG_OK), (dict(d=0), E), (dict(scale=NAN), E)])


def test_loss_backward_refusals():
    need = pg.pg_head_loss_backward_workspace_size(5, 64, 100, B)
    good = dict(h=FAKE, dtype=B, n=5, d=64, ld=64, table=table(), scale=1.0, targets=FAKE, lse=FAKE,
                dloss=FAKE, dlse=None, dh=FAKE, ld_dh=64, dw=FAKE, dw_dtype=B, accumulate=0, ws=FAKE,
                bytes=1 << 40, stream=None)
    check("pg_head_loss_backward", good, COMMON + GRADS + [
        (dict(targets=None), E), (dict(targets=FAKE + 2), E), (dict(dlse=FAKE + 2), E),
        (dict(bytes=1024), E)])
    assert need > 1024
    # nothing to do: no rows and the gradient added
    none = dict(h=None, n=0, targets=None, lse=None, dloss=None, ws=None, bytes=0)
    check("pg_head_loss_backward", {**good, **none},
          [(dict(accumulate=1, dw_dtype=F), pg.PG_OK), (dict(dw=None), pg.PG_OK)])


def test_distill_refusals():
    need = pg.pg_head_distill_workspace_size(5, 64, 100, 7, B)
    good = dict(h=FAKE, dtype=B, n=5, d=64, ld=64, table=table(), scale=1.0, ids=FAKE, teacher=FAKE,
                k=7, tau=2.0, loss=FAKE, lse=FAKE, logits=FAKE, ws=FAKE, bytes=need, stream=None)
    own = [(dict(ids=None), E), (dict(ids=FAKE + 2), E), (dict(teacher=None), E),
           (dict(teacher=FAKE + 2), E), (dict(logits=None), E), (dict(logits=FAKE + 1), E)]
    check("pg_head_distill", good, COMMON + TAU + own + [
        (dict(loss=None), E), (dict(bytes=need - 1), E)])
    back = dict(h=FAKE, dtype=B, n=5, d=64, ld=64, table=table(), scale=1.0, ids=FAKE, teacher=FAKE,
                k=7, tau=2.0, lse=FAKE, logits=FAKE, dloss=FAKE, dh=FAKE, ld_dh=64, dw=FAKE,
                dw_dtype=B, accumulate=0, ws=FAKE, bytes=1 << 40, stream=None)
    check("pg_head_distill_backward", back, COMMON + TAU + own + GRADS + [(dict(bytes=1024), E)])


SIZES = ["pg_head_loss_workspace_size", "pg_head_loss_backward_workspace_size",
         "pg_head_distill_workspace_size", "pg_head_distill_backward_workspace_size"]


@pytest.mark.parametrize("fn", SIZES)
def test_sizes_are_refused_like_the_calls(fn):
    f = getattr(pg, fn)
    k = (7,) if "distill" in fn else ()

    def size(n, d, V, dtype):
        return f(n, d, V, *k, dtype)

    assert size(0, 64, 100, B) >= 0
    for bad, status in (((-1, 5, 5, B), E), ((5, 0, 5, B), E), ((5, 5, 0, B), E),
                        ((5, 5, 5, pg.PG_NF4), E), ((5, 5, 5, 9), E), ((5, 16385, 5, F), U),
                        ((1 << 26, 5, 5, F), R), ((5, 5, 2**31, F), R),
                        ((2**70, 5, 5, F), R), ((5, 2**40, 5, F), U),
                        (((1 << 26) - 1, 5, 2**31 - 2, B), R)):
        with pytest.raises(pg.PagegramError) as err:
            size(*bad)
        assert err.value.status == status, bad
    if k:
        for kk, status in ((0, E), (257, U), (2**40, U)):
            with pytest.raises(pg.PagegramError) as err:
                f(5, 5, 5, kk, B)
            assert err.value.status == status


@pytest.mark.parametrize("fn", SIZES)
@pytest.mark.parametrize("V,d,dtype", [(100, 64, F), (50304, 768, B), (128000, 2560, B),
                                       (50303, 385, F), (128000, 33, B)])
def test_workspace_of_the_largest_batch_serves_every_smaller_one(fn, V, d, dtype):
    k = (9,) if "distill" in fn else ()
    last = 0
    for n in (0, 1, 31, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 4095, 4096, 5000, 16384, 16385,
              30000, 32768, 32769, 40000, 131072):
        size = getattr(pg, fn)(n, d, V, *k, dtype)
        assert size >= last, n
        last = size


def test_binding_refuses_tensors_off_the_gpu():
    x, one = torch.zeros(4, 8), torch.zeros(4)
    tok, ids = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32)
    t, ws = pg.make_table(F, x, 4), torch.zeros(0, dtype=torch.uint8)
    z = torch.zeros(4, 2)
    for call in (lambda h: pg.pg_head_loss(h, t, tok, one, one, ws),
                 lambda h: pg.pg_head_loss_backward(h, t, tok, one, one, x, x, ws),
                 lambda h: pg.pg_head_distill(h, t, ids, z, one, one, z, ws),
                 lambda h: pg.pg_head_distill_backward(h, t, ids, z, one, z, one, x, x, ws)):
        for h in (x, None):
            with pytest.raises(ValueError, match="not on a GPU"):
                call(h)
