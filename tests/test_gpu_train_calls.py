"""Calls of the training-step entry points at the edges of their arguments."""
import pytest
import torch

import hashed_head_gram_amd as pg

pytestmark = pytest.mark.gpu


def dev():
    return torch.device("cuda:0")


def refused(call, status):
    with pytest.raises(pg.PagegramError) as err:
        call()
    assert err.value.status == status


def test_numbers_beyond_the_c_types_are_refused():
    """Each of these would be a call of ordinary size if the number were cut to its low bits."""
    G = torch.randn(2, 30, 50, device=dev())
    out = torch.empty(2, 30, 50, dtype=torch.bfloat16, device=dev())
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev())
    refused(lambda: pg.pg_orthogonalize(G, out, ws, steps=2**32 + 5), pg.PG_EINVAL)
    x = torch.randn(4, 64, device=dev())
    tok = torch.zeros(4, dtype=torch.int32, device=dev())
    table = torch.zeros(10, 64, device=dev())
    refused(lambda: pg.pg_embed_backward_dense(x, tok, table, ws, accumulate=2**32), pg.PG_EINVAL)
    refused(lambda: pg.pg_embed_backward(x, tok, 2**64 + 10, tok.long(), x.clone(), tok.long(), ws),
            pg.PG_ERANGE)
    # one row of 2^32 + 64 columns, 17 GB (its first half as bf16 is another)
    gamma = torch.empty(2**32 + 64, device=dev())
    row = gamma.view(torch.bfloat16)[:2**32 + 64].view(1, -1)
    refused(lambda: pg.pg_embed(pg.make_table(pg.PG_F32, table.data_ptr(), 10), tok[:1], row),
            pg.PG_EUNSUPPORTED)
    refused(lambda: pg.pg_layer_norm(row, gamma, None, row), pg.PG_EUNSUPPORTED)
    refused(lambda: pg.pg_embed_backward_dense(row, tok[:1], gamma.view(1, -1), ws),
            pg.PG_EUNSUPPORTED)


def test_no_workspace_where_none_is_needed():
    """A workspace of None is a null pointer: taken for no tokens and no rows, refused otherwise;
    other tensors that are missing are a ValueError."""
    x, tok = torch.randn(4, 8, device=dev()), torch.zeros(4, dtype=torch.int32, device=dev())
    s, one = torch.ones(4, device=dev()), torch.ones(8, device=dev())
    count = torch.full((1,), 7, device=dev())
    table = torch.ones(5, 8, device=dev())
    pg.pg_embed_backward(x[:0], tok[:0], 5, tok.long(), table, count, None)
    pg.pg_embed_backward_dense(x[:0], tok[:0], table, None)
    assert count.item() == 0 and bool((table == 0).all())
    dg, db = one.clone(), one.clone()
    pg.pg_layer_norm_backward(x[:0], x[:0], one, s[:0], s[:0], x[:0], dg, db, None)
    assert bool((dg == 0).all()) and bool((db == 0).all())
    refused(lambda: pg.pg_embed_backward(x, tok, 5, tok.long(), table, count, None), pg.PG_EINVAL)
    refused(lambda: pg.pg_embed_backward_dense(x, tok, table, None), pg.PG_EINVAL)
    refused(lambda: pg.pg_layer_norm_backward(x, x.clone(), one, s, s, x, dg, db, None), pg.PG_EINVAL)
    refused(lambda: pg.pg_orthogonalize(x, x.bfloat16(), None), pg.PG_EINVAL)
    for call in (lambda: pg.pg_layer_norm(x, None, None, x),
                 lambda: pg.pg_layer_norm(x, one, None, None),
                 lambda: pg.pg_layer_norm_backward(x, x.clone(), one, None, s, x, dg, db, None),
                 lambda: pg.pg_embed_backward(x, tok, 5, None, table, count, None),
                 lambda: pg.pg_orthogonalize(x, None, None)):
        with pytest.raises(ValueError):
            call()


def test_layer_norm_at_the_ends_of_fp32():
    """A row whose squares overflow has rstd 0, equal values without eps give NaN, and no row
    reaches another."""
    x = torch.randn(5, 300, device=dev())
    x[1] *= 1e25
    x[2] = 3.0
    x[3, 4] = float("inf")
    gamma, beta = torch.rand(300, device=dev()) + 0.5, torch.randn(300, device=dev())
    y, mean, rstd = torch.empty_like(x), torch.empty(5, device=dev()), torch.empty(5, device=dev())
    pg.pg_layer_norm(x, gamma, beta, y, eps=0.0, mean=mean, rstd=rstd)
    assert rstd[1] == 0 and torch.equal(y[1], beta)
    assert bool(torch.isnan(y[2:4]).all()) and bool(torch.isfinite(y[[0, 4]]).all())
    alone = torch.empty_like(x[:1])
    for i in (0, 4):
        pg.pg_layer_norm(x[i:i + 1], gamma, beta, alone, eps=0.0)
        assert torch.equal(alone[0], y[i])
