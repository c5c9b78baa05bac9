"""Calls of the training-step entry points that the documentation allows (or
refuses) and that need no GPU: workspaces sized for a largest batch,
coefficients at the edge of what is taken, numbers beyond the C types."""
import pytest

import hashed_head_gram_amd as pg


@pytest.mark.parametrize("V,d", [(128000, 768), (128000, 2560), (50304, 64), (300, 200),
                                 (2**31 - 2, 16384), (1000, 1), (5, 5000)])
def test_embed_workspace_of_the_largest_batch_serves_every_smaller_one(V, d):
    sizes = sorted({*range(1, 3000, 7),
                    *(b + k for b in (4096, 8192, 16384, 26240, 32768, 65536, 98304, 131072,
                                      1 << 18, 1 << 19, 1 << 20, 1 << 22, 1 << 24, 1 << 26)
                      for k in (-4097, -9, -1, 0, 1, 9, 4097) if 0 < b + k < 1 << 26),
                    *range(10000, 400000, 1237)})
    need = [pg.pg_embed_workspace_size(n, V, d) for n in sizes]
    falls = [(sizes[i], need[i], sizes[i + 1], need[i + 1]) for i in range(len(need) - 1)
             if need[i] > need[i + 1]]
    assert not falls, falls[:3]


@pytest.mark.parametrize("d", [5, 385, 1001, 2560, 4096, 16384])
def test_layer_norm_workspace_of_the_largest_batch_serves_every_smaller_one(d):
    need = [pg.pg_layer_norm_workspace_size(n, d) for n in
            sorted({*range(0, 6000, 13), *(1 << k for k in range(32))})]
    assert need == sorted(need)


def test_orthogonalize_last_iterate_is_free():
    """Refusals are the two the header names: a singular value beyond 3 before a step, and
    |b s^2 + c s^4| beyond 100. The result itself may be large."""
    f = pg.lib().pg_orthogonalize

    def call(steps, a, b, c):
        return f(None, pg.PG_F32, 0, 100, 300, steps, a, b, c, 1e-7, 1.0, None, None, 0, None)

    assert call(1, 150.0, 0.0, 0.0) == pg.PG_OK
    assert call(2, 2.9, 0.0, 0.0) == pg.PG_OK
    assert call(1, 3e38, 0.0, 0.0) == pg.PG_OK
    assert call(1, 60.0, 50.0, 49.0) == pg.PG_OK
    assert call(1, 60.0, 51.0, 50.0) == pg.PG_EUNSUPPORTED
    assert call(2, 3.1, 0.0, 0.0) == pg.PG_EUNSUPPORTED
    nan, inf = float("nan"), float("inf")
    for bad in (nan, inf, -inf):
        for coef in ((bad, 0.0, 0.0), (0.0, bad, 0.0), (0.0, 0.0, bad)):
            assert call(1, *coef) == pg.PG_EUNSUPPORTED, coef


@pytest.mark.parametrize("fn,args,status", [
    ("pg_embed_workspace_size", (5, 100, 2**32 + 64), pg.PG_EUNSUPPORTED),
    ("pg_embed_workspace_size", (2**64 + 5, 100, 64), pg.PG_ERANGE),
    ("pg_embed_workspace_size", (5, 2**64 + 100, 64), pg.PG_ERANGE),
    ("pg_embed_workspace_size", (5, 100, -2**32 + 64), pg.PG_EINVAL),
    ("pg_layer_norm_workspace_size", (5, 2**32 + 64), pg.PG_EUNSUPPORTED),
    ("pg_orthogonalize_workspace_size", (1, 2**32 + 5, 5), pg.PG_EUNSUPPORTED),
    ("pg_orthogonalize_workspace_size", (1, 5, 2**32 + 5), pg.PG_EUNSUPPORTED),
    ("pg_orthogonalize_workspace_size", (2**64 + 1, 5, 5), pg.PG_ERANGE)])
def test_sizes_beyond_the_c_types_are_not_wrapped(fn, args, status):
    with pytest.raises(pg.PagegramError) as err:
        getattr(pg, fn)(*args)
    assert err.value.status == status


class _Stream:
    def __init__(self, device):
        self.device, self.cuda_stream = device, 0


def test_a_stream_of_another_device_is_refused():
    import torch
    with pytest.raises(ValueError, match="stream"):
        pg._call("pg_embed", torch.device("cuda", 0), _Stream(torch.device("cuda", 1)))


def test_a_missing_tensor_is_a_value_error():
    import torch
    with pytest.raises(ValueError, match="gamma"):
        pg._flat("pg_layer_norm", "gamma", None, torch.float32, 8, torch.device("cuda", 0))
