"""Outputs of the head's gradients that are inputs of the same call, and sizes of its
workspaces; all without a GPU."""
import ctypes

import pytest

import hashed_head_gram_amd as pg
from tests.test_head_abi import B, E, F, FAKE, U, check

H, T, DH, DW = FAKE, FAKE + (1 << 30), FAKE + (2 << 30), FAKE + (3 << 30)
WS = FAKE + (1 << 36)


def table(dtype=B):
    return ctypes.byref(pg.make_table(dtype, T, 100))


@pytest.mark.parametrize("fn", ["pg_head_loss_backward", "pg_head_distill_backward"])
def test_gradients_are_not_written_over_their_operands(fn):
    """Later pieces of the vocabulary read h again, and dh reads T beside dT."""
    lead = dict(h=H, dtype=B, n=5, d=64, ld=64, table=table(), scale=1.0)
    back = dict(dh=DH, ld_dh=64, dw=DW, dw_dtype=B, accumulate=0, ws=WS, bytes=0, stream=None)
    if "distill" in fn:
        good = dict(**lead, ids=FAKE, teacher=FAKE, k=7, tau=2.0, lse=FAKE, logits=FAKE,
                    dloss=FAKE, **back)
        size = pg.pg_head_distill_backward_workspace_size(5, 64, 100, 7, B)
    else:
        good = dict(**lead, targets=FAKE, lse=FAKE, dloss=FAKE, dlse=None, **back)
        size = pg.pg_head_loss_backward_workspace_size(5, 64, 100, B)
    assert size > 0
    check(fn, {**good, "bytes": size}, [(dict(dh=H), E), (dict(dw=T), E), (dict(dh=H, dw=None), E),
                                        (dict(dh=None, dw=T), E)])
    f32 = dict(dtype=F, table=table(F), dw_dtype=F)
    check(fn, {**good, **f32, "bytes": 1 << 40}, [(dict(dh=H), E), (dict(dw=T), E)])
    # other refusals keep their status, and without rows there is nothing to read
    check(fn, {**good, "bytes": size}, [(dict(dh=H, accumulate=1), U),
                                        (dict(dw=T, d=16385, ld=16385, ld_dh=16385), U)])
    check(fn, {**good, **f32, "n": 0}, [(dict(dh=H, dw=T, accumulate=1), pg.PG_OK)])


def test_workspaces_hold_no_copies_that_a_call_does_not_make():
    """bf16 tables of whole slots are read where they lie: one token is scored with a
    few MB, not a copy of T's rows, and few tokens' gradients need none either."""
    V, d = 128000, 2560
    assert pg.pg_head_loss_workspace_size(1, d, V, B) < 4 << 20
    assert pg.pg_head_distill_workspace_size(32, d, V, 64, B) < 64 << 20
    # dz in two halves for 128 rows, and the products' partial results
    halves, parts = 128 * 2 * 2 * V, 256 * 256 * 256 * 4
    for n in (1, 8, 128):
        need = pg.pg_head_loss_backward_workspace_size(n, d, V, B)
        assert halves + parts < need < (halves + parts) * 1.1
    # rows that have to be copied are still counted
    assert pg.pg_head_loss_workspace_size(1, 2500, V, B) > 128 << 20
    # fp32 rows of dh add up in dh itself
    copies = 2 * 32768 * 64 * 4 + 16384 * 128 * 4          # h twice and T, in two halves
    need = pg.pg_head_loss_backward_workspace_size(32768, 64, 1000, F)
    assert need < copies * 2 + 2 * 32768 * 1024 * 2 + parts + (16 << 20)
