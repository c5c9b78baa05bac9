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
