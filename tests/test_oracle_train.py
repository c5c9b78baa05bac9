"""Pins of the training-step oracle (oracle/train.py): gradients against
differences, sparse against dense, singular values against the polynomial."""
import numpy as np
import pytest

from oracle import train as ot

COEF = (3.4445, -4.7750, 2.0315)


def test_embed_rows_equal_dense_and_differences():
    rng = np.random.default_rng(1)
    V, d = 11, 5
    tokens = np.array([3, 3, 0, -1, 10, 11, 3, 7])
    T = rng.standard_normal((V, d))
    w = rng.standard_normal((len(tokens), d))
    dense = ot.embed_dense(w, tokens, V, 1.7)
    f = lambda t: np.sum(w * ot.embed(t, tokens, 1.7))  # noqa: E731
    for v in range(V):
        for j in range(d):
            up = T.copy()
            up[v, j] += 0.5
            assert abs((f(up) - f(T)) / 0.5 - dense[v, j]) < 1e-12     # linear in T
    urows, grad, cnt, mag = ot.embed_rows(w, tokens, V, 1.7)
    assert urows.tolist() == [0, 3, 7, 10] and cnt.tolist() == [1, 3, 1, 1]
    assert np.allclose(dense[urows], grad) and np.all(mag >= np.abs(grad) - 1e-12)


@pytest.mark.parametrize("d", [1, 2, 9])
def test_layer_norm_backward_against_differences(d):
    rng = np.random.default_rng(d)
    n, eps, h = 3, 1e-2, 1e-5
    x, dy, add = (rng.standard_normal((n, d)) for _ in range(3))
    g, b = rng.standard_normal(d), rng.standard_normal(d)
    y, mean, rstd = ot.layer_norm(x, g, b, eps)
    dx, dg, db = ot.layer_norm_backward(dy, x, g, mean, rstd, add)
    f = lambda x, g, b: np.sum(dy * ot.layer_norm(x, g, b, eps)[0])  # noqa: E731
    for i in range(n):
        for j in range(d):
            e = np.zeros((n, d))
            e[i, j] = h
            num = (f(x + e, g, b) - f(x - e, g, b)) / (2 * h)
            assert abs(num + add[i, j] - dx[i, j]) < 1e-6
    for j in range(d):
        e = np.zeros(d)
        e[j] = h
        assert abs((f(x, g + e, b) - f(x, g - e, b)) / (2 * h) - dg[j]) < 1e-6
        assert abs((f(x, g, b + e) - f(x, g, b - e)) / (2 * h) - db[j]) < 1e-6


@pytest.mark.parametrize("shape", [(1, 1), (5, 9), (9, 5), (24, 24)])
def test_newton_schulz_maps_singular_values(shape):
    rng = np.random.default_rng(7)
    G = rng.standard_normal(shape)
    out = ot.newton_schulz(G, 5, COEF, 0.0, scale=2.0)
    U, s, Vt = np.linalg.svd(G, full_matrices=False)
    s = s / np.sqrt((s * s).sum())
    for _ in range(5):
        s = COEF[0] * s + COEF[1] * s ** 3 + COEF[2] * s ** 5
    assert np.allclose(out, 2.0 * (U * s) @ Vt, atol=1e-10)
    assert np.array_equal(ot.newton_schulz(np.zeros(shape), 5, COEF, 1e-7), np.zeros(shape))


def test_half_storage_stays_below_the_rounding_of_the_result():
    # random matrices: the documented fp16 placement moves the result by less
    # than half a bf16 step in the 2-norm
    rng = np.random.default_rng(3)
    for shape in ((48, 160), (130, 130)):
        G = rng.standard_normal(shape)
        ref = ot.newton_schulz(G, 5, COEF, 1e-7)
        far = ot.newton_schulz_half(G, 5, COEF, 1e-7) - ref
        assert np.linalg.norm(far) < 2.0 ** -8 * np.linalg.norm(ref)
