"""CPU oracle of the training-step operators around the memory (token
embedding and its table gradient, layer norm and its backward pass, the
orthogonalised update).

TEST INFRASTRUCTURE ONLY: imported by the tests and nothing on the product
path; shares no code with the HIP library. Plain numpy, float64.
"""
import numpy as np


def embed(table, tokens, scale):
    """scale * table[tokens]; zero rows for tokens outside the table."""
    table = np.asarray(table, np.float64)
    tokens = np.asarray(tokens, np.int64)
    ok = (tokens >= 0) & (tokens < len(table))
    return np.where(ok[:, None], scale * table[np.where(ok, tokens, 0)], 0.0)


def embed_rows(dout, tokens, V, scale):
    """(urows ascending, gradient rows, lookups per row, sum of |terms| per
    element) of scale * sum of dout over the tokens of each touched row."""
    dout = np.asarray(dout, np.float64)
    tokens = np.asarray(tokens, np.int64)
    ok = (tokens >= 0) & (tokens < V)
    urows, inv, cnt = np.unique(tokens[ok], return_inverse=True, return_counts=True)
    grad = np.zeros((len(urows), dout.shape[1]))
    mag = np.zeros_like(grad)
    np.add.at(grad, inv, dout[ok])
    np.add.at(mag, inv, np.abs(dout[ok]))
    return urows, scale * grad, cnt, abs(scale) * mag


def embed_dense(dout, tokens, V, scale):
    """The same gradient as a dense [V, d] table."""
    urows, grad, _, _ = embed_rows(dout, tokens, V, scale)
    out = np.zeros((V, np.asarray(dout).shape[1]))
    out[urows] = grad
    return out


def layer_norm(x, gamma, beta, eps):
    """(y, mean, rstd) over the last dimension."""
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None] * np.asarray(gamma, np.float64)
    return (y if beta is None else y + np.asarray(beta, np.float64)), mean, rstd


def layer_norm_backward(dy, x, gamma, mean, rstd, add=None):
    """(dx, dgamma, dbeta) for rows of x and the forward's mean and rstd."""
    dy = np.asarray(dy, np.float64)
    xh = (np.asarray(x, np.float64) - np.asarray(mean, np.float64)[:, None]) \
        * np.asarray(rstd, np.float64)[:, None]
    g = dy * np.asarray(gamma, np.float64)
    m1 = g.mean(1, keepdims=True)
    m2 = (g * xh).mean(1, keepdims=True)
    dx = np.asarray(rstd, np.float64)[:, None] * (g - m1 - xh * m2)
    if add is not None:
        dx = dx + np.asarray(add, np.float64)
    return dx, (dy * xh).sum(0), dy.sum(0)


def newton_schulz(G, steps, coef, eps, scale=1.0):
    """The Newton-Schulz iterate of one matrix in float64."""
    a, b, c = coef
    G = np.asarray(G, np.float64)
    tall = G.shape[0] > G.shape[1]
    X = G.T if tall else G
    norm = np.sqrt((X * X).sum())
    X = X / (norm + eps) if norm > 0 else X * 0.0
    for _ in range(steps):
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
    return scale * (X.T if tall else X)


def newton_schulz_half(G, steps, coef, eps, scale=1.0):
    """newton_schulz with the operands of its products held in fp16 the way
    the library documents it (the iterate and the diagonals wider), all else
    in float64: how far that storage alone moves the result."""
    a, b, c = coef

    def half(x, e):
        return (x * 2.0 ** e).astype(np.float32).astype(np.float16).astype(np.float64) * 2.0 ** -e

    G = np.asarray(G, np.float64)
    tall = G.shape[0] > G.shape[1]
    X = G.T if tall else G
    X = X / (np.sqrt((X * X).sum()) + eps)
    for _ in range(steps):
        Xh = half(X, 10)
        A = Xh @ Xh.T
        D = np.diag(A).copy()
        Oh = half(A - np.diag(D), 12)
        B = b * (Oh + np.diag(D)) + c * (Oh @ Oh + (D[:, None] + D[None]) * Oh + np.diag(D * D))
        E = np.diag(B).copy()
        X = (a + E)[:, None] * X + half(B - np.diag(E), 9) @ Xh
    return scale * (X.T if tall else X)
