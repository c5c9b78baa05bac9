"""CPU oracle of the head's losses (cross entropy and distillation from a
teacher's logits over a tied table) and their gradients.

TEST INFRASTRUCTURE ONLY: imported by the tests and nothing on the product
path; shares no code with the HIP library. Plain numpy, float64.
"""
import numpy as np


def logits(h, table, scale):
    return scale * (np.asarray(h, np.float64) @ np.asarray(table, np.float64).T)


def log_sum_exp(z):
    m = z.max(1)
    m = np.where(np.isfinite(m), m, 0.0)
    with np.errstate(divide="ignore"):
        return m + np.log(np.exp(z - m[:, None]).sum(1))


def loss(h, table, targets, scale=1.0):
    """(loss, lse): cross entropy, 0 for targets outside the table."""
    z = logits(h, table, scale)
    targets = np.asarray(targets, np.int64)
    ok = (targets >= 0) & (targets < z.shape[1])
    lse = log_sum_exp(z)
    zt = z[np.arange(len(z)), np.where(ok, targets, 0)]
    return np.where(ok, lse - zt, 0.0), lse


def loss_dz(z, targets, lse, dloss, dlse=None):
    """Gradient of sum(dloss loss + dlse lse) by the logits z, with lse given."""
    targets = np.asarray(targets, np.int64)
    ok = (targets >= 0) & (targets < z.shape[1])
    w = np.where(ok, np.asarray(dloss, np.float64), 0.0)
    a = w if dlse is None else w + np.asarray(dlse, np.float64)
    dz = a[:, None] * np.exp(z - np.asarray(lse, np.float64)[:, None])
    rows = np.nonzero(ok)[0]
    dz[rows, targets[rows]] -= w[rows]
    return dz


def shares(ids, teacher, V, temperature):
    """The teacher's shares of its entries; rows without entries are zeros."""
    ids = np.asarray(ids, np.int64)
    ok = (ids >= 0) & (ids < V)
    t = np.where(ok, np.asarray(teacher, np.float64) / temperature, -np.inf)
    m = t.max(1, keepdims=True)
    e = np.exp(t - np.where(np.isfinite(m), m, 0.0))
    s = e.sum(1, keepdims=True)
    return np.where(s > 0, e / np.where(s > 0, s, 1.0), 0.0), ok


def distill(h, table, ids, teacher, temperature=1.0, scale=1.0):
    """(loss, lse, z at the ids)."""
    z = logits(h, table, scale)
    q, ok = shares(ids, teacher, z.shape[1], temperature)
    zk = np.where(ok, np.take_along_axis(z, np.where(ok, ids, 0).astype(np.int64), 1), 0.0)
    lse = log_sum_exp(z / temperature)
    logq = np.log(np.where(q > 0, q, 1.0))
    return temperature ** 2 * (q * (logq - zk / temperature + lse[:, None])).sum(1), lse, zk


def distill_dz(z, ids, teacher, lse, dloss, temperature=1.0):
    """Gradient of sum(dloss loss) by the logits z, with lse given."""
    q, ok = shares(ids, teacher, z.shape[1], temperature)
    w = np.asarray(dloss, np.float64) * temperature * (q.sum(1) > 0)
    dz = w[:, None] * np.exp(z / temperature - np.asarray(lse, np.float64)[:, None])
    r, j = np.nonzero(ok)
    np.subtract.at(dz, (r, np.asarray(ids, np.int64)[r, j]), w[r] * q[r, j])
    return dz


def grads(dz, h, table, scale=1.0):
    """(dh, dtable) of the logits' gradient dz."""
    return (scale * (dz @ np.asarray(table, np.float64)),
            scale * (dz.T @ np.asarray(h, np.float64)))
