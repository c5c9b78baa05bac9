"""Losses of a language model's head over a large vocabulary: their cases and plain forms.

The head shares the token embedding's table: logits = scale * h T^T. Cross
entropy against target tokens and distillation from a teacher's largest
logits, each with its gradients. `run` computes them in elementary torch
operations (fp32, rounded once at the end) or, with `own` set, calls this
package, which keeps no logits.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
_ZIPF = 1.1
_W_SIGMA = 0.02


def listed():
    return [
        # scoring one proposed token of each of 32 sequences, 27B vocabulary and width
        dict(name="loss_score_32", op="loss", n=32, d=2560, V=128000, dtype="bf16"),
        # the 200M workloads' batch, 8 x 2048 tokens
        dict(name="loss_200m", op="loss", n=16384, d=768, V=50304, dtype="bf16"),
        # a micro-batch of the 27B fusion's training step, 4 x 4096 tokens
        dict(name="loss_27b", op="loss", n=16384, d=2560, V=128000, dtype="bf16"),
        # a ragged fp32 batch, odd width and vocabulary
        dict(name="loss_odd", op="loss", n=4095, d=385, V=50303, dtype="f32"),
        # the tiny workload's step: latency
        dict(name="grad_tiny", op="loss_grad", n=256, d=64, V=1024, dtype="f32", zloss=False),
        # gradients of the ragged fp32 batch
        dict(name="grad_odd", op="loss_grad", n=4095, d=385, V=50303, dtype="f32", zloss=True),
        # gradients of the 200M workloads' batch, with a pull on the log of the sum
        dict(name="grad_200m", op="loss_grad", n=16384, d=768, V=50304, dtype="bf16", zloss=True),
        # gradients of the 27B micro-batch
        dict(name="grad_27b", op="loss_grad", n=16384, d=2560, V=128000, dtype="bf16",
             zloss=False),
        # a small ragged batch against 33 teacher logits a token
        dict(name="distill_odd", op="distill", n=1001, d=385, V=50303, dtype="f32", k=33,
             temperature=1.0),
        # a 27B micro-batch against a teacher's 64 largest logits
        dict(name="distill_27b", op="distill", n=8192, d=2560, V=128000, dtype="bf16", k=64,
             temperature=2.0),
        # gradients of the 200M batch against 32 teacher logits a token
        dict(name="distill_grad_200m", op="distill_grad", n=16384, d=768, V=50304, dtype="bf16",
             k=32, temperature=1.0),
        # gradients of a 27B micro-batch against 64
        dict(name="distill_grad_27b", op="distill_grad", n=8192, d=2560, V=128000, dtype="bf16",
             k=64, temperature=2.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["loss", "loss_grad", "distill", "distill_grad"])
    dt = rng.choice(["f32", "bf16", "bf16"])
    d = _log_int(rng, 16, 2560)
    if rng.random() < 0.5:                  # widths of models are mostly round
        d = max(16, d // 64 * 64)
    V = _log_int(rng, 100, 128000)
    n = _log_int(rng, 1, 16384 if op.startswith("loss") else 8192)
    if dt == "f32":                         # a ragged fp32 batch of the 200M sizes at most
        n = max(1, min(n, 16384 * 768 * 50304 // (d * V)))
    case = dict(op=op, n=n, d=d, V=V, dtype=dt)
    if op == "loss_grad":
        case["zloss"] = rng.random() < 0.5
    if op.startswith("distill"):
        case["k"] = min(_log_int(rng, 1, 64), V)
        case["temperature"] = rng.choice([1.0, 2.0, 1.5])
    return case


def _zipf_ids(shape, V, ids, g):
    p = np.arange(1, V + 1, dtype=np.float64) ** -_ZIPF
    cdf = torch.from_numpy(np.cumsum(p / p.sum())).cuda()
    u = torch.rand(shape, dtype=torch.float64, device="cuda", generator=g)
    return ids[torch.searchsorted(cdf, u).clamp_(max=V - 1)]


def _teacher(n, V, k, first, g):
    """ids int32 [n, k] of distinct tokens (the first is `first`; -1: none) and fp32 logits."""
    ids = torch.randperm(V, device="cuda", generator=g)
    # distances between the ranks of a row's tokens, mostly short
    room = max(1, (V - 1) // k)
    gap = torch.empty(n, k, device="cuda").exponential_(4.0 / room, generator=g)
    gap = gap.long().clamp_(max=room - 1) + 1
    gap[:, 0] = 0
    at = torch.empty_like(ids)
    at[ids] = torch.arange(V, device="cuda")
    rank = (at[first][:, None] + gap.cumsum(1)) % V
    tid = ids[rank].to(torch.int32)
    j = torch.arange(k, device="cuda").float()
    t = 14 - 2.2 * torch.log1p(j) + 0.4 * torch.randn(n, k, device="cuda", generator=g)
    # some teachers sent fewer entries, and padded positions none
    count = torch.full((n,), k, device="cuda")
    u = torch.rand(n, device="cuda", generator=g)
    count[u < 0.06] = (k + 1) // 2
    count[u < 0.03] = 0
    tid[torch.arange(k, device="cuda")[None] >= count[:, None]] = -1
    return tid, t


def _row_chunks(n, V, size):
    """Row ranges whose [rows, V] matrices of `size` bytes an element hold about 2 GB."""
    step = max(1, int(2e9) // (V * size))
    return [(a, min(n, a + step)) for a in range(0, n, step)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, n, d, V = case["op"], case["n"], case["d"], case["V"]
    dt = _DT[case["dtype"]]
    s = dict(case=case, scale=1.0)
    table = torch.randn(V, d, device="cuda", generator=g) * _W_SIGMA
    ids = torch.randperm(V, device="cuda", generator=g)
    target = _zipf_ids((n,), V, ids, g)
    # rows of the last norm: noise with a part along the right token's row, from
    # no knowledge of it to near certainty
    lift = torch.rand(n, 1, device="cuda", generator=g) * (1.2 * math.log(V) / _W_SIGMA / d)
    h = torch.randn(n, d, device="cuda", generator=g)
    h += lift * (table[target] / _W_SIGMA)
    s["h"], s["table"] = h.to(dt), table.to(dt)
    del h, table
    inv_t = 1.0
    if op.startswith("loss"):
        tok = target.to(torch.int32)
        tok[torch.rand(n, device="cuda", generator=g) < 0.03] = -1     # padded positions
        s["targets"] = tok
        count = max(1, int((tok >= 0).sum()))
    else:
        s["ids"], s["teacher"] = _teacher(n, V, case["k"], target, g)
        s["temperature"] = case["temperature"]
        inv_t = 1.0 / case["temperature"]
        count = max(1, int((s["ids"][:, 0] >= 0).sum()))
        s["logits"] = torch.zeros(n, case["k"], device="cuda")
    s["loss"] = torch.zeros(n, device="cuda")
    s["lse"] = torch.zeros(n, device="cuda")
    if op.endswith("grad"):
        # what the forward pass left, and the gradient of the mean
        w = s["table"].float()
        for a, b in _row_chunks(n, V, 8):
            z = s["h"][a:b].float() @ w.T
            s["lse"][a:b] = torch.logsumexp(z.double() * inv_t, 1).float()
            if "ids" in s:
                zk = z.gather(1, s["ids"][a:b].long().clamp(min=0))
                s["logits"][a:b] = torch.where(s["ids"][a:b] >= 0, zk, 0.0)
            del z
        del w
        s["dloss"] = torch.full((n,), 1.0 / count, device="cuda")
        s["dlse"] = s["lse"] * (2e-4 / count) if case.get("zloss") else None
        s["dh"] = torch.empty_like(s["h"])
        s["dw"] = torch.empty_like(s["table"])
    if own:
        import hashed_head_gram_amd as pg
        code = {"f32": pg.PG_F32, "bf16": pg.PG_BF16}[case["dtype"]]
        s["handle"] = pg.make_table(code, s["table"], V)
        if op == "loss":
            size = pg.pg_head_loss_workspace_size(n, d, V, code)
        elif op == "loss_grad":
            size = pg.pg_head_loss_backward_workspace_size(n, d, V, code)
        elif op == "distill":
            size = pg.pg_head_distill_workspace_size(n, d, V, case["k"], code)
        else:
            size = pg.pg_head_distill_backward_workspace_size(n, d, V, case["k"], code)
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


def _own(s):
    import hashed_head_gram_amd as pg
    op = s["case"]["op"]
    if op == "loss":
        pg.pg_head_loss(s["h"], s["handle"], s["targets"], s["loss"], s["lse"], s["ws"],
                        scale=s["scale"])
        return s["loss"], s["lse"]
    if op == "loss_grad":
        pg.pg_head_loss_backward(s["h"], s["handle"], s["targets"], s["lse"], s["dloss"],
                                 s["dh"], s["dw"], s["ws"], dlse=s["dlse"], scale=s["scale"])
        return s["dh"], s["dw"]
    if op == "distill":
        pg.pg_head_distill(s["h"], s["handle"], s["ids"], s["teacher"], s["loss"], s["lse"],
                           s["logits"], s["ws"], temperature=s["temperature"], scale=s["scale"])
        return s["loss"], s["lse"], s["logits"]
    pg.pg_head_distill_backward(s["h"], s["handle"], s["ids"], s["teacher"], s["lse"],
                                s["logits"], s["dloss"], s["dh"], s["dw"], s["ws"],
                                temperature=s["temperature"], scale=s["scale"])
    return s["dh"], s["dw"]


def _plain_teacher(s):
    """Shares of the teacher's entries (0 where there is none), and which are there."""
    there = s["ids"] >= 0
    t = torch.where(there, s["teacher"] / s["temperature"], -math.inf)
    m = t.max(1, keepdim=True).values
    e = torch.where(there, (t - torch.where(m > -math.inf, m, 0.0)).exp(), 0.0)
    total = e.sum(1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0), there


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    h, w = s["h"].float(), s["table"].float()
    if op == "loss":
        z = (h @ w.T).mul_(s["scale"])
        there = s["targets"] >= 0
        zt = z.gather(1, s["targets"].long().clamp(min=0)[:, None])[:, 0]
        m = z.max(1).values
        lse = m + z.sub_(m[:, None]).exp_().sum(1).log()
        return torch.where(there, lse - zt, 0.0), lse
    if op == "distill":
        T = s["temperature"]
        q, there = _plain_teacher(s)
        z = (h @ w.T).mul_(s["scale"])
        zk = torch.where(there, z.gather(1, s["ids"].long().clamp(min=0)), 0.0)
        z.mul_(1 / T)
        m = z.max(1).values
        lse = m + z.sub_(m[:, None]).exp_().sum(1).log()
        logq = torch.where(q > 0, q, 1.0).log()
        loss = T * T * (q * (logq - zk / T + lse[:, None])).sum(1)
        return loss, lse, zk
    dz = (h @ w.T).mul_(s["scale"])
    if op == "loss_grad":
        there = s["targets"] >= 0
        dl = torch.where(there, s["dloss"], 0.0)
        a = dl if s["dlse"] is None else dl + s["dlse"]
        dz.sub_(s["lse"][:, None]).exp_().mul_(a[:, None])
        dz.scatter_add_(1, s["targets"].long().clamp(min=0)[:, None], -dl[:, None])
    else:
        T = s["temperature"]
        q, there = _plain_teacher(s)
        dl = torch.where(there.any(1), s["dloss"], 0.0) * T
        dz.mul_(1 / T).sub_(s["lse"][:, None]).exp_().mul_(dl[:, None])
        dz.scatter_add_(1, s["ids"].long().clamp(min=0), -dl[:, None] * q)
    dz.mul_(s["scale"])
    return (dz @ w).to(s["h"].dtype), (dz.T @ h).to(s["table"].dtype)


def exact(case, seed):
    s = prepare(case, seed)
    op, n, V, c = case["op"], case["n"], case["V"], s["scale"]
    inv_t = 1.0 / s.get("temperature", 1.0)
    f64 = dict(dtype=torch.float64, device="cuda")
    h, w = s["h"].double(), s["table"].double()
    wt = w.T.contiguous()
    if op.startswith("loss"):
        ids = s["targets"].long()[:, None]
        share = (ids >= 0).double()
    else:
        # shares by a softmax over the entries that are there
        ids = s["ids"].long()
        t = (s["teacher"].double() * inv_t).masked_fill(ids < 0, -math.inf)
        share = torch.softmax(t, 1).nan_to_num(0.0)
    pos = ids.clamp(min=0)
    some = share.sum(1)                                   # 1, or 0 for a row without entries
    if not op.endswith("grad"):
        loss, lse = torch.empty(n, **f64), torch.empty(n, **f64)
        zk = torch.empty(ids.shape, **f64)
        for a, b in _row_chunks(n, V, 8):
            z = torch.mm(h[a:b], wt) * c
            zk[a:b] = z.gather(1, pos[a:b])
            lse[a:b] = torch.logsumexp(z * inv_t, 1)
        ent = torch.special.xlogy(share, share).sum(1)
        loss = (ent - (share * zk).sum(1) * inv_t + lse * some) / inv_t ** 2
        if op == "loss":
            return loss, lse
        return loss, lse, zk.masked_fill(ids < 0, 0.0)
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    lse, dl = s["lse"].double(), s["dloss"].double() * some / inv_t
    weight = dl.clone()
    if s["dlse"] is not None:
        weight += s["dlse"].double()
    for a, b in _row_chunks(n, V, 8):
        p = torch.exp(torch.mm(h[a:b], wt) * (c * inv_t) - lse[a:b, None]) * weight[a:b, None]
        p.scatter_add_(1, pos[a:b], -share[a:b] * dl[a:b, None])
        dh[a:b] = torch.mm(p, w) * c
        dw += torch.mm(p.T, h[a:b]) * c
    return dh, dw


def work(case):
    n, d, V, e = case["n"], case["d"], case["V"], _SIZE[case["dtype"]]
    k = case.get("k", 0)
    if case["op"].endswith("grad"):
        # logits again, then the two gradients
        return dict(bytes=2 * (n + V) * d * e + 12 * n + 12 * n * k, flops=6 * n * d * V)
    return dict(bytes=(n + V) * d * e + 12 * n + 12 * n * k, flops=2 * n * d * V)
