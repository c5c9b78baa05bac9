"""Operators of the training step around the n-gram memory: their cases and plain forms.

Token embedding (the residual stream the memory is added to) and its row
gradients, layer norm and its backward pass, and the orthogonalised update of
the projection weights. `run` computes each in elementary torch operations
(fp32, rounded once at the end) or, with `own` set, calls this package.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
_ZIPF = 1.1
_COEF = (3.4445, -4.7750, 2.0315)
_NS_STEPS = 5
_NS_EPS = 1e-7
_LN_EPS = 1e-5


def listed():
    return [
        # one decoded token for each of 32 sequences, 27B vocabulary and width
        dict(name="embed_decode_32", op="embed", n=32, d=2560, V=128000, table="bf16", out="bf16"),
        # the 27B fusion's training batch, 32 x 4096 tokens
        dict(name="embed_27b", op="embed", n=131072, d=2560, V=128000, table="bf16", out="bf16"),
        # touched rows of the 200M workloads' batch, 8 x 2048 tokens
        dict(name="embed_rows_200m", op="embed_rows", n=16384, d=768, V=50304, dtype="bf16"),
        # touched rows of the 27B batch: hot rows gather a sixth of the tokens
        dict(name="embed_rows_27b", op="embed_rows", n=131072, d=2560, V=128000, dtype="bf16"),
        # dense fp32 gradient of a small model, one ragged batch, odd width
        dict(name="embed_dense_odd", op="embed_dense", n=4095, d=385, V=50304, dtype="f32"),
        # decode: one token of 32 sequences
        dict(name="norm_decode_32", op="norm", n=32, d=2560, dtype="bf16"),
        # the 27B training batch, one pre-norm
        dict(name="norm_27b", op="norm", n=131072, d=2560, dtype="bf16"),
        # ragged fp32 batch of odd width
        dict(name="norm_grad_odd", op="norm_grad", n=4095, d=1001, dtype="f32", add=False),
        # the 27B training batch, with the gradient of the residual stream added
        dict(name="norm_grad_27b", op="norm_grad", n=131072, d=2560, dtype="bf16", add=True),
        # the tiny workload's W_V: latency
        dict(name="ortho_tiny", op="ortho", n=1, rows=64, cols=128, dtype="f32"),
        # the 200M workloads' W_V
        dict(name="ortho_200m", op="ortho", n=1, rows=768, cols=1024, dtype="f32"),
        # [W_V; W_K^(1..4)] of the 27B fusion: five matrices at once
        dict(name="ortho_27b", op="ortho", n=5, rows=2560, cols=1280, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_rows", "embed_dense", "norm", "norm_grad", "ortho"])
    dt = rng.choice(["f32", "bf16"])
    d = _log_int(rng, 16, 2560)
    if rng.random() < 0.5:                  # widths of models are mostly round
        d = max(16, d // 64 * 64)
    n = _log_int(rng, 1, 131072)
    if dt == "f32" or op == "embed_dense":
        n = min(n, 65536)
    if op == "embed":
        return dict(op=op, n=n, d=d, V=_log_int(rng, 100, 128000), table=dt,
                    out=rng.choice(["f32", "bf16"]) if n <= 65536 else "bf16")
    if op in ("embed_rows", "embed_dense"):
        return dict(op=op, n=n, d=d, V=_log_int(rng, 100, 128000), dtype=dt)
    if op == "norm":
        return dict(op=op, n=n, d=d, dtype=dt)
    if op == "norm_grad":
        return dict(op=op, n=n, d=d, dtype=dt, add=rng.random() < 0.5)
    rows, cols = _log_int(rng, 16, 2560), _log_int(rng, 16, 2560)
    if min(rows, cols) > 1280:
        rows = 1280
    return dict(op=op, n=rng.randint(1, 5), rows=rows, cols=cols, dtype=dt)


def _zipf_p(V):
    p = np.arange(1, V + 1, dtype=np.float64) ** -_ZIPF
    return p / p.sum()


def _tokens(n, V, g):
    cdf = torch.from_numpy(np.cumsum(_zipf_p(V))).cuda()
    u = torch.rand(n, dtype=torch.float64, device="cuda", generator=g)
    rank = torch.searchsorted(cdf, u).clamp_(max=V - 1)
    ids = torch.randperm(V, device="cuda", generator=g)
    return ids[rank].to(torch.int32)


def _normal(shape, dtype, g, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * scale).to(_DT[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "embed":
        s["tokens"] = _tokens(case["n"], case["V"], g)
        s["table"] = _normal((case["V"], case["d"]), case["table"], g, 0.02)
        s["scale"] = math.sqrt(case["d"])
        s["out"] = torch.empty(case["n"], case["d"], dtype=_DT[case["out"]], device="cuda")
    elif op in ("embed_rows", "embed_dense"):
        n, d, V = case["n"], case["d"], case["V"]
        s["tokens"] = _tokens(n, V, g)
        s["dout"] = _normal((n, d), case["dtype"], g)
        s["scale"] = math.sqrt(d)
        if op == "embed_rows":
            cap = min(n, V)
            s["urows"] = torch.zeros(cap, dtype=torch.int64, device="cuda")
            s["ugrad"] = torch.zeros(cap, d, device="cuda")
            s["n_unique"] = torch.zeros(1, dtype=torch.int64, device="cuda")
        else:
            s["dtable"] = torch.empty(V, d, device="cuda")
    elif op in ("norm", "norm_grad"):
        n, d = case["n"], case["d"]
        # rows of a residual stream: each with an offset and a spread of its own
        x = torch.randn(n, d, device="cuda", generator=g)
        x *= torch.rand(n, 1, device="cuda", generator=g) * 2 + 0.5
        x += torch.randn(n, 1, device="cuda", generator=g) * 0.5
        s["x"] = x.to(_DT[case["dtype"]])
        s["gamma"] = 1 + 0.2 * torch.randn(d, device="cuda", generator=g)
        s["y"] = torch.empty_like(s["x"])
        if op == "norm":
            s["beta"] = 0.2 * torch.randn(d, device="cuda", generator=g)
            s["mean"] = torch.empty(n, device="cuda")
            s["rstd"] = torch.empty(n, device="cuda")
        else:
            xd = s["x"].double()
            var, mean = torch.var_mean(xd, dim=1, correction=0)
            s["mean"], s["rstd"] = mean.float(), (var + _LN_EPS).rsqrt().float()
            s["dy"] = _normal((n, d), case["dtype"], g)
            s["add"] = _normal((n, d), case["dtype"], g) if case["add"] else None
            s["dgamma"] = torch.empty(d, device="cuda")
            s["dbeta"] = torch.empty(d, device="cuda")
    else:
        n, r, c = case["n"], case["rows"], case["cols"]
        k = min(r, c)
        # a gradient's spectrum: a few strong directions over a long tail
        u = torch.randn(n, r, k, device="cuda", generator=g)
        v = torch.randn(n, k, c, device="cuda", generator=g)
        sv = torch.arange(1, k + 1, device="cuda").float() ** -0.7
        G = (u * sv) @ v
        G = G + 0.02 * G.square().mean().sqrt() * torch.randn(n, r, c, device="cuda", generator=g)
        s["G"] = (G * 1e-3).to(_DT[case["dtype"]])
        s["out"] = torch.empty(n, r, c, dtype=torch.bfloat16, device="cuda")
    if own:
        import hashed_head_gram_amd as pg
        size = 0
        if op == "embed":
            s["handle"] = pg.make_table({"f32": pg.PG_F32, "bf16": pg.PG_BF16}[case["table"]],
                                        s["table"], case["V"])
        elif op in ("embed_rows", "embed_dense"):
            size = pg.pg_embed_workspace_size(case["n"], case["V"], case["d"])
        elif op == "norm_grad":
            size = pg.pg_layer_norm_workspace_size(case["n"], case["d"])
        elif op == "ortho":
            size = pg.pg_orthogonalize_workspace_size(case["n"], case["rows"], case["cols"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s


def _own(s):
    import hashed_head_gram_amd as pg
    case = s["case"]
    op = case["op"]
    if op == "embed":
        pg.pg_embed(s["handle"], s["tokens"], s["out"], scale=s["scale"])
        return s["out"]
    if op == "embed_rows":
        pg.pg_embed_backward(s["dout"], s["tokens"], case["V"], s["urows"], s["ugrad"],
                             s["n_unique"], s["ws"], scale=s["scale"])
        return s["urows"], s["ugrad"], s["n_unique"]
    if op == "embed_dense":
        pg.pg_embed_backward_dense(s["dout"], s["tokens"], s["dtable"], s["ws"],
                                   scale=s["scale"])
        return s["dtable"]
    if op == "norm":
        pg.pg_layer_norm(s["x"], s["gamma"], s["beta"], s["y"], eps=_LN_EPS, mean=s["mean"],
                         rstd=s["rstd"])
        return s["y"], s["mean"], s["rstd"]
    if op == "norm_grad":
        pg.pg_layer_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["y"],
                                  s["dgamma"], s["dbeta"], s["ws"], add=s["add"])
        return s["y"], s["dgamma"], s["dbeta"]
    pg.pg_orthogonalize(s["G"], s["out"], s["ws"], steps=_NS_STEPS, coef=_COEF, eps=_NS_EPS)
    return s["out"]


def _segments(tokens):
    """Ascending distinct tokens' positions: (sorted keys, segment of each token)."""
    keys, order = torch.sort(tokens, stable=True)
    new = torch.ones_like(keys, dtype=torch.int64)
    new[1:] = keys[1:] != keys[:-1]
    seg_sorted = torch.cumsum(new, 0) - 1
    seg = torch.empty_like(seg_sorted)
    seg[order] = seg_sorted
    return keys, seg_sorted, seg


def _ns_plain(G, dtype):
    a, b, c = _COEF
    X = G.to(dtype)
    if X.shape[1] > X.shape[2]:
        X = X.mT
    X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + _NS_EPS)
    for _ in range(_NS_STEPS):
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.mT if G.shape[1] > G.shape[2] else X


def run(s):
    if own:
        return _own(s)
    case = s["case"]
    op = case["op"]
    if op == "embed":
        return (s["table"][s["tokens"].long()].float() * s["scale"]).to(s["out"].dtype)
    if op == "embed_rows":
        keys, seg_sorted, seg = _segments(s["tokens"])
        urows = torch.zeros_like(s["urows"])
        urows[seg_sorted] = keys.long()
        ugrad = torch.zeros_like(s["ugrad"])
        ugrad.index_add_(0, seg, s["dout"].float() * s["scale"])
        return urows, ugrad, seg_sorted[-1:] + 1
    if op == "embed_dense":
        dt = torch.zeros(case["V"], case["d"], device="cuda")
        return dt.index_add_(0, s["tokens"].long(), s["dout"].float() * s["scale"])
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = (xc.square().mean(1, keepdim=True) + _LN_EPS).rsqrt()
        y = xc * rstd * s["gamma"] + s["beta"]
        return y.to(s["x"].dtype), mean[:, 0], rstd[:, 0]
    if op == "norm_grad":
        rstd = s["rstd"][:, None]
        xh = (s["x"].float() - s["mean"][:, None]) * rstd
        dy = s["dy"].float()
        gd = dy * s["gamma"]
        dx = rstd * (gd - gd.mean(1, keepdim=True) - xh * (gd * xh).mean(1, keepdim=True))
        if s["add"] is not None:
            dx = dx + s["add"].float()
        return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)
    return _ns_plain(s["G"], torch.float32).to(torch.bfloat16).contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        return s["table"].index_select(0, s["tokens"].long()).double() * s["scale"]
    if op in ("embed_rows", "embed_dense"):
        ids, inv = torch.unique(s["tokens"].long(), return_inverse=True)
        rows = torch.zeros(len(ids), case["d"], dtype=torch.float64, device="cuda")
        rows.index_add_(0, inv, s["dout"].double())
        rows *= s["scale"]
        if op == "embed_dense":
            out = torch.zeros(case["V"], case["d"], dtype=torch.float64, device="cuda")
            out[ids] = rows
            return out
        cap = min(case["n"], case["V"])
        urows = torch.zeros(cap, dtype=torch.int64, device="cuda")
        urows[:len(ids)] = ids
        ugrad = torch.zeros(cap, case["d"], dtype=torch.float64, device="cuda")
        ugrad[:len(ids)] = rows
        return urows, ugrad, torch.tensor([len(ids)], device="cuda")
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1 / torch.sqrt(var + _LN_EPS)
        x -= mean[:, None]
        x *= rstd[:, None]
        x *= s["gamma"].double()
        x += s["beta"].double()
        return x, mean, rstd
    if op == "norm_grad":
        d = case["d"]
        r = s["rstd"].double()[:, None]
        xh = (s["x"].double() - s["mean"].double()[:, None]) * r
        dy = s["dy"].double()
        dgamma, dbeta = (dy * xh).sum(0), dy.sum(0)
        dy *= s["gamma"].double()
        m1 = dy.sum(1, keepdim=True) / d
        m2 = (dy * xh).sum(1, keepdim=True) / d
        dx = dy.sub_(m1).addcmul_(xh, m2, value=-1).mul_(r)
        if s["add"] is not None:
            dx += s["add"].double()
        return dx, dgamma, dbeta
    a, b, c = _COEF
    out = []
    for G in s["G"].double():
        wide = G.shape[0] <= G.shape[1]
        X = G if wide else G.T.contiguous()
        X = X / (torch.linalg.norm(X) + _NS_EPS)
        eye = torch.eye(X.shape[0], dtype=torch.float64, device="cuda")
        for _ in range(_NS_STEPS):
            A = torch.mm(X, X.T.contiguous())
            X = torch.mm(a * eye + b * A + c * torch.mm(A, A), X)
        out.append(X if wide else X.T)
    return torch.stack(out)


def _distinct(n, V):
    """Expected number of distinct tokens of a Zipf batch."""
    return float(np.sum(-np.expm1(n * np.log1p(-_zipf_p(V)))))


def work(case):
    op = case["op"]
    if op == "embed":
        n, d = case["n"], case["d"]
        rows = _distinct(n, case["V"])
        return dict(bytes=4 * n + rows * d * _SIZE[case["table"]] + n * d * _SIZE[case["out"]],
                    flops=n * d)
    if op in ("embed_rows", "embed_dense"):
        n, d = case["n"], case["d"]
        written = _distinct(n, case["V"]) if op == "embed_rows" else case["V"]
        return dict(bytes=4 * n + n * d * _SIZE[case["dtype"]] + written * (4 * d + 8), flops=n * d)
    if op == "norm":
        n, d, e = case["n"], case["d"], _SIZE[case["dtype"]]
        return dict(bytes=2 * n * d * e + 8 * n + 8 * d, flops=8 * n * d)
    if op == "norm_grad":
        n, d, e = case["n"], case["d"], _SIZE[case["dtype"]]
        return dict(bytes=(4 if case["add"] else 3) * n * d * e + 8 * n + 12 * d, flops=14 * n * d)
    # symmetric products need half their tiles: X X^T and A A, then B X
    n, r, c = case["n"], case["rows"], case["cols"]
    m, k = min(r, c), max(r, c)
    return dict(bytes=n * r * c * (_SIZE[case["dtype"]] + 2),
                flops=n * _NS_STEPS * (m * m * k + m * m * m + 2 * m * m * k))
