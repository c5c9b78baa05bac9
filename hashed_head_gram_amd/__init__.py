"""Python binding of libpagegram.so (the MI355X n-gram memory path).

Argument marshalling only: every step of the path runs in the library's HIP
kernels. The functions carry the C entry points' names and take torch device
tensors (PyTorch supplies device memory and the current stream). There is no
CPU fallback: importing works without the library, but the first call raises
if libpagegram.so has not been built (python -m hashed_head_gram_amd.build).
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpagegram.so")

PG_OK, PG_EINVAL, PG_EUNSUPPORTED, PG_EHIP, PG_ERANGE = 0, -1, -2, -3, -4
PG_PAGEGRAM, PG_ENGRAM = 0, 1
PG_F32, PG_BF16, PG_NF4 = 0, 1, 2
PG_GATE_SCALAR, PG_GATE_ENGRAM = 0, 1
PG_STAGE_PAGE, PG_STAGE_ROW = 0, 1
PG_MAX_ORDERS, PG_MAX_HEADS = 4, 16

_i32, _i64, _u64, _f32, _vp = (ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64,
                               ctypes.c_float, ctypes.c_void_p)


class PgLayout(ctypes.Structure):
    _fields_ = [("kind", _i32), ("n_min", _i32), ("n_max", _i32), ("K", _i32),
                ("S", _i32), ("r", _i32),
                ("pages", _i64 * PG_MAX_ORDERS),
                ("head_rows", (_i64 * PG_MAX_HEADS) * PG_MAX_ORDERS),
                ("hash_seed", _u64), ("use_signs", _i32), ("pad_id", _i32)]


class PgTable(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("reserved", _i32), ("data", _vp),
                ("scales", _vp), ("n_rows", _i64)]


class PgFuse(ctypes.Structure):
    _fields_ = [("gate", _i32), ("dtype", _i32), ("d", _i32), ("M", _i32),
                ("g", _f32), ("eps", _f32), ("gamma_h", _vp), ("gamma_k", _vp),
                ("gamma_u", _vp), ("conv_w", _vp), ("conv_k", _i32),
                ("conv_dil", _i32), ("increment_only", _i32), ("reserved", _i32)]


class PgCacheStats(ctypes.Structure):
    _fields_ = [("tokens", _i64), ("lookups", _i64), ("distinct", _i64), ("misses", _i64)]


_P = ctypes.POINTER
_SIGS = {
    "pg_index": (_i32, [_P(PgLayout), _vp, _i64, _i64, _vp, _i64, _vp, _vp, _vp,
                        _vp, _vp, _vp, _vp]),
    "pg_gather": (_i32, [_P(PgLayout), _P(PgTable), _vp, _vp, _i64, _i32, _vp, _vp]),
    "pg_index_gather": (_i32, [_P(PgLayout), _P(PgTable), _vp, _i64, _i64, _vp,
                               _i64, _i32, _vp, _vp, _vp]),
    "pg_project_gate": (_i32, [_P(PgFuse), _vp, _i64, _i64, _i64, _vp, _vp, _vp,
                               _vp, _i64, _vp]),
    "pg_forward": (_i32, [_P(PgLayout), _P(PgTable), _P(PgFuse), _vp, _i64, _i64,
                          _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp, _vp]),
    "pg_forward_noalloc": (_i32, [_P(PgLayout), _P(PgTable), _P(PgFuse), _vp, _i64, _i64,
                                  _vp, _i64, _vp, _vp, _vp, _vp, _vp]),
    "pg_index_records": (_i32, [_P(PgLayout), _vp, _i64, _i64, _vp, _i64, _vp, _vp, _vp]),
    "pg_project_gathered": (_i32, [_P(PgLayout), _P(PgTable), _P(PgFuse), _vp, _i64, _i64,
                                   _vp, _vp, _vp, _vp]),
    "pg_stage_geometry": (_i32, [_P(PgLayout), _i32, _i32, _i64, _P(_i64), _P(_i64),
                                 _P(_i64)]),
    "pg_stage_rows": (_i32, [_P(PgLayout), _P(PgTable), _i32, _vp, _i64, _P(PgTable), _vp, _vp,
                             _vp, _vp, _i64, _vp]),
    "pg_gather_staged": (_i32, [_P(PgLayout), _P(PgTable), _vp, _vp, _i64, _i32, _vp, _vp]),
    "pg_quantize_fp8": (_i32, [_vp, _i32, _i64, _i32, _vp, _vp]),
    "pg_index_gather_fp8": (_i32, [_P(PgLayout), _P(PgTable), _vp, _i64, _i64, _vp,
                                   _i64, _i32, _vp, _vp, _vp]),
    "pg_project_gate_fp8": (_i32, [_P(PgFuse), _vp, _i64, _i64, _i64, _vp, _i32, _i32,
                                   _vp, _vp, _vp, _i64, _vp]),
    "pg_forward_fp8": (_i32, [_P(PgLayout), _P(PgTable), _P(PgFuse), _vp, _i64, _i64,
                              _vp, _i64, _vp, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _vp]),
    "pg_engram_project": (_i32, [_P(PgFuse), _vp, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp]),
    "pg_engram_project_fp8": (_i32, [_P(PgFuse), _vp, _i64, _i64, _i64, _vp, _i32, _i32, _vp,
                                     _vp, _i64, _vp]),
    "pg_engram_gate": (_i32, [_P(PgFuse), _i64, _i64, _vp, _i64, _vp]),
    "pg_engram_mix": (_i32, [_P(PgFuse), _i64, _i64, _vp, _vp, _vp, _i64, _vp]),
    "pg_read_probe": (_i32, [_vp, _i64, _vp, _vp]),
    "pg_strerror": (ctypes.c_char_p, [_i32]),
    "pg_hash_version": (ctypes.c_uint32, []),
    "pg_layout_rows": (_i32, [_P(PgLayout), _P(_i64)]),
    "pg_workspace_size": (_i64, [_P(PgLayout), _P(PgFuse), _i64, _i64]),
    "pg_backward_workspace_size": (_i64, [_P(PgLayout), _P(PgFuse), _i64, _i64]),
    "pg_backward_scalar": (_i32, [_P(PgLayout), _P(PgFuse), _vp, _vp, _vp, _vp, _vp, _i64,
                                  _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp]),
    "pg_row_rms_step": (_i32, [_P(PgLayout), _vp, _vp, _vp, _i64, _vp, _vp, _vp, _i64, _f32,
                               _f32, _f32, _f32, _vp]),
    "pg_row_rms_flush": (_i32, [_P(PgLayout), _vp, _vp, _vp, _i64, _f32, _f32, _f32, _vp]),
    "pg_embed": (_i32, [_P(PgTable), _i32, _f32, _vp, _i64, _i32, _vp, _i64, _vp, _vp]),
    "pg_embed_workspace_size": (_i64, [_i64, _i64, _i32]),
    "pg_embed_backward": (_i32, [_vp, _i32, _i64, _vp, _i64, _i64, _i32, _f32, _vp, _vp, _vp,
                                 _vp, _i64, _vp]),
    "pg_embed_backward_dense": (_i32, [_vp, _i32, _i64, _vp, _i64, _i64, _i32, _f32, _vp, _i32,
                                       _vp, _i64, _vp]),
    "pg_layer_norm": (_i32, [_vp, _i32, _i64, _i32, _i64, _vp, _vp, _f32, _vp, _i64, _vp, _vp,
                             _vp]),
    "pg_layer_norm_workspace_size": (_i64, [_i64, _i32]),
    "pg_layer_norm_backward": (_i32, [_vp, _i64, _vp, _i64, _i32, _i64, _i32, _vp, _vp, _vp, _vp,
                                      _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp]),
    "pg_orthogonalize_workspace_size": (_i64, [_i64, _i32, _i32]),
    "pg_orthogonalize": (_i32, [_vp, _i32, _i64, _i32, _i32, _i32, _f32, _f32, _f32, _f32, _f32,
                                _vp, _vp, _i64, _vp]),
    "pg_flash_blocks": (_i32, [_P(PgLayout), _i32, _vp, _i64, _vp]),
    "pg_lru_cache_sim": (_i32, [_vp, _i64, _i32, _i64, _P(PgCacheStats)]),
}

_lib = None


class PagegramError(RuntimeError):
    def __init__(self, fn, status):
        msg = lib().pg_strerror(status).decode()
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


def lib():
    """The loaded library (ctypes.CDLL); raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m hashed_head_gram_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


# ----------------------------------------------------------------------------
# Struct builders


def make_layout(kind, K, r, S=1, pages=(), head_rows=(), hash_seed=0,
                use_signs=1, n_min=2, n_max=3, pad_id=0):
    """pg_layout from plain values; ``kind`` is "pagegram"/"engram" or 0/1.
    head_rows is flat in (order, head) order."""
    L = PgLayout()
    L.kind = {"pagegram": PG_PAGEGRAM, "engram": PG_ENGRAM}.get(kind, kind)
    L.n_min, L.n_max, L.K, L.S, L.r = n_min, n_max, K, S, r
    for i, p in enumerate(pages):
        L.pages[i] = int(p)
    for q, p in enumerate(head_rows):
        L.head_rows[q // K][q % K] = int(p)
    L.hash_seed = int(hash_seed)
    L.use_signs = int(use_signs)
    L.pad_id = int(pad_id)
    return L


def make_table(dtype, data, n_rows, scales=None):
    t = PgTable()
    t.dtype = dtype
    t.data = _ptr(data)
    t.scales = _ptr(scales)
    t.n_rows = int(n_rows)
    t._keep = (data, scales)
    return t


def make_fuse(gate, dtype, d, g=0.5, M=0, eps=1e-6, gamma_h=None, gamma_k=None,
              gamma_u=None, conv_w=None, conv_k=4, conv_dil=3, increment_only=0):
    f = PgFuse()
    f.gate, f.dtype, f.d, f.M = gate, dtype, int(d), int(M)
    f.g, f.eps = float(g), float(eps)
    f.gamma_h, f.gamma_k = _ptr(gamma_h), _ptr(gamma_k)
    f.gamma_u, f.conv_w = _ptr(gamma_u), _ptr(conv_w)
    f.conv_k, f.conv_dil, f.increment_only = int(conv_k), int(conv_dil), int(increment_only)
    f._keep = (gamma_h, gamma_k, gamma_u, conv_w)
    return f


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def _check(fn, status):
    if status != PG_OK:
        raise PagegramError(fn, status)


# ----------------------------------------------------------------------------
# Entry points (same names as the C ABI)


def pg_layout_rows(layout):
    n = _i64()
    _check("pg_layout_rows", lib().pg_layout_rows(ctypes.byref(layout), ctypes.byref(n)))
    return n.value


def pg_workspace_size(layout, fuse, B, T):
    v = lib().pg_workspace_size(ctypes.byref(layout) if layout is not None else None,
                                ctypes.byref(fuse), int(B), int(T))
    if v < 0:
        raise PagegramError("pg_workspace_size", v)
    return v


def pg_hash_version():
    return lib().pg_hash_version()


def pg_index(layout, tokens, canon_map, rows_out, signs_out, canon_out=None,
             hash_out=None, pages_out=None, dev_status=None, stream=None):
    """tokens int32 [B, T]; outputs as described in include/pagegram.h."""
    B, T = tokens.shape
    _check("pg_index", lib().pg_index(
        ctypes.byref(layout), _ptr(tokens), B, T, _ptr(canon_map), canon_map.numel(),
        _ptr(canon_out), _ptr(hash_out), _ptr(rows_out), _ptr(pages_out),
        _ptr(signs_out), _ptr(dev_status), _stream(stream)))


def pg_gather(layout, table, rows, signs, e_dtype, e_out, stream=None):
    _check("pg_gather", lib().pg_gather(
        ctypes.byref(layout), ctypes.byref(table), _ptr(rows), _ptr(signs),
        rows.shape[0], e_dtype, _ptr(e_out), _stream(stream)))


def pg_index_gather(layout, table, tokens, canon_map, e_dtype, e_out,
                    dev_status=None, stream=None):
    B, T = tokens.shape
    _check("pg_index_gather", lib().pg_index_gather(
        ctypes.byref(layout), ctypes.byref(table), _ptr(tokens), B, T,
        _ptr(canon_map), canon_map.numel(), e_dtype, _ptr(e_out),
        _ptr(dev_status), _stream(stream)))


def pg_project_gate(fuse, e, B, T, W, resid, out, workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("pg_project_gate", lib().pg_project_gate(
        ctypes.byref(fuse), _ptr(e), int(B), int(T), e.shape[-1], _ptr(W),
        _ptr(resid), _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)))


def pg_forward(layout, table, fuse, tokens, canon_map, W, resid, out, workspace,
               dev_status=None, stream=None):
    B, T = tokens.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("pg_forward", lib().pg_forward(
        ctypes.byref(layout), ctypes.byref(table), ctypes.byref(fuse), _ptr(tokens),
        B, T, _ptr(canon_map), canon_map.numel(), _ptr(W), _ptr(resid), _ptr(out),
        _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream)))


def pg_forward_noalloc(layout, table, fuse, tokens, canon_map, W, resid, out,
                       dev_status=None, stream=None):
    B, T = tokens.shape
    _check("pg_forward_noalloc", lib().pg_forward_noalloc(
        ctypes.byref(layout), ctypes.byref(table), ctypes.byref(fuse), _ptr(tokens),
        B, T, _ptr(canon_map), canon_map.numel(), _ptr(W), _ptr(resid), _ptr(out),
        _ptr(dev_status), _stream(stream)))


NOALLOC_SCRATCH_BYTES = 64 << 20


def records_bytes(layout, n_tok):
    """Bytes of pg_index_records' output: 16 per (head slot, token)."""
    return 16 * n_tok * (layout.n_max - layout.n_min + 1) * layout.K


def pg_index_records(layout, tokens, canon_map, rec_out, dev_status=None, stream=None):
    B, T = tokens.shape
    _check("pg_index_records", lib().pg_index_records(
        ctypes.byref(layout), _ptr(tokens), B, T, _ptr(canon_map), canon_map.numel(),
        _ptr(rec_out), _ptr(dev_status), _stream(stream)))


def pg_project_gathered(layout, table, fuse, rec, B, T, W, resid, out, stream=None):
    _check("pg_project_gathered", lib().pg_project_gathered(
        ctypes.byref(layout), ctypes.byref(table), ctypes.byref(fuse), _ptr(rec), int(B),
        int(T), _ptr(W), _ptr(resid), _ptr(out), _stream(stream)))


# ----------------------------------------------------------------------------
# The Engram gate's three stages (pg_project_gate runs them in order)


def _ws_bytes(workspace):
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def pg_engram_project(fuse, e, B, T, W, h, workspace, stream=None):
    _check("pg_engram_project", lib().pg_engram_project(
        ctypes.byref(fuse), _ptr(e), int(B), int(T), e.shape[-1], _ptr(W), _ptr(h),
        _ptr(workspace), _ws_bytes(workspace), _stream(stream)))


def pg_engram_project_fp8(fuse, e8, B, T, W8, e_scale_exp, w_scale_exp, h, workspace,
                          stream=None):
    _check("pg_engram_project_fp8", lib().pg_engram_project_fp8(
        ctypes.byref(fuse), _ptr(e8), int(B), int(T), e8.shape[-1], _ptr(W8),
        int(e_scale_exp), int(w_scale_exp), _ptr(h), _ptr(workspace), _ws_bytes(workspace),
        _stream(stream)))


def pg_engram_gate(fuse, B, T, workspace, stream=None):
    _check("pg_engram_gate", lib().pg_engram_gate(
        ctypes.byref(fuse), int(B), int(T), _ptr(workspace), _ws_bytes(workspace),
        _stream(stream)))


def pg_engram_mix(fuse, B, T, h, out, workspace, stream=None):
    _check("pg_engram_mix", lib().pg_engram_mix(
        ctypes.byref(fuse), int(B), int(T), _ptr(h), _ptr(out), _ptr(workspace),
        _ws_bytes(workspace), _stream(stream)))


def pg_read_probe(src, sink, stream=None):
    """Streaming read of the whole tensor src (measurement utility)."""
    _check("pg_read_probe", lib().pg_read_probe(
        _ptr(src), src.numel() * src.element_size(), _ptr(sink), _stream(stream)))


# ----------------------------------------------------------------------------
# Staging from a host-resident table


def pg_stage_geometry(layout, table_dtype, n_tok, unit_kind=0):
    """(rows per unit, most units per step, workspace bytes); unit_kind
    PG_STAGE_PAGE (0) or PG_STAGE_ROW (1)."""
    u, m, w = _i64(), _i64(), _i64()
    _check("pg_stage_geometry", lib().pg_stage_geometry(
        ctypes.byref(layout), table_dtype, int(unit_kind), int(n_tok), ctypes.byref(u),
        ctypes.byref(m), ctypes.byref(w)))
    return u.value, m.value, w.value


def pg_stage_rows(layout, src, rows, cache, cache_rows, n_units, workspace, unit_first=None,
                  unit_kind=0, stream=None):
    """rows int64 [N, O, K] (device); src / cache pg_table structures."""
    _check("pg_stage_rows", lib().pg_stage_rows(
        ctypes.byref(layout), ctypes.byref(src), int(unit_kind), _ptr(rows), rows.shape[0],
        ctypes.byref(cache),
        _ptr(cache_rows), _ptr(n_units), _ptr(unit_first), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def pg_gather_staged(layout, cache, cache_rows, signs, e_dtype, e_out, stream=None):
    _check("pg_gather_staged", lib().pg_gather_staged(
        ctypes.byref(layout), ctypes.byref(cache), _ptr(cache_rows), _ptr(signs),
        cache_rows.shape[0], e_dtype, _ptr(e_out), _stream(stream)))


# ----------------------------------------------------------------------------
# FP8 (E4M3) operands


def pg_quantize_fp8(src, src_dtype, scale_exp, dst, stream=None):
    """dst (uint8, same element count) = E4M3(src * 2^scale_exp)."""
    _check("pg_quantize_fp8", lib().pg_quantize_fp8(
        _ptr(src), src_dtype, src.numel(), int(scale_exp), _ptr(dst), _stream(stream)))


def pg_index_gather_fp8(layout, table, tokens, canon_map, e_scale_exp, e_out,
                        dev_status=None, stream=None):
    B, T = tokens.shape
    _check("pg_index_gather_fp8", lib().pg_index_gather_fp8(
        ctypes.byref(layout), ctypes.byref(table), _ptr(tokens), B, T,
        _ptr(canon_map), canon_map.numel(), int(e_scale_exp), _ptr(e_out),
        _ptr(dev_status), _stream(stream)))


def pg_project_gate_fp8(fuse, e8, B, T, W8, e_scale_exp, w_scale_exp, resid, out,
                        workspace=None, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("pg_project_gate_fp8", lib().pg_project_gate_fp8(
        ctypes.byref(fuse), _ptr(e8), int(B), int(T), e8.shape[-1], _ptr(W8),
        int(e_scale_exp), int(w_scale_exp), _ptr(resid), _ptr(out), _ptr(workspace),
        ws_bytes, _stream(stream)))


def pg_forward_fp8(layout, table, fuse, tokens, canon_map, W8, e_scale_exp, w_scale_exp,
                   resid, out, workspace, dev_status=None, stream=None):
    B, T = tokens.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("pg_forward_fp8", lib().pg_forward_fp8(
        ctypes.byref(layout), ctypes.byref(table), ctypes.byref(fuse), _ptr(tokens),
        B, T, _ptr(canon_map), canon_map.numel(), _ptr(W8), int(e_scale_exp),
        int(w_scale_exp), _ptr(resid), _ptr(out), _ptr(workspace), ws_bytes,
        _ptr(dev_status), _stream(stream)))


# ----------------------------------------------------------------------------
# Backward pass and table update


def pg_backward_workspace_size(layout, fuse, B, T):
    v = lib().pg_backward_workspace_size(ctypes.byref(layout), ctypes.byref(fuse), int(B),
                                         int(T))
    if v < 0:
        raise PagegramError("pg_backward_workspace_size", v)
    return v


def pg_backward_scalar(layout, fuse, rows, signs, e, dy, W, B, T, dW, de, urows, ugrad,
                       n_unique, workspace, stream=None):
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("pg_backward_scalar", lib().pg_backward_scalar(
        ctypes.byref(layout), ctypes.byref(fuse), _ptr(rows), _ptr(signs), _ptr(e), _ptr(dy),
        _ptr(W), int(B), int(T), _ptr(dW), _ptr(de), _ptr(urows), _ptr(ugrad),
        _ptr(n_unique), _ptr(workspace), ws_bytes, _stream(stream)))


def pg_row_rms_step(layout, urows, ugrad, n_unique, max_unique, table, vhat, last_step, step,
                    lr, beta2=0.95, weight_decay=0.0, eps=1e-8, stream=None):
    _check("pg_row_rms_step", lib().pg_row_rms_step(
        ctypes.byref(layout), _ptr(urows), _ptr(ugrad), _ptr(n_unique), int(max_unique),
        _ptr(table), _ptr(vhat), _ptr(last_step), int(step), float(lr), float(beta2),
        float(weight_decay), float(eps), _stream(stream)))


def pg_row_rms_flush(layout, table, vhat, last_step, step, lr, beta2=0.95, weight_decay=0.0,
                     stream=None):
    _check("pg_row_rms_flush", lib().pg_row_rms_flush(
        ctypes.byref(layout), _ptr(table), _ptr(vhat), _ptr(last_step), int(step), float(lr),
        float(beta2), float(weight_decay), _stream(stream)))


# ----------------------------------------------------------------------------
# The training step around the memory: token embedding, layer norm,
# orthogonalised update. Rows are the last dimension; a tensor of rows may be a
# slice of wider rows (any one row stride). Every tensor of a call lives on one
# GPU; the work goes to that GPU's current stream, or to `stream`.


def _dtype(fn, name, t):
    code = _dtype_codes().get(t.dtype)
    if code is None:
        raise ValueError(f"{fn}: {name} is {t.dtype}, not float32 or bfloat16")
    return code


_codes = {}


def _dtype_codes():
    if not _codes:
        import torch
        _codes.update({torch.float32: PG_F32, torch.bfloat16: PG_BF16})
    return _codes


def _rows(fn, name, t):
    """(rows, row stride) of t, whose last dimension is a row."""
    if t.dim() != 2:
        try:
            t = t.view(-1, t.shape[-1])
        except (RuntimeError, IndexError):
            raise ValueError(f"{fn}: the rows of {name} have no single stride") from None
    n, d = t.shape
    ld, one = t.stride()
    if one != 1 and d > 1 and n:
        raise ValueError(f"{fn}: the rows of {name} are not contiguous")
    return n, ld if n > 1 else d


def _flat(fn, name, t, dtype, size, dev, at_least=False):
    """t is contiguous, of dtype, with size elements, on dev."""
    n = None if t is None else t.numel()
    if n is None or (n != size and not (at_least and n > size)) or t.dtype != dtype or \
            t.device != dev or not t.is_contiguous():
        raise ValueError(f"{fn}: {name} must be a contiguous {dtype} tensor of {size} elements "
                         f"on {dev}")


def _work(fn, t, dev):
    """A workspace: uint8 on dev, or None, which the library takes where it needs none."""
    import torch
    if t is not None:
        _flat(fn, "workspace", t, torch.uint8, 0, dev, at_least=True)


def _like(fn, name, t, ref):
    if t is None or t.shape != ref.shape or t.dtype != ref.dtype or t.device != ref.device:
        raise ValueError(f"{fn}: {name} must be a {ref.dtype} tensor of shape "
                         f"{tuple(ref.shape)} on {ref.device}")


def _gpu(fn, name, t):
    if t is None or not t.is_cuda:
        raise ValueError(f"{fn}: {name} is {'None' if t is None else t.device}, not on a GPU")
    return t.device


def _call(fn, dev, stream, *args):
    """fn(*args, stream) with dev the current device; without a stream, on dev's current one
    (its raw handle: building a torch.cuda.Stream takes longer than a small kernel's launch)."""
    import torch
    f = getattr(_lib or lib(), fn)
    index = dev.index
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    else:
        raw = _stream(stream)
        if getattr(stream, "device", dev) != dev:
            raise ValueError(f"{fn}: the stream is on {stream.device}, the tensors on {dev}")
    if index == torch._C._cuda_getDevice():
        status = f(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = f(*args, raw)
    if status != PG_OK:
        raise PagegramError(fn, status)


def _in32(v):
    """v, or the end of int32 that it lies beyond: ctypes would pass its low bits. The library
    refuses the ends like any size past its limits."""
    return v if -2**31 <= v < 2**31 else 2**31 - 1 if v > 0 else -2**31


def _in64(v):
    return v if -2**63 <= v < 2**63 else 2**63 - 1 if v > 0 else -2**63


def _size(fn, *args):
    f = getattr(lib(), fn)
    v = f(*((_in32 if t is _i32 else _in64)(int(a)) for a, t in zip(args, f.argtypes)))
    if v < 0:
        raise PagegramError(fn, v)
    return v


def pg_embed(table, tokens, out, scale=1.0, dev_status=None, stream=None):
    """out [..., d] = scale * table[tokens]; tokens int32, contiguous. table (make_table) must
    hold [n_rows, d] of float32 or bfloat16 on out's GPU."""
    import torch
    dev = _gpu("pg_embed", "out", out)
    n, ld = _rows("pg_embed", "out", out)
    _flat("pg_embed", "tokens", tokens, torch.int32, n, dev)
    if dev_status is not None:
        _flat("pg_embed", "dev_status", dev_status, torch.int32, 1, dev, at_least=True)
    d = out.shape[-1]
    data = table._keep[0] if hasattr(table, "_keep") else None
    if hasattr(data, "numel") and table.dtype != PG_NF4:
        want = torch.float32 if table.dtype == PG_F32 else torch.bfloat16
        _flat("pg_embed", "table data", data, want, table.n_rows * d, dev)
    _call("pg_embed", dev, stream, ctypes.byref(table), _in32(d), float(scale), _ptr(tokens), n,
          _dtype("pg_embed", "out", out), _ptr(out), ld, _ptr(dev_status))


def pg_embed_workspace_size(n_tok, V, d):
    return _size("pg_embed_workspace_size", n_tok, V, d)


def _embed_dout(fn, dout, tokens, workspace):
    import torch
    dev = _gpu(fn, "dout", dout)
    n, ld = _rows(fn, "dout", dout)
    _flat(fn, "tokens", tokens, torch.int32, n, dev)
    _work(fn, workspace, dev)
    return dev, n, ld, dout.shape[-1], _dtype(fn, "dout", dout)


def pg_embed_backward(dout, tokens, V, urows, ugrad, n_unique, workspace, scale=1.0,
                      stream=None):
    """Touched rows of the table gradient: urows int64 and ugrad float32 with room for
    min(n_tok, V) rows, n_unique int64 [1]; workspace uint8."""
    import torch
    fn = "pg_embed_backward"
    dev, n, ld, d, dt = _embed_dout(fn, dout, tokens, workspace)
    cap = min(n, int(V))
    _flat(fn, "urows", urows, torch.int64, cap, dev, at_least=True)
    _flat(fn, "ugrad", ugrad, torch.float32, cap * d, dev, at_least=True)
    _flat(fn, "n_unique", n_unique, torch.int64, 1, dev, at_least=True)
    _call(fn, dev, stream, _ptr(dout), dt, ld, _ptr(tokens), n, _in64(int(V)), _in32(d),
          float(scale), _ptr(urows), _ptr(ugrad), _ptr(n_unique), _ptr(workspace), _ws_bytes(workspace))


def pg_embed_backward_dense(dout, tokens, dtable, workspace, scale=1.0, accumulate=0,
                            stream=None):
    """dtable float32 [V, d], written whole or (accumulate=1) added to."""
    import torch
    fn = "pg_embed_backward_dense"
    dev, n, ld, d, dt = _embed_dout(fn, dout, tokens, workspace)
    V = dtable.shape[0]
    _flat(fn, "dtable", dtable, torch.float32, V * d, dev)
    _call(fn, dev, stream, _ptr(dout), dt, ld, _ptr(tokens), n, V, _in32(d), float(scale),
          _ptr(dtable), _in32(int(accumulate)), _ptr(workspace), _ws_bytes(workspace))


def pg_layer_norm(x, gamma, beta, y, eps=1e-5, mean=None, rstd=None, stream=None):
    """y = layer norm of the rows of x (y may be x); gamma, beta float32 [d] (beta or None);
    mean, rstd float32 [rows] or None."""
    import torch
    fn = "pg_layer_norm"
    dev = _gpu(fn, "x", x)
    n, ldx = _rows(fn, "x", x)
    _like(fn, "y", y, x)
    ldy = _rows(fn, "y", y)[1]
    d = x.shape[-1]
    _flat(fn, "gamma", gamma, torch.float32, d, dev)
    if beta is not None:
        _flat(fn, "beta", beta, torch.float32, d, dev)
    if mean is not None:
        _flat(fn, "mean", mean, torch.float32, n, dev)
    if rstd is not None:
        _flat(fn, "rstd", rstd, torch.float32, n, dev)
    _call(fn, dev, stream, _ptr(x), _dtype(fn, "x", x), n, _in32(d), ldx, _ptr(gamma), _ptr(beta),
          float(eps), _ptr(y), ldy, _ptr(mean), _ptr(rstd))


def pg_layer_norm_workspace_size(n, d):
    return _size("pg_layer_norm_workspace_size", n, d)


def pg_layer_norm_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, workspace, add=None,
                           stream=None):
    """dx (may be dy or add), dgamma and dbeta (or None) from pg_layer_norm's mean and rstd; add:
    a gradient added to dx, or None."""
    import torch
    fn = "pg_layer_norm_backward"
    dev = _gpu(fn, "x", x)
    n, ldx = _rows(fn, "x", x)
    d = x.shape[-1]
    _like(fn, "dy", dy, x)
    _like(fn, "dx", dx, x)
    ldadd = 0
    if add is not None:
        _like(fn, "add", add, x)
        ldadd = _rows(fn, "add", add)[1]
    _flat(fn, "gamma", gamma, torch.float32, d, dev)
    _flat(fn, "mean", mean, torch.float32, n, dev)
    _flat(fn, "rstd", rstd, torch.float32, n, dev)
    _flat(fn, "dgamma", dgamma, torch.float32, d, dev)
    if dbeta is not None:
        _flat(fn, "dbeta", dbeta, torch.float32, d, dev)
    _work(fn, workspace, dev)
    _call(fn, dev, stream, _ptr(dy), _rows(fn, "dy", dy)[1], _ptr(x), ldx, _dtype(fn, "x", x), n,
          _in32(d), _ptr(gamma), _ptr(mean), _ptr(rstd), _ptr(add), ldadd, _ptr(dx),
          _rows(fn, "dx", dx)[1], _ptr(dgamma), _ptr(dbeta), _ptr(workspace),
          _ws_bytes(workspace))


def pg_orthogonalize_workspace_size(n_mat, rows, cols):
    return _size("pg_orthogonalize_workspace_size", n_mat, rows, cols)


def pg_orthogonalize(G, out, workspace, steps=5, coef=(3.4445, -4.7750, 2.0315), eps=1e-7,
                     scale=1.0, stream=None):
    """out (bfloat16) = scale * the Newton-Schulz iterate of each matrix of G [..., rows, cols]
    (float32 or bfloat16, contiguous)."""
    import torch
    fn = "pg_orthogonalize"
    dev = _gpu(fn, "G", G)
    if G.dim() < 2 or not G.is_contiguous() or out is None or out.shape != G.shape:
        raise ValueError(f"{fn}: G must be contiguous [..., rows, cols], out of its shape")
    rows, cols = G.shape[-2:]
    n_mat = 1
    for s in G.shape[:-2]:
        n_mat *= s
    _flat(fn, "out", out, torch.bfloat16, G.numel(), dev)
    _work(fn, workspace, dev)
    a, b, c = (float(v) for v in coef)
    _call(fn, dev, stream, _ptr(G), _dtype(fn, "G", G), n_mat, _in32(rows), _in32(cols),
          _in32(int(steps)), a, b, c, float(eps), float(scale), _ptr(out), _ptr(workspace),
          _ws_bytes(workspace))


# ----------------------------------------------------------------------------
# Flash page-cache simulation (host arrays)


def pg_flash_blocks(layout, table_dtype, rows):
    """4 KiB block of each row; rows: host int64 numpy array of any shape."""
    import numpy as np
    rows = np.ascontiguousarray(rows, dtype=np.int64)
    out = np.empty_like(rows)
    _check("pg_flash_blocks", lib().pg_flash_blocks(
        ctypes.byref(layout), int(table_dtype), rows.ctypes.data, rows.size,
        out.ctypes.data))
    return out


def pg_lru_cache_sim(blocks, capacity_blocks):
    """LRU run over blocks [n_tok, per_token] (host int64); returns the counters."""
    import numpy as np
    blocks = np.ascontiguousarray(blocks, dtype=np.int64)
    n_tok = blocks.shape[0]
    per = int(blocks.size // n_tok) if n_tok else 1
    st = PgCacheStats()
    _check("pg_lru_cache_sim", lib().pg_lru_cache_sim(
        blocks.ctypes.data, n_tok, per, int(capacity_blocks), ctypes.byref(st)))
    return dict(tokens=st.tokens, lookups=st.lookups, distinct=st.distinct,
                misses=st.misses)
