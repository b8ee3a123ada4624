"""Python binding of the decoder operators (include/oeq.h, "Decoder operators"): embedding lookup and
its gradient, root-mean-square norm with the residual's addition, causal attention over packed
sequences.  Names follow the C ABI; argument marshalling only, as in readout.py.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _check, lib
from .readout import (_DTYPES, _F32, _I32, _I64, _attn, _attn_desc, _dense, _head, _like, _raw_stream, _row_stride, _scratch,
                      _typed)

_E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------

def _index(index, dev):
    """(rows, bytes of an element) of an index vector."""
    if not isinstance(index, torch.Tensor) or index.get_device() != dev:
        raise TypeError(f"index must be a tensor on device cuda:{dev}")
    if index.dtype is not _I64 and index.dtype is not torch.int32:
        raise TypeError(f"index must be int32 or int64, got {index.dtype}")
    if index.dim() != 1 or not index.is_contiguous():
        raise ValueError("index must be a contiguous vector")
    return index.shape[0], 8 if index.dtype is _I64 else 4


def oeq_embedding_fwd(table, index, scale: float = 1.0, out=None):
    """scale * table[index] for table [table rows, columns] and index [rows] (int32 or int64); an index
    outside the table gives a row of zeros.  The rows of table and out may be strided."""
    code, dev = _head(table, "table")
    ld = _row_stride(table, "table")
    n_table, cols = table.shape
    rows, size = _index(index, dev)
    if out is None:
        out, ld_o = table.new_empty((rows, cols)), cols
    else:
        _typed(out, table.dtype, dev, "out")
        if out.shape != (rows, cols):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {(rows, cols)}")
        ld_o = _row_stride(out, "out")
    st = lib().oeq_embedding_fwd(code, n_table, cols, rows, table.data_ptr(), ld, index.data_ptr(), size, scale,
                                 out.data_ptr(), ld_o, _raw_stream(dev))
    if st:
        _check(st)
    return out


@functools.lru_cache(maxsize=4096)
def _embedding_bytes(code, n_table, n_cols, n_rows):
    b = ctypes.c_size_t()
    _check(lib().oeq_embedding_workspace_size(code, n_table, n_cols, n_rows, ctypes.byref(b)))
    return b.value


def oeq_embedding_workspace_size(n_table: int, n_cols: int, n_rows: int, dtype=torch.float32):
    """Workspace bytes of the gradient."""
    return _embedding_bytes(_DTYPES[dtype], n_table, n_cols, n_rows)


def oeq_embedding_bwd(index, grad_out, n_table: int, scale: float = 1.0, out=None, workspace=None):
    """Gradient [n_table, columns] of <grad_out, oeq_embedding_fwd(table, index, scale)> to the table, of
    grad_out's type.  `out` may supply it."""
    code, dev = _head(grad_out, "grad_out")
    ld = _row_stride(grad_out, "grad_out")
    rows, cols = grad_out.shape
    n, size = _index(index, dev)
    if n != rows:
        raise ValueError(f"index has {n} rows, grad_out {rows}")
    need = _embedding_bytes(code, n_table, cols, rows)
    if out is None:
        out, ld_o = grad_out.new_empty((n_table, cols)), cols
    else:
        _typed(out, grad_out.dtype, dev, "out")
        if out.shape != (n_table, cols):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {(n_table, cols)}")
        ld_o = _row_stride(out, "out")
    keep, ws, nbytes = _scratch(need, workspace, grad_out.device)
    st = lib().oeq_embedding_bwd(code, n_table, cols, rows, index.data_ptr(), size, scale, grad_out.data_ptr(), ld,
                                 out.data_ptr(), ld_o, ws, nbytes, _raw_stream(dev))
    if st:
        _check(st)
    return out


# ---------------------------------------------------------------------------
# rms norm
# ---------------------------------------------------------------------------

@functools.lru_cache(maxsize=4096)
def oeq_rms_norm_workspace_size(n_rows: int, n_cols: int):
    """Workspace bytes of the backward."""
    b = ctypes.c_size_t()
    _check(lib().oeq_rms_norm_workspace_size(n_rows, n_cols, ctypes.byref(b)))
    return b.value


def _rms_fwd(x, weight, residual, eps, out, total, out_dtype):
    """(out, scale, rstd, sum)"""
    code, dev = _head(x, "x")
    ld = _row_stride(x, "x")
    rows, cols = x.shape
    out_dtype = out_dtype or x.dtype
    w = _dense(weight, (cols,), _F32, dev, "weight")
    res, ld_r, at, ld_s = None, 0, None, 0
    if residual is not None:
        ld_r = _like(residual, x, dev, "residual")
        res = residual.data_ptr()
        if total is None:
            total, ld_s = x.new_empty((rows, cols)), cols
        else:
            ld_s = _like(total, x, dev, "sum")
        at = total.data_ptr()
    elif total is not None:
        raise ValueError("sum without a residual")
    else:
        total = x
    if out is None:
        out, ld_o = x.new_empty((rows, cols), dtype=out_dtype), cols
    else:
        _typed(out, out_dtype, dev, "out")
        if out.shape != (rows, cols):
            raise ValueError(f"out has shape {tuple(out.shape)}, expected {(rows, cols)}")
        ld_o = _row_stride(out, "out")
    rstd = x.new_empty(rows, dtype=_F32)
    scale = x.new_empty(rows, dtype=_F32) if out_dtype is _E4M3 else None
    st = lib().oeq_rms_norm_fwd(code, rows, cols, eps, x.data_ptr(), ld, res, ld_r, w, at, ld_s, out.data_ptr(), ld_o,
                                None if scale is None else scale.data_ptr(), rstd.data_ptr(), _raw_stream(dev))
    if st:
        _check(st)
    return out, scale, rstd, total


def oeq_rms_norm_fwd(x, weight=None, residual=None, eps: float = 1e-5, out=None, sum=None):
    """(out, rstd, sum): root-mean-square norm of the rows of x + residual [rows, columns], times weight
    (fp32 [columns]).  sum is x + residual in x's type (the residual stream; x itself where there is
    no residual), rstd fp32 [rows].  `sum` may supply that tensor, x and residual themselves among
    them.  Rows may be strided."""
    out, _, rstd, total = _rms_fwd(x, weight, residual, eps, out, sum, None)
    return out, rstd, total


def oeq_rms_norm_e4m3_fwd(x, weight=None, residual=None, eps: float = 1e-5, out=None, sum=None):
    """(out, scale, rstd, sum): oeq_rms_norm_fwd with out in 8 bits (float8_e4m3fn) and a scale for each
    row (fp32 [rows]): the norm is out * scale[:, None]."""
    return _rms_fwd(x, weight, residual, eps, out, sum, _E4M3)


def oeq_rms_norm_bwd(sum, rstd, grad_out, weight=None, grad_sum=None, need=("x", "weight"), out=None, workspace=None):
    """(grad_x, grad_weight) of <grad_out, norm> + <grad_sum, sum> from the forward's sum and rstd; grad_x is
    the gradient to x and to the residual alike.  Entries not in `need` are None; `out` may supply
    grad_x, grad_out and grad_sum themselves among them."""
    code, dev = _head(sum, "sum")
    ld = _row_stride(sum, "sum")
    rows, cols = sum.shape
    w, rs = _dense(weight, (cols,), _F32, dev, "weight"), _dense(rstd, (rows,), _F32, dev, "rstd")
    ld_g = _like(grad_out, sum, dev, "grad_out")
    gs, ld_gs = None, 0
    if grad_sum is not None:
        ld_gs = _like(grad_sum, sum, dev, "grad_sum")
        gs = grad_sum.data_ptr()
    gx = gw = keep = ws = None
    ld_x = nbytes = 0
    if "x" in need:
        if out is None:
            gx, ld_x = sum.new_empty((rows, cols)), cols
        else:
            gx, ld_x = out, _like(out, sum, dev, "grad_x")
    if "weight" in need:
        gw = sum.new_empty(cols, dtype=_F32)
        keep, ws, nbytes = _scratch(oeq_rms_norm_workspace_size(rows, cols), workspace, sum.device)
    st = lib().oeq_rms_norm_bwd(code, rows, cols, sum.data_ptr(), ld, w, rs, grad_out.data_ptr(), ld_g, gs, ld_gs,
                                None if gx is None else gx.data_ptr(), ld_x, None if gw is None else gw.data_ptr(), ws,
                                nbytes, _raw_stream(dev))
    if st:
        _check(st)
    return gx, gw


# ---------------------------------------------------------------------------
# causal attention
# ---------------------------------------------------------------------------

def oeq_causal_attn_workspace_size(q_shape, k_shape, n_struct: int, dtype=torch.float32):
    """Workspace bytes (forward, backward) for q of shape [Tq, H, D] and k, v of [Tk, Hkv, D]."""
    (tq, h, d), (tk, hk, _) = q_shape, k_shape
    return _attn_desc(True, _DTYPES[dtype], n_struct, h, hk, d, tq, tk, 0, 0, 0, 0, 0, 0, 1.0, 0.0)[1:]


def oeq_causal_attn_fwd(q, k, v, q_ptr, k_ptr, scale=None, key_mask=None, k_len=None, p_drop: float = 0.0, rng=None,
                        out=None, lse=None, workspace=None):
    """(out, lse): causal attention of q [Tq, H, D] to the states k, v [Tk, Hkv, D] of their sequence
    (q_ptr, k_ptr: int32 row pointers over the same sequences; the last query stands at the last
    state).  k_len (int32 [sequences]): the states in use of each, the first of its rows, for caches
    with rows to spare.  The other arguments are those of oeq_cross_attn_fwd."""
    dev, (desc, fwd_bytes, _), operands = _attn(q, k, v, q_ptr, k_ptr, scale, key_mask, p_drop, rng, True)
    used = _dense(k_len, (q_ptr.shape[0] - 1,), _I32, dev, "k_len")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _dense(out, q.shape, q.dtype, dev, "out")
    if lse is None:
        lse = torch.empty(q.shape[:2], dtype=_F32, device=q.device)
    else:
        _dense(lse, q.shape[:2], _F32, dev, "lse")
    keep, ws, nbytes = _scratch(fwd_bytes, workspace, q.device)
    st = lib().oeq_causal_attn_fwd(desc, *operands[:2], used, *operands[2:], out.data_ptr(), lse.data_ptr(), ws, nbytes,
                                   _raw_stream(dev))
    if st:
        _check(st)
    return out, lse


def oeq_causal_attn_bwd(q, k, v, q_ptr, k_ptr, out, lse, grad_out, scale=None, key_mask=None, p_drop: float = 0.0,
                        rng=None, need=("q", "k", "v"), grads=None, workspace=None):
    """(grad_q, grad_k, grad_v) of <grad_out, out> from the forward's operands (without k_len), out and lse;
    entries not in `need` are None.  `grads` may supply preallocated gradients (contiguous)."""
    dev, (desc, _, bwd_bytes), operands = _attn(q, k, v, q_ptr, k_ptr, scale, key_mask, p_drop, rng, True)
    saved = (_dense(out, q.shape, q.dtype, dev, "out"), _dense(lse, q.shape[:2], _F32, dev, "lse"),
             _dense(grad_out, q.shape, q.dtype, dev, "grad_out"))
    if grads is None:
        grads = tuple(torch.empty_like(t, memory_format=torch.contiguous_format) if n in need else None
                      for n, t in (("q", q), ("k", k), ("v", k)))
    addresses = tuple(_dense(g, t.shape, q.dtype, dev, n)
                      for g, t, n in zip(grads, (q, k, k), ("grad_q", "grad_k", "grad_v")))
    keep, ws, nbytes = _scratch(bwd_bytes, workspace, q.device)
    st = lib().oeq_causal_attn_bwd(desc, *operands, *saved, *addresses, ws, nbytes, _raw_stream(dev))
    if st:
        _check(st)
    return tuple(grads)
