"""Python binding of the readout operators (include/oeq.h, "Readout operators"): group norm
with an activation, dropout from a counter-based generator, cross attention over ragged
structures.  Names follow the C ABI.

Argument marshalling only, as in the rest of the package.  The calls are small next to a
convolution, and a step on a few molecules is bound by the host, so the checks read each
tensor's properties once and the workspace sizes, a function of the shapes alone, are
remembered per shape.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import OEQ_BF16, OEQ_F16, OEQ_F32, _AttnDesc, _check, lib

_DTYPES = {torch.float32: OEQ_F32, torch.float16: OEQ_F16, torch.bfloat16: OEQ_BF16}
_ACTS = {"none": 0, "silu": 1}
_F32, _I32, _I64, _U8 = torch.float32, torch.int32, torch.int64, torch.uint8

_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _head(t, name):
    """(oeq_dtype, device number) of the operand that decides both."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    dev = t.get_device()
    if dev != _current_device():
        raise ValueError(f"{name} is on device {dev}, the current device is {_current_device()}")
    return code, dev


def _typed(t, dtype, dev, name):
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:  # -1 on the host
        raise TypeError(f"{name} must be a tensor on device cuda:{dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _dense(t, shape, dtype, dev, name):
    """Address of a contiguous operand (None: not given)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype is not dtype:
        _typed(t, dtype, dev, name)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _row_stride(t, name):
    """Row stride of a 2-D operand whose rows are contiguous and do not overlap."""
    if t.dim() != 2:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [rows, columns]")
    cols = t.shape[1]
    if t.is_contiguous():
        return cols
    rows, columns = t.stride()
    if cols > 1 and columns != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    if t.shape[0] < 2:
        return cols
    if rows < cols:
        raise ValueError(f"the rows of {name} overlap")
    return rows


def _like(t, x, dev, name):
    """Row stride of a 2-D operand of x's shape and type."""
    _typed(t, x.dtype, dev, name)
    if t.shape != x.shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(x.shape)}")
    return _row_stride(t, name)


def _scratch(nbytes, workspace, device):
    """(tensor to keep, address, bytes): the caller's workspace, or a 256-byte aligned one."""
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device != device:
            raise TypeError(f"workspace must be a tensor on device {device}")
        if not workspace.is_contiguous():  # else it may own fewer bytes than it counts
            raise ValueError("workspace must be contiguous")
        return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if nbytes == 0:
        return None, None, 0
    raw = torch.empty(nbytes + 256, dtype=_U8, device=device)
    at = raw.data_ptr()
    return raw, at + (-at) % 256, nbytes


# ---------------------------------------------------------------------------
# group norm
# ---------------------------------------------------------------------------

def _structures(ptr, dev, name="ptr"):
    if not isinstance(ptr, torch.Tensor) or ptr.get_device() != dev or ptr.dtype is not _I32:
        _typed(ptr, _I32, dev, name)
    if ptr.dim() != 1 or ptr.shape[0] < 1 or not ptr.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of [structures + 1] values")
    return ptr.shape[0] - 1


@functools.lru_cache(maxsize=4096)
def oeq_group_norm_workspace_size(n_rows: int, n_struct: int, n_channels: int, n_groups: int):
    """Workspace bytes (forward, backward)."""
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().oeq_group_norm_workspace_size(n_rows, n_struct, n_channels, n_groups, ctypes.byref(f),
                                               ctypes.byref(b)))
    return f.value, b.value


def _act(act):
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    return code


def oeq_group_norm_fwd(x, ptr, n_groups: int, weight=None, bias=None, eps: float = 1e-5, act: str = "none", out=None,
                       workspace=None):
    """(out, mean, rstd): group norm of x [rows, C] over the rows of each structure
    (ptr [structures + 1] int32), channels last, with an activation ("none" or "silu").
    weight and bias are fp32 [C]; mean and rstd are fp32 [structures, n_groups].  The rows
    of x and out may be strided."""
    code, dev = _head(x, "x")
    ld = _row_stride(x, "x")
    rows, C = x.shape
    B = _structures(ptr, dev)
    w, b = _dense(weight, (C,), _F32, dev, "weight"), _dense(bias, (C,), _F32, dev, "bias")
    if out is None:
        out = x.new_empty((rows, C))
        ld_out = C
    else:
        ld_out = _like(out, x, dev, "out")
    need = oeq_group_norm_workspace_size(rows, B, C, n_groups)[0]
    mean, rstd = torch.empty((2, B, n_groups), dtype=_F32, device=x.device).unbind(0)
    keep, ws, nbytes = _scratch(need, workspace, x.device)
    st = lib().oeq_group_norm_fwd(code, rows, B, C, n_groups, _act(act), eps, ptr.data_ptr(), x.data_ptr(), ld, w, b,
                                  out.data_ptr(), ld_out, mean.data_ptr(), rstd.data_ptr(), ws, nbytes,
                                  _raw_stream(dev))
    if st:
        _check(st)
    return out, mean, rstd


def oeq_group_norm_bwd(x, ptr, n_groups: int, mean, rstd, grad_out, weight=None, bias=None, act: str = "none",
                       need=("x", "weight", "bias"), out=None, workspace=None):
    """(grad_x, grad_weight, grad_bias) of <grad_out, oeq_group_norm_fwd(x, ...)>; entries not in
    `need` are None.  `out` may supply the grad_x tensor."""
    code, dev = _head(x, "x")
    ld = _row_stride(x, "x")
    rows, C = x.shape
    B = _structures(ptr, dev)
    w, b = _dense(weight, (C,), _F32, dev, "weight"), _dense(bias, (C,), _F32, dev, "bias")
    nbytes = oeq_group_norm_workspace_size(rows, B, C, n_groups)[1]
    mu, rs = _dense(mean, (B, n_groups), _F32, dev, "mean"), _dense(rstd, (B, n_groups), _F32, dev, "rstd")
    ld_g = _like(grad_out, x, dev, "grad_out")
    gx, ld_gx = None, C
    if "x" in need:
        if out is None:
            gx = x.new_empty((rows, C))
        else:
            gx, ld_gx = out, _like(out, x, dev, "grad_x")
    gw = gb = None
    if "weight" in need or "bias" in need:
        both = torch.empty((2, C), dtype=_F32, device=x.device).unbind(0)
        gw, gb = (t if n in need else None for t, n in zip(both, ("weight", "bias")))
    keep, ws, nbytes = _scratch(nbytes, workspace, x.device)
    st = lib().oeq_group_norm_bwd(code, rows, B, C, n_groups, _act(act), ptr.data_ptr(), x.data_ptr(), ld, w, b, mu,
                                  rs, grad_out.data_ptr(), ld_g, None if gx is None else gx.data_ptr(), ld_gx,
                                  None if gw is None else gw.data_ptr(), None if gb is None else gb.data_ptr(), ws,
                                  nbytes, _raw_stream(dev))
    if st:
        _check(st)
    return gx, gw, gb


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------

def oeq_dropout_fwd(x, p: float, rng, residual=None, out=None):
    """residual + dropout(x) for x [rows, columns], rows possibly strided; rng is an int64 device
    tensor (seed, offset) read when the call runs.  The mask depends on rng and (row, column)
    only (see oeq.h).  `out` may be x or residual itself."""
    code, dev = _head(x, "x")
    ld = _row_stride(x, "x")
    rows, cols = x.shape
    key = _dense(rng, (2,), _I64, dev, "rng")
    res, ld_r = None, 0
    if residual is not None:
        ld_r = _like(residual, x, dev, "residual")
        res = residual.data_ptr()
    if out is None:
        out, ld_o = x.new_empty((rows, cols)), cols
    else:
        ld_o = _like(out, x, dev, "out")
    st = lib().oeq_dropout_fwd(code, rows, cols, x.data_ptr(), ld, res, ld_r, p, key, out.data_ptr(), ld_o,
                               _raw_stream(dev))
    if st:
        _check(st)
    return out


def oeq_dropout_bwd(grad_out, p: float, rng, out=None):
    """Gradient to x of <grad_out, oeq_dropout_fwd(x, p, rng, ...)>."""
    code, dev = _head(grad_out, "grad_out")
    ld = _row_stride(grad_out, "grad_out")
    rows, cols = grad_out.shape
    key = _dense(rng, (2,), _I64, dev, "rng")
    if out is None:
        out, ld_o = grad_out.new_empty((rows, cols)), cols
    else:
        ld_o = _like(out, grad_out, dev, "grad_x")
    st = lib().oeq_dropout_bwd(code, rows, cols, grad_out.data_ptr(), ld, p, key, out.data_ptr(), ld_o,
                               _raw_stream(dev))
    if st:
        _check(st)
    return out


# ---------------------------------------------------------------------------
# cross attention
# ---------------------------------------------------------------------------

def _heads(t, shape, dtype, dev, name):
    """Row and head strides of a [rows, heads, dim] operand with contiguous heads."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev or t.dtype is not dtype:
        _typed(t, dtype, dev, name)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    row, head, last = t.stride()
    if last != 1 and shape[2] > 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    # the stride of a dimension of one is arbitrary: it is never stepped over
    return (row if shape[0] > 1 else 0), (head if shape[1] > 1 else 0)


def _number(v, name):
    """v as a float: what is remembered by value must not be an object that can change (a tensor)."""
    if type(v) is float:
        return v
    try:
        return v.__float__()
    except AttributeError:
        raise TypeError(f"{name} must be a number") from None


@functools.lru_cache(maxsize=4096)
def _attn_desc(*fields):
    """(descriptor, workspace bytes forward, backward), a function of sizes, strides and numbers."""
    d = _AttnDesc(*fields)
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().oeq_cross_attn_workspace_size(ctypes.byref(d), ctypes.byref(f), ctypes.byref(b)))
    return ctypes.byref(d), f.value, b.value


def oeq_cross_attn_workspace_size(q_shape, k_shape, n_struct: int, dtype=torch.float32):
    """Workspace bytes (forward, backward) for q of shape [Tq, H, D] and k, v of [Tk, Hkv, D]."""
    (tq, h, d), (tk, hk, _) = q_shape, k_shape
    return _attn_desc(_DTYPES[dtype], n_struct, h, hk, d, tq, tk, 0, 0, 0, 0, 0, 0, 1.0, 0.0)[1:]


def _attn(q, k, v, q_ptr, k_ptr, scale, key_mask, p_drop, rng):
    """(device, what _attn_desc gives, addresses of the operands both directions read)"""
    code, dev = _head(q, "q")
    if q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("q and k must be [rows, heads, dim]")
    dt, shape = q.dtype, q.shape
    tq, h, d = shape
    tk, hk, _ = k.shape
    kv = (tk, hk, d)
    B = _structures(q_ptr, dev, "q_ptr")
    if _structures(k_ptr, dev, "k_ptr") != B:
        raise ValueError("q_ptr and k_ptr must hold the same structures")
    mask = None
    if key_mask is not None:
        mask = _dense(key_mask, (tk,), torch.bool if key_mask.dtype is torch.bool else _U8, dev, "key_mask")
    desc = _attn_desc(code, B, h, hk, d, tq, tk, *_heads(q, shape, dt, dev, "q"), *_heads(k, kv, dt, dev, "k"),
                      *_heads(v, kv, dt, dev, "v"), d ** -0.5 if scale is None else _number(scale, "scale"),
                      _number(p_drop, "p_drop"))
    return dev, desc, (q_ptr.data_ptr(), k_ptr.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), mask,
                       _dense(rng, (2,), _I64, dev, "rng"))


def oeq_cross_attn_fwd(q, k, v, q_ptr, k_ptr, scale=None, key_mask=None, p_drop: float = 0.0, rng=None, out=None,
                       lse=None, workspace=None):
    """(out, lse): attention of q [Tq, H, D] to the states k, v [Tk, Hkv, D] of their structure
    (q_ptr, k_ptr: int32 row pointers over the same structures).  scale defaults to
    1 / sqrt(D); key_mask [Tk] (bool or uint8) is nonzero where a state is visible; rng (see
    oeq_dropout_fwd) is needed for p_drop > 0.  Rows and heads of q, k and v may be strided;
    out and lse (fp32 [Tq, H]) are contiguous."""
    dev, (desc, fwd_bytes, _), operands = _attn(q, k, v, q_ptr, k_ptr, scale, key_mask, p_drop, rng)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _dense(out, q.shape, q.dtype, dev, "out")
    if lse is None:
        lse = torch.empty(q.shape[:2], dtype=_F32, device=q.device)
    else:
        _dense(lse, q.shape[:2], _F32, dev, "lse")
    keep, ws, nbytes = _scratch(fwd_bytes, workspace, q.device)
    st = lib().oeq_cross_attn_fwd(desc, *operands, out.data_ptr(), lse.data_ptr(), ws,
                                  nbytes, _raw_stream(dev))
    if st:
        _check(st)
    return out, lse


def oeq_cross_attn_bwd(q, k, v, q_ptr, k_ptr, out, lse, grad_out, scale=None, key_mask=None, p_drop: float = 0.0,
                       rng=None, need=("q", "k", "v"), grads=None, workspace=None):
    """(grad_q, grad_k, grad_v) of <grad_out, out> from the forward's operands, out and lse;
    entries not in `need` are None.  `grads` may supply preallocated gradients (contiguous)."""
    dev, (desc, _, bwd_bytes), operands = _attn(q, k, v, q_ptr, k_ptr, scale, key_mask, p_drop, rng)
    saved = (_dense(out, q.shape, q.dtype, dev, "out"), _dense(lse, q.shape[:2], _F32, dev, "lse"),
             _dense(grad_out, q.shape, q.dtype, dev, "grad_out"))
    if grads is None:
        grads = tuple(torch.empty_like(t, memory_format=torch.contiguous_format) if n in need else None
                      for n, t in (("q", q), ("k", k), ("v", k)))
    addresses = tuple(_dense(g, t.shape, q.dtype, dev, n)
                      for g, t, n in zip(grads, (q, k, k), ("grad_q", "grad_k", "grad_v")))
    keep, ws, nbytes = _scratch(bwd_bytes, workspace, q.device)
    st = lib().oeq_cross_attn_bwd(desc, *operands, *saved, *addresses, ws, nbytes,
                                  _raw_stream(dev))
    if st:
        _check(st)
    return tuple(grads)
