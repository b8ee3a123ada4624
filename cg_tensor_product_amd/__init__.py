"""Python binding of liboeq.so, the MI355X library for the fused channel-wise
(UVU) Clebsch-Gordan tensor-product graph convolution.

Argument marshalling only: every step of the computation runs in the library's
HIP kernels.  PyTorch provides device memory and the current HIP stream.  The
binding allocates outputs (and the deterministic-mode workspace) with torch and
passes raw pointers; the library itself never allocates in a compute call.

Names follow the C ABI (include/oeq.h):
  Plan (oeq_plan_create / oeq_plan_dims / oeq_plan_paths / oeq_plan_destroy)
  oeq_tp_conv_fwd, oeq_tp_conv_bwd, oeq_tp_conv_dbwd, oeq_workspace_size,
  oeq_cg_table, oeq_sender_csr, oeq_csr_check.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liboeq.so")

OEQ_F32, OEQ_F64, OEQ_F16, OEQ_BF16 = 0, 1, 2, 3
ACTS = {"none": 0, "silu": 1}
OEQ_BWD_ATOMIC, OEQ_BWD_DETERMINISTIC = 0, 1
_MODES = {"atomic": OEQ_BWD_ATOMIC, "deterministic": OEQ_BWD_DETERMINISTIC}
STATUS = {0: "OEQ_OK", 1: "OEQ_ERR_INVALID_ARG", 2: "OEQ_ERR_UNSUPPORTED", 3: "OEQ_ERR_WORKSPACE",
          4: "OEQ_ERR_HIP", 5: "OEQ_ERR_JIT"}

EXPORTED = ["oeq_plan_create", "oeq_plan_create_cached", "oeq_plan_destroy", "oeq_plan_dims", "oeq_plan_paths", "oeq_plan_code_key",
            "oeq_cg_table",
            "oeq_workspace_size", "oeq_tp_conv_fwd", "oeq_tp_conv_bwd", "oeq_tp_conv_bwd_noalloc", "oeq_tp_conv_dbwd",
            "oeq_csr_workspace_size", "oeq_sender_csr", "oeq_csr_check", "oeq_status_string",
            "oeq_last_error", "oeq_plan_schedule", "oeq_sender_view", "oeq_tp_conv_fwd_sender",
            "oeq_tp_conv_bwd_sender", "oeq_sph_harm", "oeq_sph_harm_bwd", "oeq_tp_conv_fwd_vec",
            "oeq_workspace_size_vec", "oeq_tp_conv_bwd_vec", "oeq_radial_workspace_size", "oeq_radial_fwd",
            "oeq_radial_bwd", "oeq_tp_conv_fwd_radial", "oeq_workspace_size_radial", "oeq_tp_conv_bwd_radial",
            "oeq_tp_conv_fwd_pos", "oeq_workspace_size_pos", "oeq_tp_conv_bwd_pos",
            "oeq_group_norm_workspace_size", "oeq_group_norm_fwd", "oeq_group_norm_bwd", "oeq_dropout_fwd",
            "oeq_dropout_bwd", "oeq_cross_attn_workspace_size", "oeq_cross_attn_fwd", "oeq_cross_attn_bwd"]
SCHEDULES = {0: "receiver", 1: "sender"}


class OeqError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class _Irrep(ctypes.Structure):
    _fields_ = [("mul", ctypes.c_int32), ("l", ctypes.c_int32), ("parity", ctypes.c_int32)]


class _Path(ctypes.Structure):
    _fields_ = [("in1", ctypes.c_int32), ("in2", ctypes.c_int32), ("out", ctypes.c_int32)]


class _Desc(ctypes.Structure):
    _fields_ = [("x_irreps", ctypes.POINTER(_Irrep)), ("n_x", ctypes.c_int32),
                ("y_irreps", ctypes.POINTER(_Irrep)), ("n_y", ctypes.c_int32),
                ("y_lmax", ctypes.c_int32), ("out_irreps", ctypes.POINTER(_Irrep)),
                ("n_out", ctypes.c_int32), ("paths", ctypes.POINTER(_Path)),
                ("n_paths", ctypes.c_int32), ("lmax_out", ctypes.c_int32), ("dtype", ctypes.c_int)]


class _AttnDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("n_struct", ctypes.c_int32), ("n_heads", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("q_rows", ctypes.c_int64),
                ("k_rows", ctypes.c_int64), ("q_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("k_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("v_head_stride", ctypes.c_int64), ("scale", ctypes.c_double), ("p_drop", ctypes.c_double)]


_lib = None


def lib():
    """The loaded liboeq.so.  Raises if the library has not been built: there is
    no fallback implementation."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    st = ctypes.c_int
    L.oeq_plan_create.argtypes = [ctypes.POINTER(_Desc), ctypes.POINTER(P)]
    L.oeq_plan_create.restype = st
    L.oeq_plan_create_cached.argtypes = [ctypes.POINTER(_Desc), ctypes.POINTER(P)]
    L.oeq_plan_create_cached.restype = st
    L.oeq_plan_destroy.argtypes = [P]
    L.oeq_plan_destroy.restype = None
    L.oeq_plan_dims.argtypes = [P] + [ctypes.POINTER(I64)] * 5
    L.oeq_plan_dims.restype = st
    L.oeq_plan_paths.argtypes = [P, P, I32]
    L.oeq_plan_paths.restype = st
    L.oeq_plan_code_key.argtypes = [P, ctypes.c_char_p, SZ]
    L.oeq_plan_code_key.restype = st
    L.oeq_cg_table.argtypes = [I32, I32, I32, P]
    L.oeq_cg_table.restype = st
    L.oeq_workspace_size.argtypes = [P, I64, I64, ctypes.c_int, ctypes.POINTER(SZ)]
    L.oeq_workspace_size.restype = st
    L.oeq_tp_conv_fwd.argtypes = [P, I64, I64, P, P, P, P, P, P, P]
    L.oeq_tp_conv_fwd.restype = st
    L.oeq_tp_conv_bwd.argtypes = [P, I64, I64, P, P, P, P, P, P, P, P, P, ctypes.c_int, P, SZ, P]
    L.oeq_tp_conv_bwd.restype = st
    L.oeq_tp_conv_bwd_noalloc.argtypes = [P, I64, I64, P, P, P, P, P, P, P, P, P, ctypes.c_int, P]
    L.oeq_tp_conv_bwd_noalloc.restype = st
    L.oeq_tp_conv_dbwd.argtypes = [P, I64, I64, P, P, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_int, P, SZ, P]
    L.oeq_tp_conv_dbwd.restype = st
    L.oeq_csr_workspace_size.argtypes = [I64, I64, ctypes.POINTER(SZ)]
    L.oeq_csr_workspace_size.restype = st
    L.oeq_sender_csr.argtypes = [I64, I64, P, P, P, P, SZ, P]
    L.oeq_sender_csr.restype = st
    L.oeq_csr_check.argtypes = [I64, I64, P, P, P]
    L.oeq_csr_check.restype = st
    L.oeq_plan_schedule.argtypes = [P, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
                                     ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]
    L.oeq_plan_schedule.restype = st
    L.oeq_sender_view.argtypes = [I64, I64, P, P, P, P, P, P, SZ, P]
    L.oeq_sender_view.restype = st
    L.oeq_tp_conv_fwd_sender.argtypes = [P, I64, I64, P, P, P, P, P, P, P, P]
    L.oeq_tp_conv_fwd_sender.restype = st
    L.oeq_tp_conv_bwd_sender.argtypes = [P, I64, I64, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
    L.oeq_tp_conv_bwd_sender.restype = st
    L.oeq_sph_harm.argtypes = [P, I64, P, P, P]
    L.oeq_sph_harm.restype = st
    L.oeq_sph_harm_bwd.argtypes = [P, I64, P, P, P, P]
    L.oeq_sph_harm_bwd.restype = st
    L.oeq_tp_conv_fwd_vec.argtypes = [P, I64, I64, P, P, P, P, P, P, P]
    L.oeq_tp_conv_fwd_vec.restype = st
    L.oeq_workspace_size_vec.argtypes = [P, I64, I64, ctypes.c_int, ctypes.POINTER(SZ)]
    L.oeq_workspace_size_vec.restype = st
    L.oeq_tp_conv_bwd_vec.argtypes = [P, I64, I64, P, P, P, P, P, P, P, P, P, ctypes.c_int, P, SZ, P]
    L.oeq_tp_conv_bwd_vec.restype = st
    L.oeq_tp_conv_fwd_pos.argtypes = [P, I64, I64, P, P, P, P, P, P, P]
    L.oeq_tp_conv_fwd_pos.restype = st
    L.oeq_workspace_size_pos.argtypes = [P, I64, I64, ctypes.c_int, ctypes.POINTER(SZ)]
    L.oeq_workspace_size_pos.restype = st
    L.oeq_tp_conv_bwd_pos.argtypes = [P, I64, I64, P, P, P, P, P, P, P, P, P, ctypes.c_int, P, SZ, P]
    L.oeq_tp_conv_bwd_pos.restype = st
    D = ctypes.c_double
    L.oeq_radial_workspace_size.argtypes = [P, I64, I32, ctypes.POINTER(SZ)]
    L.oeq_radial_workspace_size.restype = st
    L.oeq_radial_fwd.argtypes = [P, I64, P, D, I32, P, P, P, P, SZ, P]
    L.oeq_radial_fwd.restype = st
    L.oeq_radial_bwd.argtypes = [P, I64, P, D, I32, P, P, P, P, P, P, P, SZ, P]
    L.oeq_radial_bwd.restype = st
    L.oeq_tp_conv_fwd_radial.argtypes = [P, I64, I64, P, P, P, P, P, D, P, P, P, P, SZ, P]
    L.oeq_tp_conv_fwd_radial.restype = st
    L.oeq_workspace_size_radial.argtypes = [P, I64, I64, ctypes.c_int, ctypes.POINTER(SZ)]
    L.oeq_workspace_size_radial.restype = st
    L.oeq_tp_conv_bwd_radial.argtypes = [P, I64, I64, P, P, P, P, P, D, P, P, P, P, P, P, P, P, ctypes.c_int, P, SZ,
                                         P]
    L.oeq_tp_conv_bwd_radial.restype = st
    I = ctypes.c_int
    SZP = ctypes.POINTER(SZ)
    L.oeq_group_norm_workspace_size.argtypes = [I64, I32, I32, I32, SZP, SZP]
    L.oeq_group_norm_workspace_size.restype = st
    L.oeq_group_norm_fwd.argtypes = [I, I64, I32, I32, I32, I, D, P, P, I64, P, P, P, I64, P, P, P, SZ, P]
    L.oeq_group_norm_fwd.restype = st
    L.oeq_group_norm_bwd.argtypes = [I, I64, I32, I32, I32, I, P, P, I64, P, P, P, P, P, I64, P, I64, P, P, P, SZ, P]
    L.oeq_group_norm_bwd.restype = st
    L.oeq_dropout_fwd.argtypes = [I, I64, I64, P, I64, P, I64, D, P, P, I64, P]
    L.oeq_dropout_fwd.restype = st
    L.oeq_dropout_bwd.argtypes = [I, I64, I64, P, I64, D, P, P, I64, P]
    L.oeq_dropout_bwd.restype = st
    AD = ctypes.POINTER(_AttnDesc)
    L.oeq_cross_attn_workspace_size.argtypes = [AD, SZP, SZP]
    L.oeq_cross_attn_workspace_size.restype = st
    L.oeq_cross_attn_fwd.argtypes = [AD] + [P] * 10 + [SZ, P]
    L.oeq_cross_attn_fwd.restype = st
    L.oeq_cross_attn_bwd.argtypes = [AD] + [P] * 14 + [SZ, P]
    L.oeq_cross_attn_bwd.restype = st
    L.oeq_status_string.argtypes = [ctypes.c_int]
    L.oeq_status_string.restype = ctypes.c_char_p
    L.oeq_last_error.argtypes = []
    L.oeq_last_error.restype = ctypes.c_char_p
    _lib = L
    return L


def _check(status: int):
    if status != 0:
        raise OeqError(status, lib().oeq_last_error().decode())


def _irreps(seq) -> tuple:
    if isinstance(seq, str):
        out = []
        for part in seq.split("+"):
            mul, rest = part.strip().split("x")
            out.append((int(mul), int(rest[:-1]), 1 if rest[-1] == "e" else -1))
        return tuple(out)
    return tuple(tuple(int(v) for v in t) for t in seq)


class Plan:
    """oeq_plan_create for an irreps descriptor.  dtype: "f32" or "f64".

    x and output blocks have U channels (the largest x multiplicity) or one: a
    one-channel x block is broadcast against the U channels, a one-channel output
    block (out_irreps) receives their sum.

    Y: y_irreps (one-channel irreps in row order, e.g. "1x0e+1x2e+1x1e"), or by
    default the spherical harmonics of degrees 0..y_lmax.  paths=None enumerates
    every triangle-allowed path up to lmax_out; an explicit list holds
    (x block, Y block, output block) triples and needs out_irreps (with the default
    Y the Y block index is the degree)."""

    def __init__(self, x_irreps, y_lmax: int, lmax_out: int = 3, dtype: str = "f32",
                 paths: Optional[Sequence] = None, out_irreps=None, y_irreps=None):
        self.x_irreps = _irreps(x_irreps)
        self.y_irreps = None if y_irreps is None else _irreps(y_irreps)
        self.y_lmax = int(y_lmax)
        self.lmax_out = int(lmax_out)
        self.dtype = dtype
        xs = (_Irrep * len(self.x_irreps))(*[_Irrep(*t) for t in self.x_irreps])
        d = _Desc()
        d.x_irreps = xs
        d.n_x = len(self.x_irreps)
        d.y_lmax = self.y_lmax
        d.lmax_out = self.lmax_out
        d.dtype = OEQ_F64 if dtype == "f64" else OEQ_F32
        if dtype not in ("f32", "f64"):
            d.dtype = 7  # rejected by the library
        keep = [xs]
        if self.y_irreps is not None:
            ys = (_Irrep * len(self.y_irreps))(*[_Irrep(*t) for t in self.y_irreps])
            d.y_irreps, d.n_y = ys, len(self.y_irreps)
            keep.append(ys)
        if out_irreps is not None:
            oi = _irreps(out_irreps)
            os_ = (_Irrep * len(oi))(*[_Irrep(*t) for t in oi])
            d.out_irreps, d.n_out = os_, len(oi)
            keep.append(os_)
        if paths is not None:
            ps = (_Path * len(paths))(*[_Path(*t) for t in paths])
            d.paths, d.n_paths = ps, len(paths)
            keep.append(ps)
        h = ctypes.c_void_p()
        # the library compiles a plan missing from its code-object cache in its compiler
        # helper (a child process), so the kernels do not depend on what this process loaded
        st = lib().oeq_plan_create(ctypes.byref(d), ctypes.byref(h))
        _check(st)
        self._h = h
        dims = [ctypes.c_int64() for _ in range(5)]
        _check(lib().oeq_plan_dims(h, *[ctypes.byref(v) for v in dims]))
        self.x_dim, self.y_dim, self.out_dim, self.n_paths, self.w_per_edge = (int(v.value) for v in dims)
        self.U = self.w_per_edge // self.n_paths  # channels: the largest x multiplicity

    @property
    def handle(self):
        return self._h

    def paths(self):
        """[(x block, l1, l2, l3, output block, output parity), ...]"""
        buf = np.zeros(6 * self.n_paths, dtype=np.int32)
        _check(lib().oeq_plan_paths(self._h, buf.ctypes.data, self.n_paths))
        return [tuple(int(v) for v in buf[6 * k:6 * k + 6]) for k in range(self.n_paths)]

    @property
    def code_key(self) -> str:
        """Hash identifying the compiled kernels of this plan."""
        buf = ctypes.create_string_buffer(64)
        _check(lib().oeq_plan_code_key(self._h, buf, 64))
        return buf.value.decode()

    def schedule(self):
        """oeq_plan_schedule: {"fwd": "receiver"|"sender", "bwd": ..., "move_fwd": [r, s],
        "move_bwd": [r, s]} (the data-movement model's per-edge, per-channel elements)."""
        f, b = ctypes.c_int(), ctypes.c_int()
        mf, mb = (ctypes.c_double * 2)(), (ctypes.c_double * 2)()
        _check(lib().oeq_plan_schedule(self._h, ctypes.byref(f), ctypes.byref(b), mf, mb))
        return {"fwd": SCHEDULES[f.value], "bwd": SCHEDULES[b.value], "move_fwd": list(mf), "move_bwd": list(mb)}

    def torch_dtype(self):
        import torch
        return torch.float64 if self.dtype == "f64" else torch.float32

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _lib is not None:
            _lib.oeq_plan_destroy(h)
            self._h = None


def oeq_cg_table(l1: int, l2: int, l3: int) -> np.ndarray:
    out = np.zeros((2 * l1 + 1) * (2 * l2 + 1) * (2 * l3 + 1))
    _check(lib().oeq_cg_table(l1, l2, l3, out.ctypes.data))
    return out.reshape(2 * l1 + 1, 2 * l2 + 1, 2 * l3 + 1)


def oeq_workspace_size(plan: Plan, n_nodes: int, n_edges: int, mode: str = "atomic") -> int:
    b = ctypes.c_size_t()
    _check(lib().oeq_workspace_size(plan.handle, n_nodes, n_edges, _MODES[mode], ctypes.byref(b)))
    return int(b.value)


# ---------------------------------------------------------------------------
# tensor helpers
# ---------------------------------------------------------------------------

def _stream():
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _want(t, shape, dtype, name):
    import torch
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _graph(rowptr, src):
    import torch
    N = rowptr.shape[0] - 1
    E = src.shape[0]
    _want(rowptr, (N + 1,), torch.int32, "rowptr")
    _want(src, (E,), torch.int32, "src")
    return N, E


def _empty(shape, dtype, device):
    import torch
    return torch.empty(shape, dtype=dtype, device=device)


def _workspace(plan, N, E, mode, device):
    import torch
    nbytes = oeq_workspace_size(plan, N, E, mode)
    if nbytes == 0:
        return None, 0
    ws = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + nbytes], nbytes


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def oeq_tp_conv_fwd(plan: Plan, rowptr, src, x, Y, W, out=None):
    """out[N, out_dim] = f(x, Y, W) (receiver-stationary forward)."""
    N, E = _graph(rowptr, src)
    dt = plan.torch_dtype()
    _want(x, (N, plan.x_dim), dt, "x")
    _want(Y, (E, plan.y_dim), dt, "Y")
    _want(W, (E, plan.n_paths, plan.U), dt, "W")
    if out is None:
        out = _empty((N, plan.out_dim), dt, rowptr.device)
    _want(out, (N, plan.out_dim), dt, "out")
    _check(lib().oeq_tp_conv_fwd(plan.handle, N, E, _ptr(rowptr), _ptr(src), _ptr(x), _ptr(Y), _ptr(W),
                                 _ptr(out), _stream()))
    return out


def oeq_tp_conv_bwd(plan: Plan, rowptr, src, x, Y, W, grad_out, mode: str = "atomic",
                    need=("x", "Y", "W"), out=None, workspace=None):
    """(grad_x, grad_Y, grad_W) of <grad_out, f(x, Y, W)>; entries not in `need`
    are None.  `out` may supply preallocated (grad_x, grad_Y, grad_W)."""
    N, E = _graph(rowptr, src)
    dt = plan.torch_dtype()
    _want(x, (N, plan.x_dim), dt, "x")
    _want(Y, (E, plan.y_dim), dt, "Y")
    _want(W, (E, plan.n_paths, plan.U), dt, "W")
    _want(grad_out, (N, plan.out_dim), dt, "grad_out")
    dev = rowptr.device
    shapes = ((N, plan.x_dim), (E, plan.y_dim), (E, plan.n_paths, plan.U))
    if out is None:
        out = tuple(_empty(s, dt, dev) if k in need else None for k, s in zip(("x", "Y", "W"), shapes))
    gx, gY, gW = (_want(t, s, dt, n) for t, s, n in zip(out, shapes, ("grad_x", "grad_Y", "grad_W")))
    ws, nbytes = (workspace, workspace.numel()) if workspace is not None else _workspace(plan, N, E, mode, dev)
    _check(lib().oeq_tp_conv_bwd(plan.handle, N, E, _ptr(rowptr), _ptr(src), _ptr(x), _ptr(Y), _ptr(W),
                                 _ptr(grad_out), _ptr(gx), _ptr(gY), _ptr(gW), _MODES[mode], _ptr(ws), nbytes,
                                 _stream()))
    return gx, gY, gW


def oeq_tp_conv_bwd_noalloc(plan: Plan, rowptr, src, x, Y, W, grad_out, out, mode: str = "atomic"):
    """oeq_tp_conv_bwd into preallocated (grad_x, grad_Y, grad_W) (None: not computed),
    with the library's fixed device scratch in place of a workspace."""
    N, E = _graph(rowptr, src)
    dt = plan.torch_dtype()
    _want(x, (N, plan.x_dim), dt, "x")
    _want(Y, (E, plan.y_dim), dt, "Y")
    _want(W, (E, plan.n_paths, plan.U), dt, "W")
    _want(grad_out, (N, plan.out_dim), dt, "grad_out")
    shapes = ((N, plan.x_dim), (E, plan.y_dim), (E, plan.n_paths, plan.U))
    gx, gY, gW = (_want(t, s, dt, n) for t, s, n in zip(out, shapes, ("grad_x", "grad_Y", "grad_W")))
    _check(lib().oeq_tp_conv_bwd_noalloc(plan.handle, N, E, _ptr(rowptr), _ptr(src), _ptr(x), _ptr(Y), _ptr(W),
                                         _ptr(grad_out), _ptr(gx), _ptr(gY), _ptr(gW), _MODES[mode], _stream()))
    return gx, gY, gW


def oeq_tp_conv_dbwd(plan: Plan, rowptr, src, x, Y, W, grad_out, gg_x=None, gg_Y=None, gg_W=None,
                     mode: str = "atomic", want=("x", "Y", "W", "grad_out"), workspace=None, out=None):
    """Double backward: dict with d_x, d_Y, d_W, d_grad_out (None if not in want).
    out: optional dict of preallocated outputs with the same keys (a missing or None
    entry is not requested); it overrides want."""
    N, E = _graph(rowptr, src)
    dt = plan.torch_dtype()
    _want(x, (N, plan.x_dim), dt, "x")
    _want(Y, (E, plan.y_dim), dt, "Y")
    _want(W, (E, plan.n_paths, plan.U), dt, "W")
    _want(grad_out, (N, plan.out_dim), dt, "grad_out")
    _want(gg_x, (N, plan.x_dim), dt, "gg_x")
    _want(gg_Y, (E, plan.y_dim), dt, "gg_Y")
    _want(gg_W, (E, plan.n_paths, plan.U), dt, "gg_W")
    dev = rowptr.device
    shapes = {"x": (N, plan.x_dim), "Y": (E, plan.y_dim), "W": (E, plan.n_paths, plan.U),
              "grad_out": (N, plan.out_dim)}
    if out is not None:
        d = {k: out.get(k) for k in shapes}
        for k, t in d.items():
            _want(t, shapes[k], dt, "d_" + k)
    else:
        d = {k: _empty(shp, dt, dev) if k in want else None for k, shp in shapes.items()}
    ws, nbytes = (workspace, workspace.numel()) if workspace is not None else _workspace(plan, N, E, mode, dev)
    _check(lib().oeq_tp_conv_dbwd(plan.handle, N, E, _ptr(rowptr), _ptr(src), _ptr(x), _ptr(Y), _ptr(W),
                                  _ptr(grad_out), _ptr(gg_x), _ptr(gg_Y), _ptr(gg_W), _ptr(d["x"]), _ptr(d["Y"]),
                                  _ptr(d["W"]), _ptr(d["grad_out"]), _MODES[mode], _ptr(ws), nbytes, _stream()))
    return d


def oeq_sender_csr(src, n_nodes: int):
    """Device sender CSR: (srowptr[N+1], sperm[E]) int32."""
    import torch
    E = src.shape[0]
    _want(src, (E,), torch.int32, "src")
    b = ctypes.c_size_t()
    _check(lib().oeq_csr_workspace_size(n_nodes, E, ctypes.byref(b)))
    ws = torch.empty(int(b.value) + 256, dtype=torch.uint8, device=src.device)
    off = (-ws.data_ptr()) % 256
    ws = ws[off:off + int(b.value)]
    srowptr = torch.empty(n_nodes + 1, dtype=torch.int32, device=src.device)
    sperm = torch.empty(E, dtype=torch.int32, device=src.device)
    _check(lib().oeq_sender_csr(n_nodes, E, _ptr(src), _ptr(srowptr), _ptr(sperm), _ptr(ws), int(b.value),
                                _stream()))
    return srowptr, sperm


def oeq_csr_check(rowptr, src) -> None:
    N, E = _graph(rowptr, src)
    _check(lib().oeq_csr_check(N, E, _ptr(rowptr), _ptr(src), _stream()))


def oeq_sender_view(rowptr, src):
    """Device sender view (srowptr[N+1], sperm[E], sdst[E]) int32 of a receiver CSR."""
    import torch
    N, E = _graph(rowptr, src)
    dev = src.device
    srowptr = torch.empty(N + 1, dtype=torch.int32, device=dev)
    sperm = torch.empty(max(E, 1), dtype=torch.int32, device=dev)[:E]
    sdst = torch.empty(max(E, 1), dtype=torch.int32, device=dev)[:E]
    nbytes = ctypes.c_size_t()
    _check(lib().oeq_csr_workspace_size(N, E, ctypes.byref(nbytes)))
    raw = torch.empty(nbytes.value + 256, dtype=torch.uint8, device=dev)
    off = (-raw.data_ptr()) % 256
    ws = raw[off:off + nbytes.value]
    _check(lib().oeq_sender_view(N, E, _ptr(rowptr), _ptr(src), _ptr(srowptr), _ptr(sperm), _ptr(sdst), _ptr(ws),
                                 nbytes.value, _stream()))
    return srowptr, sperm, sdst


def oeq_tp_conv_fwd_sender(plan: Plan, view, x, Y, W, out=None):
    """Sender-stationary forward; view = oeq_sender_view(rowptr, src)."""
    srowptr, sperm, sdst = view
    N, E = srowptr.shape[0] - 1, sperm.shape[0]
    dt = plan.torch_dtype()
    _want(x, (N, plan.x_dim), dt, "x")
    _want(Y, (E, plan.y_dim), dt, "Y")
    _want(W, (E, plan.n_paths, plan.U), dt, "W")
    if out is None:
        out = _empty((N, plan.out_dim), dt, x.device)
    _want(out, (N, plan.out_dim), dt, "out")
    _check(lib().oeq_tp_conv_fwd_sender(plan.handle, N, E, _ptr(srowptr), _ptr(sperm), _ptr(sdst), _ptr(x), _ptr(Y),
                                        _ptr(W), _ptr(out), _stream()))
    return out


def oeq_tp_conv_bwd_sender(plan: Plan, view, x, Y, W, grad_out, want=("x", "Y", "W"), out=None, workspace=None):
    """Sender-stationary VJP: (grad_x, grad_Y, grad_W), None where not in want."""
    srowptr, sperm, sdst = view
    N, E = srowptr.shape[0] - 1, sperm.shape[0]
    dt = plan.torch_dtype()
    _want(x, (N, plan.x_dim), dt, "x")
    _want(Y, (E, plan.y_dim), dt, "Y")
    _want(W, (E, plan.n_paths, plan.U), dt, "W")
    _want(grad_out, (N, plan.out_dim), dt, "grad_out")
    shapes = ((N, plan.x_dim), (E, plan.y_dim), (E, plan.n_paths, plan.U))
    if out is None:
        out = tuple(_empty(shp, dt, x.device) if k in want else None for k, shp in zip(("x", "Y", "W"), shapes))
    for t, shp, k in zip(out, shapes, ("grad_x", "grad_Y", "grad_W")):
        _want(t, shp, dt, k)
    ws, nbytes = (workspace, workspace.numel()) if workspace is not None else _workspace(plan, N, E, "atomic",
                                                                                        x.device)
    _check(lib().oeq_tp_conv_bwd_sender(plan.handle, N, E, _ptr(srowptr), _ptr(sperm), _ptr(sdst), _ptr(x), _ptr(Y),
                                        _ptr(W), _ptr(grad_out), _ptr(out[0]), _ptr(out[1]), _ptr(out[2]), _ptr(ws),
                                        nbytes, _stream()))
    return out


def oeq_sph_harm(plan: Plan, vec, out=None):
    """Y[E, (L+1)^2] of edge vectors vec[E, 3]."""
    E = vec.shape[0]
    dt = plan.torch_dtype()
    _want(vec, (E, 3), dt, "vec")
    if out is None:
        out = _empty((E, plan.y_dim), dt, vec.device)
    _want(out, (E, plan.y_dim), dt, "Y")
    _check(lib().oeq_sph_harm(plan.handle, E, _ptr(vec), _ptr(out), _stream()))
    return out


def oeq_sph_harm_bwd(plan: Plan, vec, grad_Y, out=None):
    """grad_vec[E, 3] = sum_m grad_Y[e, m] dY[e, m] / dvec[e]."""
    E = vec.shape[0]
    dt = plan.torch_dtype()
    _want(vec, (E, 3), dt, "vec")
    _want(grad_Y, (E, plan.y_dim), dt, "grad_Y")
    if out is None:
        out = _empty((E, 3), dt, vec.device)
    _want(out, (E, 3), dt, "grad_vec")
    _check(lib().oeq_sph_harm_bwd(plan.handle, E, _ptr(vec), _ptr(grad_Y), _ptr(out), _stream()))
    return out


def oeq_tp_conv_fwd_vec(plan: Plan, rowptr, src, x, vec, W, out=None):
    """Forward with Y evaluated in the kernel from the edge vectors."""
    N, E = _graph(rowptr, src)
    dt = plan.torch_dtype()
    _want(x, (N, plan.x_dim), dt, "x")
    _want(vec, (E, 3), dt, "vec")
    _want(W, (E, plan.n_paths, plan.U), dt, "W")
    if out is None:
        out = _empty((N, plan.out_dim), dt, rowptr.device)
    _want(out, (N, plan.out_dim), dt, "out")
    _check(lib().oeq_tp_conv_fwd_vec(plan.handle, N, E, _ptr(rowptr), _ptr(src), _ptr(x), _ptr(vec), _ptr(W),
                                     _ptr(out), _stream()))
    return out


def oeq_workspace_size_vec(plan: Plan, n_nodes: int, n_edges: int, mode: str = "atomic") -> int:
    b = ctypes.c_size_t()
    _check(lib().oeq_workspace_size_vec(plan.handle, n_nodes, n_edges, _MODES[mode], ctypes.byref(b)))
    return b.value


def oeq_tp_conv_bwd_vec(plan: Plan, rowptr, src, x, vec, W, grad_out, mode: str = "atomic",
                        want=("x", "vec", "W"), out=None, workspace=None):
    """VJP to (x, vec, W) of the forward from edge vectors."""
    import torch
    N, E = _graph(rowptr, src)
    dt = plan.torch_dtype()
    _want(x, (N, plan.x_dim), dt, "x")
    _want(vec, (E, 3), dt, "vec")
    _want(W, (E, plan.n_paths, plan.U), dt, "W")
    _want(grad_out, (N, plan.out_dim), dt, "grad_out")
    shapes = ((N, plan.x_dim), (E, 3), (E, plan.n_paths, plan.U))
    if out is None:
        out = tuple(_empty(shp, dt, x.device) if k in want else None for k, shp in zip(("x", "vec", "W"), shapes))
    for t, shp, k in zip(out, shapes, ("grad_x", "grad_vec", "grad_W")):
        _want(t, shp, dt, k)
    if workspace is None:
        nbytes = oeq_workspace_size_vec(plan, N, E, mode)
        raw = torch.empty(nbytes + 256, dtype=torch.uint8, device=x.device)
        workspace = raw[(-raw.data_ptr()) % 256:][:nbytes]
    _check(lib().oeq_tp_conv_bwd_vec(plan.handle, N, E, _ptr(rowptr), _ptr(src), _ptr(x), _ptr(vec), _ptr(W),
                                     _ptr(grad_out), _ptr(out[0]), _ptr(out[1]), _ptr(out[2]), _MODES[mode],
                                     _ptr(workspace), workspace.numel(), _stream()))
    return out


def oeq_tp_conv_fwd_pos(plan: Plan, rowptr, src, x, pos, W, out=None):
    """Forward with Y evaluated in the kernel from atom positions pos[N, 3]
    (vec[e] = pos[src[e]] - pos[receiver])."""
    N, E = _graph(rowptr, src)
    dt = plan.torch_dtype()
    _want(x, (N, plan.x_dim), dt, "x")
    _want(pos, (N, 3), dt, "pos")
    _want(W, (E, plan.n_paths, plan.U), dt, "W")
    if out is None:
        out = _empty((N, plan.out_dim), dt, rowptr.device)
    _want(out, (N, plan.out_dim), dt, "out")
    _check(lib().oeq_tp_conv_fwd_pos(plan.handle, N, E, _ptr(rowptr), _ptr(src), _ptr(x), _ptr(pos), _ptr(W),
                                     _ptr(out), _stream()))
    return out


def oeq_workspace_size_pos(plan: Plan, n_nodes: int, n_edges: int, mode: str = "atomic") -> int:
    b = ctypes.c_size_t()
    _check(lib().oeq_workspace_size_pos(plan.handle, n_nodes, n_edges, _MODES[mode], ctypes.byref(b)))
    return b.value


def oeq_tp_conv_bwd_pos(plan: Plan, rowptr, src, x, pos, W, grad_out, mode: str = "atomic",
                        want=("x", "pos", "W"), out=None, workspace=None):
    """VJP to (x, pos, W) of the forward from atom positions."""
    import torch
    N, E = _graph(rowptr, src)
    dt = plan.torch_dtype()
    _want(x, (N, plan.x_dim), dt, "x")
    _want(pos, (N, 3), dt, "pos")
    _want(W, (E, plan.n_paths, plan.U), dt, "W")
    _want(grad_out, (N, plan.out_dim), dt, "grad_out")
    shapes = ((N, plan.x_dim), (N, 3), (E, plan.n_paths, plan.U))
    if out is None:
        out = tuple(_empty(shp, dt, x.device) if k in want else None for k, shp in zip(("x", "pos", "W"), shapes))
    for t, shp, k in zip(out, shapes, ("grad_x", "grad_pos", "grad_W")):
        _want(t, shp, dt, k)
    if workspace is None:
        nbytes = oeq_workspace_size_pos(plan, N, E, mode)
        raw = torch.empty(nbytes + 256, dtype=torch.uint8, device=x.device)
        workspace = raw[(-raw.data_ptr()) % 256:][:nbytes]
    _check(lib().oeq_tp_conv_bwd_pos(plan.handle, N, E, _ptr(rowptr), _ptr(src), _ptr(x), _ptr(pos), _ptr(W),
                                     _ptr(grad_out), _ptr(out[0]), _ptr(out[1]), _ptr(out[2]), _MODES[mode],
                                     _ptr(workspace), workspace.numel(), _stream()))
    return out


def _radial_ws(plan, E, hidden, device):
    import torch
    b = ctypes.c_size_t()
    _check(lib().oeq_radial_workspace_size(plan.handle, E, hidden, ctypes.byref(b)))
    raw = torch.empty(b.value + 256, dtype=torch.uint8, device=device)
    return raw[(-raw.data_ptr()) % 256:][:b.value]


def oeq_radial_fwd(plan: Plan, vec, r_cut: float, W1, W2, out=None, workspace=None):
    """Radial weights W [E, P, U] from edge vectors (see oeq.h for the form)."""
    E = vec.shape[0]
    dt = plan.torch_dtype()
    H = W1.shape[1]
    _want(vec, (E, 3), dt, "vec")
    _want(W1, (8, H), dt, "W1")
    _want(W2, (H, plan.n_paths * plan.U), dt, "W2")
    if out is None:
        out = _empty((E, plan.n_paths, plan.U), dt, vec.device)
    _want(out, (E, plan.n_paths, plan.U), dt, "W")
    ws = workspace if workspace is not None else _radial_ws(plan, E, H, vec.device)
    _check(lib().oeq_radial_fwd(plan.handle, E, _ptr(vec), float(r_cut), H, _ptr(W1), _ptr(W2), _ptr(out), _ptr(ws),
                                ws.numel(), _stream()))
    return out


def oeq_radial_bwd(plan: Plan, vec, r_cut: float, W1, W2, grad_W, want=("vec", "W1", "W2"), workspace=None):
    """(grad_vec, grad_W1, grad_W2) of <grad_W, W(vec, W1, W2)>; None where not in want."""
    E = vec.shape[0]
    dt = plan.torch_dtype()
    H = W1.shape[1]
    _want(vec, (E, 3), dt, "vec")
    _want(W1, (8, H), dt, "W1")
    _want(W2, (H, plan.n_paths * plan.U), dt, "W2")
    _want(grad_W, (E, plan.n_paths, plan.U), dt, "grad_W")
    gv = _empty((E, 3), dt, vec.device) if "vec" in want else None
    g1 = _empty((8, H), dt, vec.device) if "W1" in want else None
    g2 = _empty((H, plan.n_paths * plan.U), dt, vec.device) if "W2" in want else None
    ws = workspace if workspace is not None else _radial_ws(plan, E, H, vec.device)
    _check(lib().oeq_radial_bwd(plan.handle, E, _ptr(vec), float(r_cut), H, _ptr(W1), _ptr(W2), _ptr(grad_W),
                                _ptr(gv), _ptr(g1), _ptr(g2), _ptr(ws), ws.numel(), _stream()))
    return gv, g1, g2


def oeq_tp_conv_fwd_radial(plan: Plan, rowptr, src, x, Y, vec, r_cut: float, W1, W2, out=None, workspace=None):
    """Forward with W formed in the kernel from a hidden width of 8 (W1 [8, 8], W2 [8, P*U])."""
    N, E = _graph(rowptr, src)
    dt = plan.torch_dtype()
    _want(x, (N, plan.x_dim), dt, "x")
    _want(Y, (E, plan.y_dim), dt, "Y")
    _want(vec, (E, 3), dt, "vec")
    _want(W1, (8, 8), dt, "W1")
    _want(W2, (8, plan.n_paths * plan.U), dt, "W2")
    if out is None:
        out = _empty((N, plan.out_dim), dt, x.device)
    _want(out, (N, plan.out_dim), dt, "out")
    ws = workspace if workspace is not None else _radial_ws(plan, E, 8, x.device)
    _check(lib().oeq_tp_conv_fwd_radial(plan.handle, N, E, _ptr(rowptr), _ptr(src), _ptr(x), _ptr(Y), _ptr(vec),
                                        float(r_cut), _ptr(W1), _ptr(W2), _ptr(out), _ptr(ws), ws.numel(),
                                        _stream()))
    return out


def oeq_tp_conv_bwd_radial(plan: Plan, rowptr, src, x, Y, vec, r_cut: float, W1, W2, grad_out, mode: str = "atomic",
                           want=("x", "Y", "vec", "W1", "W2"), workspace=None):
    """VJP of oeq_tp_conv_fwd_radial: dict with grad_x, grad_Y, grad_vec, grad_W1, grad_W2
    (None where not in want)."""
    import torch
    N, E = _graph(rowptr, src)
    dt = plan.torch_dtype()
    _want(x, (N, plan.x_dim), dt, "x")
    _want(Y, (E, plan.y_dim), dt, "Y")
    _want(vec, (E, 3), dt, "vec")
    _want(W1, (8, 8), dt, "W1")
    _want(W2, (8, plan.n_paths * plan.U), dt, "W2")
    _want(grad_out, (N, plan.out_dim), dt, "grad_out")
    shapes = {"x": (N, plan.x_dim), "Y": (E, plan.y_dim), "vec": (E, 3), "W1": (8, 8),
              "W2": (8, plan.n_paths * plan.U)}
    out = {k: _empty(shp, dt, x.device) if k in want else None for k, shp in shapes.items()}
    if workspace is None:
        b = ctypes.c_size_t()
        _check(lib().oeq_workspace_size_radial(plan.handle, N, E, _MODES[mode], ctypes.byref(b)))
        raw = torch.empty(b.value + 256, dtype=torch.uint8, device=x.device)
        workspace = raw[(-raw.data_ptr()) % 256:][:b.value]
    _check(lib().oeq_tp_conv_bwd_radial(plan.handle, N, E, _ptr(rowptr), _ptr(src), _ptr(x), _ptr(Y), _ptr(vec),
                                        float(r_cut), _ptr(W1), _ptr(W2), _ptr(grad_out), _ptr(out["x"]),
                                        _ptr(out["Y"]), _ptr(out["vec"]), _ptr(out["W1"]), _ptr(out["W2"]),
                                        _MODES[mode], _ptr(workspace), workspace.numel(), _stream()))
    return out


# ---------------------------------------------------------------------------
# readout operators
# ---------------------------------------------------------------------------

def _elem(t, name):
    """oeq_dtype of a readout operand."""
    import torch
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    code = {torch.float32: OEQ_F32, torch.float16: OEQ_F16, torch.bfloat16: OEQ_BF16}.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    return code


def _rows(t, like, name):
    """A 2-D operand whose rows may be strided (each row contiguous); returns its row stride."""
    import torch
    if not isinstance(t, torch.Tensor) or t.device != like.device:
        raise TypeError(f"{name} must be a tensor on {like.device}")
    if t.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
    if t.dim() != 2 or t.shape != like.shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(like.shape) if like.dim() == 2 else '[rows, columns]'}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    if rows < 2:
        return max(cols, 1)
    if t.stride(0) < cols:
        raise ValueError(f"the rows of {name} overlap")
    return t.stride(0)


def _scratch(nbytes, workspace, device):
    """(tensor, bytes): the caller's workspace, or a 256-byte aligned one."""
    import torch
    if workspace is not None:
        return workspace, workspace.numel() * workspace.element_size()
    if nbytes == 0:
        return None, 0
    raw = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    return raw[(-raw.data_ptr()) % 256:][:nbytes], nbytes


def oeq_group_norm_workspace_size(n_rows: int, n_struct: int, n_channels: int, n_groups: int):
    """Workspace bytes (forward, backward)."""
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().oeq_group_norm_workspace_size(n_rows, n_struct, n_channels, n_groups, ctypes.byref(f),
                                               ctypes.byref(b)))
    return f.value, b.value


def oeq_group_norm_fwd(x, ptr, n_groups: int, weight=None, bias=None, eps: float = 1e-5, act: str = "none", out=None,
                       workspace=None):
    """(out, mean, rstd): group norm of x [rows, C] over the rows of each structure
    (ptr [structures + 1] int32), channels last, with an activation ("none" or "silu").
    weight and bias are fp32 [C]; mean and rstd are fp32 [structures, n_groups]."""
    import torch
    code = _elem(x, "x")
    ld = _rows(x, x, "x")
    T, C = x.shape
    B = ptr.shape[0] - 1
    _want(ptr, (B + 1,), torch.int32, "ptr")
    _want(weight, (C,), torch.float32, "weight")
    _want(bias, (C,), torch.float32, "bias")
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    if out is None:
        out = _empty((T, C), x.dtype, x.device)
    ld_out = _rows(out, x, "out")
    need = oeq_group_norm_workspace_size(T, B, C, n_groups)[0]
    stats = _empty((2, B, n_groups), torch.float32, x.device)
    mean, rstd = stats[0], stats[1]
    ws, nbytes = _scratch(need, workspace, x.device)
    _check(lib().oeq_group_norm_fwd(code, T, B, C, n_groups, ACTS[act], float(eps), _ptr(ptr), _ptr(x), ld,
                                    _ptr(weight), _ptr(bias), _ptr(out), ld_out, _ptr(mean), _ptr(rstd), _ptr(ws),
                                    nbytes, _stream()))
    return out, mean, rstd


def oeq_group_norm_bwd(x, ptr, n_groups: int, mean, rstd, grad_out, weight=None, bias=None, act: str = "none",
                       need=("x", "weight", "bias"), out=None, workspace=None):
    """(grad_x, grad_weight, grad_bias) of <grad_out, oeq_group_norm_fwd(x, ...)>; entries not in
    `need` are None.  `out` may supply the grad_x tensor."""
    import torch
    code = _elem(x, "x")
    ld = _rows(x, x, "x")
    T, C = x.shape
    B = ptr.shape[0] - 1
    _want(ptr, (B + 1,), torch.int32, "ptr")
    _want(weight, (C,), torch.float32, "weight")
    _want(bias, (C,), torch.float32, "bias")
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    nbytes = oeq_group_norm_workspace_size(T, B, C, n_groups)[1]
    _want(mean, (B, n_groups), torch.float32, "mean")
    _want(rstd, (B, n_groups), torch.float32, "rstd")
    ld_g = _rows(grad_out, x, "grad_out")
    gx = None
    if "x" in need:
        gx = out if out is not None else _empty((T, C), x.dtype, x.device)
    ld_gx = _rows(gx, x, "grad_x") if gx is not None else C
    gw = _empty((C,), torch.float32, x.device) if "weight" in need else None
    gb = _empty((C,), torch.float32, x.device) if "bias" in need else None
    ws, nbytes = _scratch(nbytes, workspace, x.device)
    _check(lib().oeq_group_norm_bwd(code, T, B, C, n_groups, ACTS[act], _ptr(ptr), _ptr(x), ld, _ptr(weight),
                                    _ptr(bias), _ptr(mean), _ptr(rstd), _ptr(grad_out), ld_g, _ptr(gx), ld_gx,
                                    _ptr(gw), _ptr(gb), _ptr(ws), nbytes, _stream()))
    return gx, gw, gb


def oeq_dropout_fwd(x, p: float, rng, residual=None, out=None):
    """residual + dropout(x) for x [rows, columns]; rng is an int64 device tensor (seed, offset)
    read when the call runs.  The mask depends on rng and (row, column) only (see oeq.h).
    `out` may be x or residual itself."""
    import torch
    code = _elem(x, "x")
    ld = _rows(x, x, "x")
    _want(rng, (2,), torch.int64, "rng")
    ld_r = _rows(residual, x, "residual") if residual is not None else 0
    if out is None:
        out = _empty(x.shape, x.dtype, x.device)
    ld_o = _rows(out, x, "out")
    _check(lib().oeq_dropout_fwd(code, x.shape[0], x.shape[1], _ptr(x), ld, _ptr(residual), ld_r, float(p), _ptr(rng),
                                 _ptr(out), ld_o, _stream()))
    return out


def oeq_dropout_bwd(grad_out, p: float, rng, out=None):
    """Gradient to x of <grad_out, oeq_dropout_fwd(x, p, rng, ...)>."""
    import torch
    code = _elem(grad_out, "grad_out")
    ld = _rows(grad_out, grad_out, "grad_out")
    _want(rng, (2,), torch.int64, "rng")
    if out is None:
        out = _empty(grad_out.shape, grad_out.dtype, grad_out.device)
    ld_o = _rows(out, grad_out, "grad_x")
    _check(lib().oeq_dropout_bwd(code, grad_out.shape[0], grad_out.shape[1], _ptr(grad_out), ld, float(p), _ptr(rng),
                                 _ptr(out), ld_o, _stream()))
    return out


def _heads(t, shape, like, name):
    """A [rows, heads, dim] operand with strided rows and heads: its two strides."""
    import torch
    if not isinstance(t, torch.Tensor) or t.device != like.device:
        raise TypeError(f"{name} must be a tensor on {like.device}")
    if t.dtype != like.dtype:
        raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.stride(2) != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    # the stride of a dimension of one is arbitrary: it is never stepped over
    return (t.stride(0) if t.shape[0] > 1 else 0), (t.stride(1) if t.shape[1] > 1 else 0)


def _attn_desc(q, k, v, q_ptr, k_ptr, scale, key_mask, p_drop, rng):
    import torch
    code = _elem(q, "q")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [rows, heads, dim]")
    Tq, H, D = q.shape
    Tk, Hk = k.shape[0], k.shape[1]
    qs, ks, vs = _heads(q, (Tq, H, D), q, "q"), _heads(k, (Tk, Hk, D), q, "k"), _heads(v, (Tk, Hk, D), q, "v")
    B = q_ptr.shape[0] - 1
    _want(q_ptr, (B + 1,), torch.int32, "q_ptr")
    _want(k_ptr, (B + 1,), torch.int32, "k_ptr")
    if key_mask is not None:
        _want(key_mask, (Tk,), torch.bool if key_mask.dtype == torch.bool else torch.uint8, "key_mask")
    _want(rng, (2,), torch.int64, "rng")
    return _AttnDesc(code, B, H, Hk, D, Tq, Tk, *qs, *ks, *vs, D ** -0.5 if scale is None else float(scale),
                     float(p_drop))


def oeq_cross_attn_fwd(q, k, v, q_ptr, k_ptr, scale=None, key_mask=None, p_drop: float = 0.0, rng=None, out=None,
                       lse=None, workspace=None):
    """(out, lse): attention of q [Tq, H, D] to the states k, v [Tk, Hkv, D] of their structure
    (q_ptr, k_ptr: row pointers over the same structures).  scale defaults to 1 / sqrt(D);
    key_mask [Tk] (bool or uint8) is nonzero where a state is visible; rng (see
    oeq_dropout_fwd) is needed for p_drop > 0.  lse is fp32 [Tq, H]."""
    import torch
    d = _attn_desc(q, k, v, q_ptr, k_ptr, scale, key_mask, p_drop, rng)
    if out is None:
        out = _empty(q.shape, q.dtype, q.device)
    if lse is None:
        lse = _empty(q.shape[:2], torch.float32, q.device)
    _want(out, q.shape, q.dtype, "out")
    _want(lse, q.shape[:2], torch.float32, "lse")
    need = ctypes.c_size_t()
    _check(lib().oeq_cross_attn_workspace_size(ctypes.byref(d), ctypes.byref(need), None))
    ws, nbytes = _scratch(need.value, workspace, q.device)
    _check(lib().oeq_cross_attn_fwd(ctypes.byref(d), _ptr(q_ptr), _ptr(k_ptr), _ptr(q), _ptr(k), _ptr(v),
                                    _ptr(key_mask), _ptr(rng), _ptr(out), _ptr(lse), _ptr(ws), nbytes, _stream()))
    return out, lse


def oeq_cross_attn_bwd(q, k, v, q_ptr, k_ptr, out, lse, grad_out, scale=None, key_mask=None, p_drop: float = 0.0,
                       rng=None, need=("q", "k", "v"), grads=None, workspace=None):
    """(grad_q, grad_k, grad_v) of <grad_out, out> from the forward's operands, out and lse;
    entries not in `need` are None.  `grads` may supply preallocated gradients."""
    import torch
    d = _attn_desc(q, k, v, q_ptr, k_ptr, scale, key_mask, p_drop, rng)
    _want(out, q.shape, q.dtype, "out")
    _want(lse, q.shape[:2], torch.float32, "lse")
    _want(grad_out, q.shape, q.dtype, "grad_out")
    shapes = (q.shape, k.shape, k.shape)
    if grads is None:
        grads = tuple(_empty(s, q.dtype, q.device) if n in need else None for n, s in zip(("q", "k", "v"), shapes))
    gq, gk, gv = (_want(t, s, q.dtype, "grad_" + n) for t, s, n in zip(grads, shapes, ("q", "k", "v")))
    nb = ctypes.c_size_t()
    _check(lib().oeq_cross_attn_workspace_size(ctypes.byref(d), None, ctypes.byref(nb)))
    ws, nbytes = _scratch(nb.value, workspace, q.device)
    _check(lib().oeq_cross_attn_bwd(ctypes.byref(d), _ptr(q_ptr), _ptr(k_ptr), _ptr(q), _ptr(k), _ptr(v),
                                    _ptr(key_mask), _ptr(rng), _ptr(out), _ptr(lse), _ptr(grad_out), _ptr(gq),
                                    _ptr(gk), _ptr(gv), _ptr(ws), nbytes, _stream()))
    return gq, gk, gv
