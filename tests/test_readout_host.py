"""Host-side checks of the readout operators' C ABI (no GPU needed): every refusal comes back
as a status code before any device work, and workspace sizes are functions of the shapes."""
import ctypes

import pytest

oeq = pytest.importorskip("cg_tensor_product_amd")

P = ctypes.c_void_p
A = P(4096)  # an address that is never followed: the calls below stop before any device work


def _message():
    return oeq.lib().oeq_last_error().decode()


# ---- group norm ---------------------------------------------------------------------------

def _gn(dtype=0, rows=10, n=2, c=8, g=2, act=0, eps=1e-5, ptr=A, x=A, ld=8, w=None, b=None, out=A, ld_out=8, mean=A,
        rstd=A, ws=None, wsb=0):
    return oeq.lib().oeq_group_norm_fwd(dtype, rows, n, c, g, act, eps, ptr, x, ld, w, b, out, ld_out, mean, rstd, ws,
                                        wsb, None)


def _gn_bwd(dtype=0, rows=10, n=2, c=8, g=2, act=0, ptr=A, x=A, ld=8, mean=A, rstd=A, go=A, ld_go=8, gx=A, ld_gx=8,
            gw=A, gb=A, ws=None, wsb=0):
    return oeq.lib().oeq_group_norm_bwd(dtype, rows, n, c, g, act, ptr, x, ld, None, None, mean, rstd, go, ld_go, gx,
                                        ld_gx, gw, gb, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=1), 2), (dict(dtype=9), 2), (dict(act=2), 1), (dict(rows=-1), 1), (dict(n=-1), 1),
    (dict(n=0), 1), (dict(rows=2**31), 2), (dict(c=0), 1), (dict(g=3), 1), (dict(g=0), 1), (dict(g=-2), 1),
    (dict(c=4096, g=1, ld=4096, ld_out=4096), 2), (dict(ptr=None), 1), (dict(x=None), 1), (dict(out=None), 1),
    (dict(mean=None), 1), (dict(rstd=None), 1), (dict(ld=7), 1), (dict(ld_out=7), 1), (dict(eps=0.0), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(x=P(4098)), 1),
    (dict(ptr=P(4097)), 1), (dict(rows=5000, n=1), 3), (dict(rows=5000, n=1, ws=P(4104), wsb=1 << 30), 3),
    (dict(n=1 << 28, g=8), 2),
])
def test_group_norm_forward_refusals(kw, status):
    assert _gn(**kw) == status, _message()


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=1), 2), (dict(go=None), 1), (dict(ld_go=7), 1), (dict(ld_gx=7), 1), (dict(mean=None), 1),
    (dict(gx=P(4097), dtype=2), 1), (dict(), 3), (dict(ws=A, wsb=8), 3),
])
def test_group_norm_backward_refusals(kw, status):
    assert _gn_bwd(**kw) == status, _message()


def test_group_norm_empty_calls_do_nothing():
    assert _gn(rows=0, n=0, ptr=None, x=None, out=None, mean=None, rstd=None) == 0
    assert _gn_bwd(gx=None, gw=None, gb=None) == 0


def test_group_norm_workspace_sizes():
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    size = oeq.lib().oeq_group_norm_workspace_size
    assert size(100, 4, 64, 8, ctypes.byref(f), ctypes.byref(b)) == 0
    assert f.value == 0 and b.value >= 4 * 64 * 2 * 4          # one split: the channel sums alone
    assert size(10**6, 1, 64, 8, ctypes.byref(f), None) == 0 and f.value > 0
    assert size(0, 0, 64, 8, ctypes.byref(f), ctypes.byref(b)) == 0 and f.value == b.value == 0
    assert size(10, 1, 64, 7, ctypes.byref(f), None) == 1


# ---- dropout -----------------------------------------------------------------------------------

def _drop(dtype=0, rows=4, cols=8, x=A, ld=8, res=None, ld_r=0, p=0.1, rng=A, out=A, ld_o=8):
    return oeq.lib().oeq_dropout_fwd(dtype, rows, cols, x, ld, res, ld_r, p, rng, out, ld_o, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=1), 2), (dict(rows=-1), 1), (dict(cols=-1), 1), (dict(rows=2**32), 2), (dict(cols=2**31), 2),
    (dict(p=1.0), 1), (dict(p=-1e-9), 1), (dict(p=float("nan")), 1), (dict(rng=None), 1), (dict(rng=P(4100)), 1),
    (dict(x=None), 1), (dict(out=None), 1), (dict(ld=7), 1), (dict(ld_o=7), 1), (dict(res=A, ld_r=7), 1),
    (dict(x=P(4097), dtype=3), 1),
])
def test_dropout_refusals(kw, status):
    assert _drop(**kw) == status, _message()
    if "res" not in kw:
        k = {**dict(dtype=0, rows=4, cols=8, x=A, ld=8, p=0.1, rng=A, out=A, ld_o=8), **kw}
        assert oeq.lib().oeq_dropout_bwd(k["dtype"], k["rows"], k["cols"], k["x"], k["ld"], k["p"], k["rng"], k["out"],
                                         k["ld_o"], None) == status


def test_dropout_empty_calls_do_nothing():
    assert _drop(rows=0, x=None, out=None) == 0 and _drop(cols=0, x=None, out=None) == 0


# ---- cross attention -----------------------------------------------------------------------------

FIELDS = dict(dtype=0, n_struct=2, n_heads=4, n_kv_heads=2, head_dim=16, q_rows=6, k_rows=9, q_stride=64,
              q_head_stride=16, k_stride=32, k_head_stride=16, v_stride=32, v_head_stride=16, scale=0.25, p_drop=0.0)


def _desc(**kw):
    return oeq._AttnDesc(*{**FIELDS, **kw}.values())


def _attn(desc, q_ptr=A, k_ptr=A, q=A, k=A, v=A, mask=None, rng=None, out=A, lse=A, ws=None, wsb=0):
    return oeq.lib().oeq_cross_attn_fwd(None if desc is None else ctypes.byref(desc), q_ptr, k_ptr, q, k, v, mask, rng,
                                        out, lse, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=1), 2), (dict(n_struct=-1), 1), (dict(n_struct=0), 1), (dict(n_heads=3), 1), (dict(n_heads=0), 1),
    (dict(n_kv_heads=0), 1), (dict(head_dim=0), 1), (dict(head_dim=12), 2), (dict(head_dim=136), 2),
    (dict(q_rows=-1), 1), (dict(k_rows=-1), 1), (dict(q_rows=2**29), 2), (dict(k_rows=2**31), 2), (dict(scale=0.0), 1),
    (dict(scale=-0.25), 1), (dict(scale=float("inf")), 1), (dict(scale=1e-60), 1), (dict(p_drop=1.0), 1),
    (dict(p_drop=-0.1), 1), (dict(p_drop=0.1), 1), (dict(q_stride=66), 1), (dict(k_stride=-32), 1),
    (dict(v_head_stride=2), 1), (dict(n_struct=1 << 26, n_heads=64, n_kv_heads=64), 2),
])
def test_cross_attn_descriptor_refusals(kw, status):
    assert _attn(_desc(**kw)) == status, _message()


@pytest.mark.parametrize("kw,status", [
    (dict(q_ptr=None), 1), (dict(k_ptr=None), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(out=None), 1), (dict(lse=None), 1), (dict(q=P(4104)), 1), (dict(k=P(4100)), 1), (dict(out=P(4100)), 1),
    (dict(q_ptr=P(4098)), 1),
])
def test_cross_attn_operand_refusals(kw, status):
    assert _attn(_desc(), **kw) == status, _message()
    assert _attn(None) == 1


def test_cross_attn_backward_refusals():
    bwd = oeq.lib().oeq_cross_attn_bwd

    def call(desc=_desc(), out=A, lse=A, go=A, gq=A, gk=A, gv=A, ws=None, wsb=0):
        return bwd(ctypes.byref(desc), A, A, A, A, A, None, None, out, lse, go, gq, gk, gv, ws, wsb, None)

    assert call(out=None) == 1 and call(lse=None) == 1 and call(go=None) == 1
    assert call(gk=P(4104)) == 1 and call(go=P(4104)) == 1
    assert call(gq=None, gk=None, gv=None) == 0  # nothing asked for
    long = _desc(n_struct=1, q_rows=8, k_rows=100000)
    assert call(long) == 3 and call(long, ws=P(4104), wsb=1 << 40) == 3


def test_cross_attn_workspace_sizes():
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    size = oeq.lib().oeq_cross_attn_workspace_size
    assert size(ctypes.byref(_desc()), ctypes.byref(f), ctypes.byref(b)) == 0 and f.value == 0
    # long states, few rows: fp32 outputs and log sums of each split
    d = _desc(n_struct=1, q_rows=1, k_rows=100000)
    assert size(ctypes.byref(d), ctypes.byref(f), None) == 0 and f.value >= 2 * 4 * (16 + 1) * 4
    assert _attn(d) == 3
    empty = _desc(n_struct=0, q_rows=0, k_rows=0)
    assert size(ctypes.byref(empty), ctypes.byref(f), ctypes.byref(b)) == 0 and f.value == b.value == 0
    assert _attn(empty, q_ptr=None, k_ptr=None, q=None, k=None, v=None, out=None, lse=None) == 0
