"""Host-side checks of the decoder operators' C ABI (no GPU needed): every refusal comes back as a
status code before any device work, and workspace sizes are functions of the shapes."""
import ctypes

import pytest

oeq = pytest.importorskip("cg_tensor_product_amd")

P = ctypes.c_void_p
A = P(4096)  # an address that is never followed: the calls below stop before any device work


def _message():
    return oeq.lib().oeq_last_error().decode()


# ---- embedding ----------------------------------------------------------------------------

def _emb(dtype=0, table=5, cols=8, rows=4, t=A, ld_t=8, index=A, size=8, scale=1.0, out=A, ld_o=8):
    return oeq.lib().oeq_embedding_fwd(dtype, table, cols, rows, t, ld_t, index, size, scale, out, ld_o, None)


def _emb_bwd(dtype=0, table=50, cols=8, rows=4, index=A, size=8, scale=1.0, go=A, ld_go=8, gt=A, ld_gt=8, ws=A,
             wsb=1 << 20):
    return oeq.lib().oeq_embedding_bwd(dtype, table, cols, rows, index, size, scale, go, ld_go, gt, ld_gt, ws, wsb, None)


SHARED = [
    (dict(dtype=1), 2), (dict(dtype=9), 2), (dict(table=-1), 1), (dict(cols=-1), 1), (dict(rows=-1), 1),
    (dict(table=2**31 - 1), 2), (dict(rows=2**31 - 1), 2), (dict(cols=2**31 - 1), 2), (dict(cols=2**23), 2), (dict(size=2), 1), (dict(size=0), 1),
    (dict(index=None), 1), (dict(index=P(4100)), 1), (dict(index=P(4098), size=4), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(scale=1e300), 1),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(t=None), 1), (dict(out=None), 1), (dict(ld_t=7), 1), (dict(ld_o=7), 1), (dict(t=P(4098)), 1),
    (dict(out=P(4097), dtype=2), 1),
])
def test_embedding_refusals(kw, status):
    assert _emb(**kw) == status, _message()


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(go=None), 1), (dict(gt=None), 1), (dict(ld_go=7), 1), (dict(ld_gt=7), 1), (dict(go=P(4098)), 1),
    (dict(gt=P(4097), dtype=3), 1), (dict(ws=None), 3), (dict(wsb=31), 3), (dict(ws=P(4104)), 3),
])
def test_embedding_backward_refusals(kw, status):
    assert _emb_bwd(**kw) == status, _message()


def test_embedding_empty_calls_do_nothing():
    assert _emb(rows=0, index=None, out=None, t=None) == 0 and _emb(cols=0, out=None, t=None) == 0
    assert _emb_bwd(table=0, gt=None) == 0 and _emb_bwd(cols=0, gt=None, ws=None) == 0


def test_embedding_workspace_sizes():
    b = ctypes.c_size_t()
    size = oeq.lib().oeq_embedding_workspace_size
    assert size(0, 100, 64, 0, ctypes.byref(b)) == 0 and b.value == 0
    assert size(0, 100, 64, 10, ctypes.byref(b)) == 0 and b.value >= 2 * 10 * 4  # keys and positions
    assert size(0, 1 << 20, 64, 10**6, ctypes.byref(b)) == 0 and b.value >= 4 * 10**6 * 4
    assert size(0, 0, 64, 10, ctypes.byref(b)) == 0 and b.value == 0
    assert size(0, 100, 64, 10, None) == 0
    # a table of few rows: sums of strips of rows, none where one strip holds them all
    assert size(0, 5, 64, 10, ctypes.byref(b)) == 0 and b.value == 0
    assert size(0, 5, 64, 10**6, ctypes.byref(b)) == 0 and b.value >= 2 * 5 * 64 * 4
    assert size(0, 16, 2**31 - 2, 10, ctypes.byref(b)) == 2  # a launch of too many workgroups


# ---- rms norm -------------------------------------------------------------------------------

def _rms(dtype=0, rows=3, cols=8, eps=1e-5, x=A, ld=8, res=None, ld_r=0, w=None, s=None, ld_s=0, out=A, ld_o=8,
         scale=None, rstd=A):
    return oeq.lib().oeq_rms_norm_fwd(dtype, rows, cols, eps, x, ld, res, ld_r, w, s, ld_s, out, ld_o, scale, rstd, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=1), 2), (dict(rows=-1), 1), (dict(cols=0), 1), (dict(cols=16385), 2), (dict(rows=2**40), 2),
    (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(eps=1e-60), 1), (dict(x=None), 1), (dict(out=None), 1), (dict(ld=7), 1), (dict(ld_o=7), 1),
    (dict(x=P(4098)), 1), (dict(out=P(4098)), 1), (dict(w=P(4098)), 1), (dict(rstd=P(4098)), 1),
    (dict(scale=P(4097)), 1), (dict(res=A, ld_r=8), 1), (dict(res=A, ld_r=7, s=A, ld_s=8), 1),
    (dict(res=A, ld_r=8, s=A, ld_s=7), 1), (dict(res=P(4098), ld_r=8, s=A, ld_s=8), 1),
    (dict(res=A, ld_r=8, s=P(4098), ld_s=8), 1),
])
def test_rms_norm_refusals(kw, status):
    assert _rms(**kw) == status, _message()


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=1), 2), (dict(cols=0), 1), (dict(cols=16385), 2), (dict(s=None), 1), (dict(go=None), 1),
    (dict(rstd=None), 1), (dict(ld_s=7), 1), (dict(ld_go=7), 1), (dict(gs=A, ld_gs=7), 1), (dict(ld_gx=7), 1),
    (dict(gx=P(4098)), 1), (dict(gw=P(4098)), 1), (dict(w=P(4098)), 1), (dict(ws=None), 3), (dict(wsb=31), 3),
    (dict(ws=P(4104)), 3), (dict(gx=None, gw=None), 0), (dict(rows=0, s=None, go=None, rstd=None, gx=None, gw=None), 0),
])
def test_rms_norm_backward_refusals(kw, status):
    k = {**dict(dtype=0, rows=3, cols=8, s=A, ld_s=8, w=None, rstd=A, go=A, ld_go=8, gs=None, ld_gs=0, gx=A, ld_gx=8,
                gw=A, ws=A, wsb=1 << 20), **kw}
    assert oeq.lib().oeq_rms_norm_bwd(*k.values(), None) == status, _message()


def test_rms_norm_empty_calls_do_nothing():
    assert _rms(rows=0, x=None, out=None, rstd=None) == 0


def test_rms_norm_workspace_sizes():
    b = ctypes.c_size_t()
    size = oeq.lib().oeq_rms_norm_workspace_size
    assert size(0, 64, ctypes.byref(b)) == 0 and b.value == 0
    assert size(10, 4096, ctypes.byref(b)) == 0 and b.value >= 4096 * 4
    assert size(10, 0, ctypes.byref(b)) == 1 and size(-1, 8, None) == 1 and size(10, 16385, None) == 2


# ---- causal attention -------------------------------------------------------------------------

FIELDS = dict(dtype=0, n_struct=2, n_heads=4, n_kv_heads=2, head_dim=16, q_rows=6, k_rows=9, q_stride=64,
              q_head_stride=16, k_stride=32, k_head_stride=16, v_stride=32, v_head_stride=16, scale=0.25, p_drop=0.0)


def _desc(**kw):
    return oeq._AttnDesc(*{**FIELDS, **kw}.values())


def _attn(desc, q_ptr=A, k_ptr=A, k_len=None, q=A, k=A, v=A, mask=None, rng=None, out=A, lse=A, ws=None, wsb=0):
    return oeq.lib().oeq_causal_attn_fwd(None if desc is None else ctypes.byref(desc), q_ptr, k_ptr, k_len, q, k, v, mask,
                                         rng, out, lse, ws, wsb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=1), 2), (dict(n_struct=-1), 1), (dict(n_struct=0), 1), (dict(n_heads=3), 1), (dict(n_heads=0), 1),
    (dict(n_kv_heads=0), 1), (dict(head_dim=0), 1), (dict(head_dim=12), 2), (dict(head_dim=136), 2),
    (dict(q_rows=-1), 1), (dict(k_rows=-1), 1), (dict(q_rows=2**29), 2), (dict(q_rows=2**29 - 256), 2),
    (dict(k_rows=2**31), 2), (dict(scale=0.0), 1), (dict(scale=float("inf")), 1), (dict(p_drop=1.0), 1),
    (dict(p_drop=0.1), 1), (dict(q_stride=66), 1), (dict(k_stride=-32), 1), (dict(v_head_stride=2), 1),
    (dict(n_struct=1 << 26, n_heads=64, n_kv_heads=64), 2),
])
def test_causal_attn_descriptor_refusals(kw, status):
    assert _attn(_desc(**kw)) == status, _message()


@pytest.mark.parametrize("kw,status", [
    (dict(q_ptr=None), 1), (dict(k_ptr=None), 1), (dict(k_len=P(4098)), 1), (dict(q=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(out=None), 1), (dict(lse=None), 1), (dict(q=P(4104)), 1), (dict(k=P(4100)), 1),
    (dict(out=P(4100)), 1), (dict(q_ptr=P(4098)), 1),
])
def test_causal_attn_operand_refusals(kw, status):
    assert _attn(_desc(), **kw) == status, _message()
    assert _attn(None) == 1


def test_causal_attn_backward_refusals():
    def call(desc=_desc(), out=A, lse=A, go=A, gq=A, gk=A, gv=A, ws=None, wsb=0):
        return oeq.lib().oeq_causal_attn_bwd(ctypes.byref(desc), A, A, A, A, A, None, None, out, lse, go, gq, gk, gv, ws,
                                             wsb, None)

    assert call(out=None) == 1 and call(lse=None) == 1 and call(go=None) == 1
    assert call(gk=P(4104)) == 1 and call(go=P(4104)) == 1
    assert call(gq=None, gk=None, gv=None) == 0  # nothing asked for
    assert call() == 3 and call(ws=P(4104), wsb=1 << 40) == 3  # delta needs a workspace


def test_causal_attn_workspace_sizes():
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    size = oeq.lib().oeq_causal_attn_workspace_size
    assert size(ctypes.byref(_desc()), ctypes.byref(f), ctypes.byref(b)) == 0 and f.value == 0
    assert b.value >= 6 * 4 * 4  # delta
    d = _desc(n_struct=1, q_rows=1, k_rows=100000)  # long states, few rows: outputs and log sums of each split
    assert size(ctypes.byref(d), ctypes.byref(f), None) == 0 and f.value >= 2 * 4 * (16 + 1) * 4
    assert _attn(d) == 3
    empty = _desc(n_struct=0, q_rows=0, k_rows=0)
    assert size(ctypes.byref(empty), ctypes.byref(f), ctypes.byref(b)) == 0 and f.value == b.value == 0
    assert _attn(empty, q_ptr=None, k_ptr=None, q=None, k=None, v=None, out=None, lse=None) == 0


@pytest.mark.parametrize("rows", [1 << 24, 1 << 26, (1 << 26) + 777777, (1 << 27) - 400])
@pytest.mark.parametrize("n_struct", [1, 2, 3, 1000])
@pytest.mark.parametrize("dtype", [0, 2, 3])
def test_causal_attn_workspace_of_the_longest_walks(rows, n_struct, dtype):
    # enough rows to fill the chip without cutting a walk: no partial results, however long the walks are
    d = _desc(n_struct=n_struct, n_heads=8, n_kv_heads=8, head_dim=32, q_rows=rows, k_rows=rows, dtype=dtype)
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    status = oeq.lib().oeq_causal_attn_workspace_size(ctypes.byref(d), ctypes.byref(f), ctypes.byref(b))
    if 2 * 8 * (rows // 128 + n_struct) >= 1 << 24:  # the backward's workgroups, of both roles
        assert status == 2
        return
    assert status == 0, _message()
    assert f.value == 0 and rows * 8 * 4 <= b.value < rows * 8 * 4 + 4096  # delta
