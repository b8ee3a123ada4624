"""Cross attention on the GPU where values leave the middle of their type's range, where a batch
mixes very short structures with long ones, and where rows belong to no structure; against the
fp64 oracle.

Bounds are relative L2 errors.  Of 16-bit types the result itself is rounded, so its own error is
measured by rounding the oracle's result, and the bounds are multiples of that: it holds also
where the result is subnormal.
"""
import numpy as np
import pytest

from helpers import RTOL, rel_l2
from oracle import readout

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
oeq = pytest.importorskip("cg_tensor_product_amd")

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def host(t):
    return t.detach().double().cpu().numpy()


def ptr(lengths):
    return [0, *np.cumsum(lengths).tolist()]


def index(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rounded(a, kind):
    return torch.from_numpy(a).to(TYPES[kind]).double().numpy()


def operands(kind, q_len, k_len, heads, kv_heads, dim, seed, grad=1.0):
    r = np.random.default_rng(seed)
    nq, nk = sum(q_len), sum(k_len)

    def rand(*shape, s=1.0):
        return torch.from_numpy(r.normal(0, s, shape)).to("cuda", TYPES[kind])

    return (rand(nq, heads, dim, s=1.5), rand(nk, kv_heads, dim), rand(nk, kv_heads, dim),
            rand(nq, heads, dim, s=grad))


def both(q, k, v, g, q_len, k_len, p=0.0, key=None, mask=None):
    """(the library's results, the oracle's), by name"""
    qp, kp = index(ptr(q_len)), index(ptr(k_len))
    kw = dict(p_drop=p, rng=None if key is None else torch.tensor(key, device="cuda"), key_mask=mask)
    out, lse = oeq.oeq_cross_attn_fwd(q, k, v, qp, kp, **kw)
    grads = oeq.oeq_cross_attn_bwd(q, k, v, qp, kp, out, lse, g, **kw)
    got = dict(zip(("out", "lse", "grad_q", "grad_k", "grad_v"), (out, lse, *grads)))
    return got, readout.cross_attn(host(q), host(k), host(v), ptr(q_len), ptr(k_len), q.shape[2] ** -0.5,
                                   None if mask is None else host(mask), p, key, host(g))


# ---- structures of few states beside long ones ------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("mates", [[], [2000], [9, 1, 300]])
@pytest.mark.parametrize("rows,p", [(8, 0.0), (100, 0.0), (40, 0.25)])
def test_gradients_of_few_states_do_not_depend_on_the_batch(rows, p, mates, kind):
    # With few states the rounding of the saved out is most of what delta = grad_out out loses, so
    # delta is summed from p dp there: grad_q and grad_k then only carry their own rounding
    k_len = [2, 4, 7, 31, 32, *mates]
    q_len = [rows] * len(k_len)
    q, k, v, g = operands(kind, q_len, k_len, 4, 2, 32, 29)
    mask = torch.ones(sum(k_len), dtype=torch.uint8, device="cuda")
    mask[[9, 20, 21]] = 0  # of the third and the fourth structure
    got, ref = both(q, k, v, g, q_len, k_len, p, (11, 12) if p else None, mask)
    qp, kp = ptr(q_len), ptr(k_len)
    for s in range(5):
        for n, rows_of in (("grad_q", slice(qp[s], qp[s + 1])), ("grad_k", slice(kp[s], kp[s + 1]))):
            want = ref[n][rows_of]
            own = rel_l2(rounded(want, kind), want)
            e = rel_l2(host(got[n])[rows_of], want)
            assert e <= 1.35 * own + RTOL["f32"], (n, k_len[s], e, own)


# ---- rows of no structure -----------------------------------------------------------------------------

@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("first,q_end,k_end,q_rows,k_rows", [(0, 2, 3000, 4, 3000), (1, 3, 2900, 4, 3000),
                                                             (30, 800, 1500, 900, 1600), (0, 2000, 20, 2100, 30)])
def test_rows_of_no_structure_are_not_written(first, q_end, k_end, q_rows, k_rows, kind):
    # long states and long queries: keys and queries are split over workgroups and joined
    q, k, v, g = operands(kind, [q_rows], [k_rows], 2, 1, 64, 31)
    qp, kp = index([first, q_end]), index([first, k_end])
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    oeq.oeq_cross_attn_fwd(q, k, v, qp, kp, out=out, lse=lse)
    grads = tuple(torch.full_like(t, 7.0) for t in (q, k, k))
    oeq.oeq_cross_attn_bwd(q, k, v, qp, kp, out, lse, g, grads=grads)
    held_q, held_k = slice(first, q_end), slice(first, k_end)
    for t, held in ((out, held_q), (lse, held_q), (grads[0], held_q), (grads[1], held_k), (grads[2], held_k)):
        inside = torch.zeros(t.shape[0], dtype=torch.bool, device="cuda")
        inside[held] = True
        assert torch.all(t[~inside] == 7)
    # what the same structure gives on its own
    args = [t[held].contiguous() for t, held in ((q, held_q), (k, held_k), (v, held_k))]
    got, ref = both(*args, g[held_q].contiguous(), [q_end - first], [k_end - first])
    u = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[kind]
    assert rel_l2(host(out[held_q]), ref["out"]) <= 2 * u + RTOL["f32"]
    for t, n, held in zip(grads, ("grad_q", "grad_k", "grad_v"), (held_q, held_k, held_k)):
        assert rel_l2(host(t[held]), ref[n]) <= 4 * u + RTOL["f32"], n


# ---- infinite states ------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("q_len,k_len", [([5], [20]), ([33, 1], [70, 200]), ([1], [9]), ([129], [40])])
def test_gradients_of_states_with_minus_infinite_scores(q_len, k_len, kind):
    # every other visible state has the score -infinity for every row, so a probability of zero: its
    # gradients are zero and the other states' are what they would be without it.  (grad_q takes
    # zero times the infinite state, which is NaN in the formula too.)
    q, k, v, g = operands(kind, q_len, k_len, 2, 1, 32, 37)
    q = q.abs() + 0.125
    k[::2] = -float("inf")
    got, ref = both(q, k, v, g, q_len, k_len)
    u = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[kind]
    assert rel_l2(host(got["out"]), ref["out"]) <= 2 * u + RTOL["f32"]
    for n in ("grad_k", "grad_v"):
        assert torch.all(got[n][::2] == 0), n
        assert rel_l2(host(got[n]), ref[n]) <= 4 * u + RTOL["f32"], n
