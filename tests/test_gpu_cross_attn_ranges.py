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


# ---- score gradients and probabilities far from one ----------------------------------------------

# Query rows, states, size of grad_out.  The score gradients of a row are about grad_out / states:
# down to 1e-7 here, below fp16's smallest normal number (6e-5) and its last bit (6e-8).
SMALL = [(64, 2048, 1e-2), (64, 2048, 1e-3), (1024, 2048, 1e-3), (20, 8192, 1e-2), (130, 8192, 1e-3)]


@pytest.mark.parametrize("rows,states,size", SMALL)
def test_half_gradients_of_small_score_gradients(rows, states, size):
    # grad_q and grad_k: the result's rounding and a tenth of it from out within delta (its share is
    # 1 / sqrt(states in use)); grad_v: the probabilities are rounded as well, sqrt(2) of it
    q, k, v, g = operands("f16", [rows], [states], 1, 1, 64, rows + states, size)
    got, ref = both(q, k, v, g, [rows], [states])
    for n, times in (("grad_q", 1.35), ("grad_k", 1.35), ("grad_v", 1.75)):
        own = rel_l2(rounded(ref[n], "f16"), ref[n])
        e = rel_l2(host(got[n]), ref[n])
        assert e <= times * own + RTOL["f32"], (n, e, own)


def test_half_gradient_to_values_of_many_states():
    # probabilities near 1e-5, where fp16's steps of 6e-8 are 0.6 % of them
    q, k, v, g = operands("f16", [40], [100000], 1, 1, 32, 5)
    got, ref = both(q, k, v, g, [40], [100000])
    own = rel_l2(rounded(ref["grad_v"], "f16"), ref["grad_v"])
    e = rel_l2(host(got["grad_v"]), ref["grad_v"])
    assert e <= 1.75 * own + RTOL["f32"], (e, own)


@pytest.mark.parametrize("q_len,k_len", [([40], [5]), ([100, 3], [40, 3]), ([2, 1], [90, 70])])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_half_gradients_of_large_score_gradients(q_len, k_len, p):
    # score gradients past 65504, the largest fp16 number, whose gradients to q and k are not.
    # 2^-11 four times (probabilities, out within delta, the rest, the result), as everywhere
    q, k, v, g = operands("f16", q_len, k_len, 2, 2, 64, 17, 4000.0)
    k, q = k * 0.125, q * 0.125
    v = v * 4
    got, ref = both(q, k, v, g, q_len, k_len, p, (3, 4) if p else None)
    for n in ("grad_q", "grad_k", "grad_v"):
        assert np.abs(ref[n]).max() < 65504, n  # the exact results fit
        assert torch.isfinite(got[n]).all(), n
        assert rel_l2(host(got[n]), ref[n]) <= 4 * 2.0 ** -11 + RTOL["f32"], n


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows", [3, 70])
def test_gradients_of_score_gradients_that_grow_and_vanish(rows, kind):
    # values, and with them the score gradients, grow by 2^20 along the states (each wave's running
    # scale has to follow) and are exactly zero for the first hundred and the last
    q, k, v, g = operands(kind, [rows], [700], 2, 1, 32, 23)
    steps = torch.linspace(-12, 8, 700, device="cuda").exp2()
    steps[:100] = 0
    steps[-100:] = 0
    v = (v.float() * steps[:, None, None]).to(v.dtype)
    g[: rows // 2] = 0
    got, ref = both(q, k, v, g, [rows], [700])
    u = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[kind]
    for n in ("grad_q", "grad_k", "grad_v"):
        assert rel_l2(host(got[n]), ref[n]) <= 4 * u + RTOL["f32"], n
    assert torch.all(got["grad_q"][: rows // 2] == 0)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("q_len,k_len", [([500], [70]), ([300, 9], [1000, 40]), ([40], [600])])
@pytest.mark.parametrize("down", [False, True])
def test_gradients_of_rows_of_very_different_size(q_len, k_len, down, kind):
    # grad_out grows (or falls) by 2^20 along the rows, so what the first rows of a walk suggest for the
    # others is far off
    q, k, v, g = operands(kind, q_len, k_len, 4, 2, 64, 43)
    steps = torch.linspace(-14, 6, q.shape[0], device="cuda").exp2()
    g = (g.float() * (steps.flip(0) if down else steps)[:, None, None]).to(g.dtype)
    got, ref = both(q, k, v, g, q_len, k_len)
    u = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[kind]
    for n in ("grad_q", "grad_k", "grad_v"):
        assert rel_l2(host(got[n]), ref[n]) <= 4 * u + RTOL["f32"], n


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows", [3, 200])
def test_gradients_of_values_whose_output_cancels(rows, kind):
    # pairs of states with the same scores and opposite values (size 1000), so that the output, which tells
    # the size of a row's values, is a small rest.  Their keys are opposite where the queries are zero,
    # and there the two gradients of a pair add up
    q, k, v, g = operands(kind, [rows], [80], 2, 1, 32, 59)
    q[..., 16:] = 0
    v *= 1000
    k[1::2], v[1::2] = k[::2], -v[::2]
    k[1::2, :, 16:] *= -1
    v[0, 0, :] *= 1.0078125
    got, ref = both(q, k, v, g, [rows], [80])
    # delta, of an output of the rest's size, is small against the gradients: 4 u as everywhere
    u = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[kind]
    for n in ("grad_q", "grad_k", "grad_v"):
        assert rel_l2(host(got[n]), ref[n]) <= 4 * u + RTOL["f32"], n


@pytest.mark.parametrize("size", [1e-2, 1e-4, 3e-6, 300.0])
@pytest.mark.parametrize("grad", [1e-3, 1.0, 50.0])
def test_half_gradients_of_small_and_large_values(grad, size):
    # the score gradients go with the product of the two sizes, and each has to fit the type as well.  The
    # saved out is subnormal here for small values, so the reference takes delta from it, as the formula
    # of the call does; then grad_q and grad_k carry their own rounding alone, grad_v that of the probabilities too
    q, k, v, g = operands("f16", [90], [300], 2, 1, 64, 61, grad)
    v = (v.float() * size).to(v.dtype)
    qp, kp = index([0, 90]), index([0, 300])
    out, lse = oeq.oeq_cross_attn_fwd(q, k, v, qp, kp)
    got = oeq.oeq_cross_attn_bwd(q, k, v, qp, kp, out, lse, g)
    Q, K, V, G, O = (host(t) for t in (q, k[:, 0], v[:, 0], g, out))
    ref = [np.empty(Q.shape), np.zeros(K.shape), np.zeros(K.shape)]
    for h in range(2):
        S = 0.125 * Q[:, h] @ K.T
        P = np.exp(S - S.max(1, keepdims=True))
        P /= P.sum(1, keepdims=True)
        dS = P * (G[:, h] @ V.T - (G[:, h] * O[:, h]).sum(1, keepdims=True))
        ref[0][:, h] = 0.125 * dS @ K
        ref[1] += 0.125 * dS.T @ Q[:, h]
        ref[2] += P.T @ G[:, h]
    for t, want, times in zip(got, ref, (1.35, 1.35, 1.75)):
        own = rel_l2(rounded(want, "f16"), want)
        e = rel_l2(host(t).reshape(want.shape), want)
        assert e <= times * own + RTOL["f32"], (e, own)


def test_half_gradients_of_bad_values_stay_with_their_rows():
    # NaN and infinite rows of grad_out reach every state of their structure and nothing else
    q, k, v, g = operands("f16", [70, 40], [90, 50], 2, 1, 32, 53)
    clean, _ = both(q, k, v, g, [70, 40], [90, 50])
    for bad in (float("nan"), float("inf")):
        h = g.clone()
        h[5, 1, 3] = bad
        got, _ = both(q, k, v, h, [70, 40], [90, 50])
        assert torch.isnan(got["grad_q"][5, 1]).all()
        assert torch.equal(got["grad_q"][:5], clean["grad_q"][:5]) and torch.equal(got["grad_q"][6:], clean["grad_q"][6:])
        assert not torch.isfinite(got["grad_k"][:90]).any()
        assert torch.equal(got["grad_k"][90:], clean["grad_k"][90:])
        assert torch.equal(got["grad_v"][90:], clean["grad_v"][90:])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("states", [32, 34, 66, 96, 290, 322, 1022])
def test_walks_that_are_done_again_are_repeatable(states, kind):
    # outputs that cancel (see above) make fp16's first walk of the keys fail, at every number of tiles and for
    # four waves that share them
    q, k, v, g = operands(kind, [200], [states], 2, 1, 32, 71)
    q[..., 16:] = 0
    v *= 1000
    k[1::2], v[1::2] = k[::2], -v[::2]
    k[1::2, :, 16:] *= -1
    v[0, 0, :] *= 1.0078125
    args = (q, k, v, index([0, 200]), index([0, states]))
    out, lse = oeq.oeq_cross_attn_fwd(*args)
    first = oeq.oeq_cross_attn_bwd(*args, out, lse, g)
    for _ in range(5):
        again = oeq.oeq_cross_attn_bwd(*args, out, lse, g)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    ref = readout.cross_attn(host(q), host(k), host(v), [0, 200], [0, states], 32 ** -0.5, grad_out=host(g))
    u = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[kind]
    for t, n in zip(first, ("grad_q", "grad_k", "grad_v")):
        assert rel_l2(host(t), ref[n]) <= 4 * u + RTOL["f32"], n


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("q_len,k_len", [([64], [96]), ([300], [9]), ([5, 40], [1000, 33])])
@pytest.mark.parametrize("p", [0.0, 0.25])
def test_half_gradient_to_values_is_near_the_rounded_result(q_len, k_len, p, kind):
    # nothing but the result is rounded to the type: its own error, and a tenth for the sample
    q, k, v, g = operands(kind, q_len, k_len, 4, 2, 32, 67)
    got, ref = both(q, k, v, g, q_len, k_len, p, (21, 22) if p else None)
    own = rel_l2(rounded(ref["grad_v"], kind), ref["grad_v"])
    e = rel_l2(host(got["grad_v"]), ref["grad_v"])
    assert e <= 1.1 * own + RTOL["f32"], (e, own)


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


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("q_len,k_len", [([5], [70]), ([150], [90]), ([40, 3], [33, 200])])
def test_gradients_beside_one_infinite_column_of_the_states(q_len, k_len, kind):
    # every fifth state is unseen by -infinity in one column: grad_q is NaN there, zero times infinity, and in
    # the other columns what it is without these states
    q, k, v, g = operands(kind, q_len, k_len, 2, 1, 32, 73)
    q[..., 3] = q[..., 3].abs() + 0.125
    mask = torch.ones(k.shape[0], dtype=torch.uint8, device="cuda")
    mask[::5] = 0
    _, ref = both(q, k, v, g, q_len, k_len, mask=mask)
    k[::5, :, 3] = -float("inf")
    qp, kp = index(ptr(q_len)), index(ptr(k_len))
    out, lse = oeq.oeq_cross_attn_fwd(q, k, v, qp, kp)
    got = dict(zip(("grad_q", "grad_k", "grad_v"), oeq.oeq_cross_attn_bwd(q, k, v, qp, kp, out, lse, g)))
    others = [c for c in range(32) if c != 3]
    u = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[kind]
    assert torch.isnan(got["grad_q"][..., 3]).all()
    assert rel_l2(host(got["grad_q"])[..., others], ref["grad_q"][..., others]) <= 4 * u + RTOL["f32"]
    for n in ("grad_k", "grad_v"):
        assert rel_l2(host(got[n]), ref[n]) <= 4 * u + RTOL["f32"], n


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("states", [2, 20, 32, 33, 200])
@pytest.mark.parametrize("gap", [20.0, 80.0, 84.0, 86.0, 87.0, 110.0])
@pytest.mark.parametrize("low", [0.0, -1.0])
def test_gradients_of_rows_that_see_one_state(low, gap, states, kind):
    # the other states' probabilities are e^-gap, down to below the normal fp32 numbers, and so are all score
    # gradients: nothing that fp16 holds, and nothing that is not finite.  With one probability within 2^-24 of one,
    # (dP - delta) is the rounding of a sum of size 10 in 16-bit types (and of the saved out): 4 u of it
    r = np.random.default_rng(79)
    q = torch.zeros((40, 2, 32), dtype=TYPES[kind], device="cuda")
    k = torch.from_numpy(r.normal(size=(states, 1, 32))).to("cuda", TYPES[kind])
    q[..., 0], k[..., 0] = 8.0, low * gap
    k[states // 2, 0, 0] = (low + 1.0) * gap  # at a score of zero its probability is one without rounding
    v, g = (torch.from_numpy(r.normal(size=s)).to("cuda", TYPES[kind]) for s in (k.shape, q.shape))
    args = (q, k, v, index([0, 40]), index([0, states]))
    out, lse = oeq.oeq_cross_attn_fwd(*args, scale=0.125)
    got = oeq.oeq_cross_attn_bwd(*args, out, lse, g, scale=0.125)
    ref = readout.cross_attn(host(q), host(k), host(v), [0, 40], [0, states], 0.125, grad_out=host(g))
    u = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[kind]
    assert rel_l2(host(got[2]), ref["grad_v"]) <= 4 * u + RTOL["f32"]
    # scale |k| u |dP| a row, over 40 rows and 2 heads for grad_k
    assert np.abs(host(got[0]) - ref["grad_q"]).max() <= 0.125 * gap * 4 * u * 20 + 1e-3
    assert np.abs(host(got[1]) - ref["grad_k"]).max() <= 0.125 * 8 * 80 * 4 * u * 20 + 1e-3


# ---- the call's own numbers ---------------------------------------------------------------------------

def test_scale_and_probability_are_read_at_each_call():
    # numbers that a program holds in tensors and changes in place between two calls
    q, k, v, _ = operands("f32", [4], [9], 2, 1, 16, 41)
    args = (q, k, v, index([0, 4]), index([0, 9]))
    key = torch.tensor([1, 2], device="cuda")
    scale, p = torch.tensor(0.25, dtype=torch.float64), torch.tensor(0.5, dtype=torch.float64)
    for s, drop in ((0.25, 0.5), (0.75, 0.5), (0.75, 0.125)):
        scale.fill_(s)
        p.fill_(drop)
        got = oeq.oeq_cross_attn_fwd(*args, scale=scale, p_drop=p, rng=key)
        want = oeq.oeq_cross_attn_fwd(*args, scale=s, p_drop=drop, rng=key)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (s, drop)
    got = oeq.oeq_cross_attn_fwd(*args, scale=np.float32(0.5))
    assert torch.equal(got[0], oeq.oeq_cross_attn_fwd(*args, scale=0.5)[0])
    with pytest.raises(TypeError):
        oeq.oeq_cross_attn_fwd(*args, scale="0.25")
