"""Cross attention on the GPU against the fp64 oracle.

Bounds, relative L2 per output tensor on the same (rounded) inputs, with u the unit roundoff of
a 16-bit type (2^-11 for fp16, 2^-8 for bf16) and the suite's 1e-5 for fp32 arithmetic:
  out: 2 u + 1e-5 (the probabilities are rounded once for their product, the result once);
  gradients: 4 u + 1e-5 (probabilities and score gradients, the saved out within delta, the
  result); lse is fp32: 1e-5.
fp32 rounds none of these: 1e-5 throughout.
"""
import math

import numpy as np
import pytest

from helpers import RTOL, rel_l2
from oracle import readout

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
oeq = pytest.importorskip("cg_tensor_product_amd")

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}

# query rows and states of each structure, heads, key heads, head dimension
CASES = {
    "tokens": ([1, 1, 1], [5, 17, 1], 4, 2, 16),
    "empty_sides": ([0, 3, 0, 5, 2], [4, 0, 0, 70, 3], 2, 2, 32),
    "odd_lengths": ([33, 1, 129], [31, 65, 200], 3, 1, 40),
    "one_tile": ([32, 32], [32, 64], 2, 1, 64),
    "past_a_tile": ([129], [65], 2, 2, 64),
    "shared_token": ([1, 1], [200, 33], 8, 1, 24),
    "long_states": ([1, 2], [3000, 10], 2, 1, 128),
    "long_states_many_rows": ([200], [2500], 1, 1, 96),
    "long_queries": ([2000, 3], [20, 33], 2, 1, 32),
    "many_structures": ([1 + i % 3 for i in range(70)], [i % 9 for i in range(70)], 2, 2, 8),
    "wide_head": ([70], [90], 2, 2, 120),
    "dim_80": ([40, 7], [100, 37], 4, 2, 80),
    "two_splits": ([150], [600], 1, 1, 48),
    "few_states_many_rows": ([300, 5], [9, 24], 4, 1, 104),
    "many_shared_heads": ([3, 40], [90, 33], 12, 1, 16),
}


def host(t):
    return t.detach().double().cpu().numpy()


def ptr(lengths):
    return [0, *np.cumsum(lengths).tolist()]


def index(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rng_state(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


class Case:
    def __init__(self, name, kind, seed=0, masked=0.0, scale=None):
        self.q_len, self.k_len, self.H, self.Hk, self.D = CASES[name]
        self.kind = kind
        self.q_ptr, self.k_ptr = ptr(self.q_len), ptr(self.k_len)
        r = np.random.default_rng(seed + len(name))

        def rand(*shape, s=1.0):
            return torch.from_numpy(r.normal(0, s, shape)).to("cuda", TYPES[kind])

        self.q = rand(self.q_ptr[-1], self.H, self.D, s=1.5)
        kv = rand(self.k_ptr[-1], 2, self.Hk, self.D)
        self.k, self.v = kv[:, 0], kv[:, 1]  # strided, as a fused projection leaves them
        self.g = rand(*self.q.shape)
        self.mask = None
        if masked:
            self.mask = torch.from_numpy((r.random(self.k_ptr[-1]) >= masked).astype(np.uint8)).cuda()
        self.scale = 1 / math.sqrt(self.D) if scale is None else scale

    def run(self, p=0.0, rng=None, need=("q", "k", "v")):
        kw = dict(scale=self.scale, key_mask=self.mask, p_drop=p, rng=rng)
        qp, kp = index(self.q_ptr), index(self.k_ptr)
        out, lse = oeq.oeq_cross_attn_fwd(self.q, self.k, self.v, qp, kp, **kw)
        gq, gk, gv = oeq.oeq_cross_attn_bwd(self.q, self.k, self.v, qp, kp, out, lse, self.g, need=need, **kw)
        return {"out": out, "lse": lse, "grad_q": gq, "grad_k": gk, "grad_v": gv}

    def reference(self, p=0.0, rng=None):
        return readout.cross_attn(host(self.q), host(self.k), host(self.v), self.q_ptr, self.k_ptr, self.scale,
                                  None if self.mask is None else host(self.mask), p, rng, host(self.g))

    def check(self, got, ref):
        u = UNIT[self.kind]
        lse = host(got["lse"])
        seen = np.isfinite(ref["lse"])
        assert np.array_equal(np.isfinite(lse), seen) and np.all(lse[~seen] == -np.inf)
        assert rel_l2(lse[seen], ref["lse"][seen]) <= RTOL["f32"]
        for name, times in (("out", 2), ("grad_q", 4), ("grad_k", 4), ("grad_v", 4)):
            assert got[name].dtype == TYPES[self.kind]
            e = rel_l2(host(got[name]), ref[name])
            assert e <= times * u + RTOL["f32"], (name, e)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("masked", [0.0, 0.3])
@pytest.mark.parametrize("name", list(CASES))
def test_cross_attn(name, masked, kind):
    c = Case(name, kind, masked=masked)
    c.check(c.run(), c.reference())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("name", list(CASES))
def test_cross_attn_with_dropout(name, kind):
    c = Case(name, kind, seed=1, masked=0.2)
    seed, offset, p = 0x123456789ABCDEF, (7 << 32) + 3, 0.25
    c.check(c.run(p, rng_state(seed, offset)), c.reference(p, (seed, offset)))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("name", ["odd_lengths", "long_states", "tokens"])
def test_cross_attn_of_large_scores(name, kind):
    # scores of a few hundred: without the maximum taken out every exponential would overflow
    c = Case(name, kind, seed=2, scale=20.0)
    got, ref = c.run(), c.reference()
    # a score of size S carries rounding 2^-23 S (its terms' sums), which the exponential takes
    # as a relative error of the probabilities
    size = float(np.abs(ref["lse"][np.isfinite(ref["lse"])]).max())
    extra = size * 2.0 ** -21
    assert rel_l2(host(got["lse"]), ref["lse"]) <= RTOL["f32"]
    for n, times in (("out", 2), ("grad_v", 4)):
        assert rel_l2(host(got[n]), ref[n]) <= times * UNIT[kind] + RTOL["f32"] + extra


@pytest.mark.parametrize("name", ["tokens", "odd_lengths", "long_states", "long_queries"])
def test_cross_attn_never_uses_masked_states(name):
    c = Case(name, "bf16", seed=3, masked=0.4)
    clean = c.run(0.1, rng_state(1, 1))
    c.k, c.v = c.k.clone(), c.v.clone()
    hidden = c.mask == 0
    c.k[hidden] = float("nan")
    c.v[hidden] = float("inf")
    dirty = c.run(0.1, rng_state(1, 1))
    for n in clean:
        assert torch.equal(clean[n], dirty[n]), n
    assert torch.all(dirty["grad_k"][hidden] == 0) and torch.all(dirty["grad_v"][hidden] == 0)


@pytest.mark.parametrize("name", ["tokens", "odd_lengths", "long_states", "long_queries"])
@pytest.mark.parametrize("kind", list(TYPES))
def test_cross_attn_rows_that_see_nothing(name, kind):
    c = Case(name, kind, seed=4)
    c.mask = torch.ones(c.k_ptr[-1], dtype=torch.uint8, device="cuda")
    c.mask[:c.k_ptr[1]] = 0  # the whole first structure
    got = c.run()
    rows, states = slice(0, c.q_ptr[1]), slice(0, c.k_ptr[1])
    assert torch.all(got["out"][rows] == 0) and torch.all(got["lse"][rows] == -math.inf)
    assert torch.all(got["grad_q"][rows] == 0)
    assert torch.all(got["grad_k"][states] == 0) and torch.all(got["grad_v"][states] == 0)
    if c.q_ptr[1] < c.q_ptr[-1]:
        c.check(got, c.reference())


@pytest.mark.parametrize("name", ["tokens", "past_a_tile"])
def test_cross_attn_of_minus_infinite_scores(name):
    # states whose score is -infinity count as unseen; a row of them alone is a zero row
    c = Case(name, "f32", seed=5)
    c.k = c.k.clone()
    c.q = c.q.abs() + 0.1
    some = torch.zeros(c.k_ptr[-1], dtype=torch.bool, device="cuda")
    some[c.k_ptr[0]:c.k_ptr[1]:2] = True
    c.k[some] = -math.inf
    qp, kp = index(c.q_ptr), index(c.k_ptr)
    out, lse = oeq.oeq_cross_attn_fwd(c.q, c.k, c.v, qp, kp)
    k2 = c.k.clone()
    k2[some] = 0
    want, lse2 = oeq.oeq_cross_attn_fwd(c.q, k2, c.v, qp, kp, key_mask=(~some).to(torch.uint8))
    assert rel_l2(host(out), host(want)) <= 1e-6 and rel_l2(host(lse), host(lse2)) <= 1e-6
    k2[:] = -math.inf
    out, lse = oeq.oeq_cross_attn_fwd(c.q, k2, c.v, qp, kp)
    assert torch.all(out == 0) and torch.all(lse == -math.inf)


def test_cross_attn_passes_on_nan_of_visible_states():
    c = Case("odd_lengths", "f32", seed=6)
    c.v = c.v.clone()
    c.v[3, 0, 5] = float("nan")  # a state of the first structure
    got = c.run()
    assert torch.isnan(got["out"][:33, :, 5]).all()
    assert torch.isfinite(got["out"][33:]).all() and torch.isfinite(got["grad_q"][33:]).all()
    c.k = c.k.clone()
    c.k[3] = float("nan")
    got = c.run()
    assert torch.isnan(got["out"][:33]).all() and torch.isnan(got["lse"][:33]).all()
    assert torch.isfinite(got["out"][33:]).all()


def test_cross_attn_of_one_state():
    # one state: its probability is one whatever the score, so out = v and the scores get nothing
    r = np.random.default_rng(7)
    q = torch.from_numpy(r.normal(size=(5, 2, 16))).float().cuda()
    k, v, g = q[:1].clone(), q[1:2].clone(), q.flip(0).contiguous()
    qp, kp = index([0, 5]), index([0, 1])
    out, lse = oeq.oeq_cross_attn_fwd(q, k, v, qp, kp)
    gq, gk, gv = oeq.oeq_cross_attn_bwd(q, k, v, qp, kp, out, lse, g)
    # eps times the largest score (about 10) of error in a probability, times gradients of order 10
    assert (out - v).abs().max() <= 1e-5
    assert gq.abs().max() <= 1e-3 and gk.abs().max() <= 1e-3
    assert rel_l2(host(gv), host(g).sum(0, keepdims=True)) <= RTOL["f32"]


def test_cross_attn_gradients_of_half_types_are_near_the_rounded_result():
    # of 96 states the rounding of out within delta is left (0.6 of the result's own at most, by
    # its share 1 / sqrt(states in use)): sqrt(1 + 0.6^2) = 1.17, with room for the sample
    for kind in ("bf16", "f16"):
        r = np.random.default_rng(15)
        q, g = (torch.from_numpy(r.normal(0, s, (64, 2, 32))).to("cuda", TYPES[kind]) for s in (1.5, 1.0))
        k, v = (torch.from_numpy(r.normal(size=(96, 2, 32))).to("cuda", TYPES[kind]) for _ in range(2))
        args = (index([0, 64]), index([0, 96]))
        out, lse = oeq.oeq_cross_attn_fwd(q, k, v, *args)
        got = oeq.oeq_cross_attn_bwd(q, k, v, *args, out, lse, g, need=("q", "k"))
        ref = readout.cross_attn(host(q), host(k), host(v), [0, 64], [0, 96], 32 ** -0.5, grad_out=host(g))
        for t, n in zip(got, ("grad_q", "grad_k")):
            rounded = torch.from_numpy(ref[n]).to(TYPES[kind]).double().numpy()
            assert rel_l2(host(t), ref[n]) <= 1.35 * rel_l2(rounded, ref[n]), n


@pytest.mark.parametrize("need", [("q",), ("k",), ("v",), ("k", "v"), ()])
@pytest.mark.parametrize("name", ["odd_lengths", "long_queries", "long_states"])
def test_cross_attn_gradients_on_request(name, need):
    c = Case(name, "f16", seed=8)
    every, some = c.run(), c.run(need=need)
    for n in ("q", "k", "v"):
        a, b = every["grad_" + n], some["grad_" + n]
        assert (b is None) if n not in need else torch.equal(a, b)


@pytest.mark.parametrize("name", ["long_states", "long_queries", "odd_lengths", "long_states_many_rows"])
def test_cross_attn_is_bitwise_repeatable(name):
    c = Case(name, "bf16", seed=9)
    first = c.run(0.2, rng_state(4, 4))
    for _ in range(3):
        again = c.run(0.2, rng_state(4, 4))
        assert all(torch.equal(first[n], again[n]) for n in first)


def test_cross_attn_takes_strided_and_broadcast_operands():
    c = Case("odd_lengths", "bf16", seed=10)
    want = c.run()
    # heads before rows in memory, and a bool mask of ones
    c.q = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    c.k = c.k.transpose(0, 1).contiguous().transpose(0, 1)
    c.mask = torch.ones(c.k_ptr[-1], dtype=torch.bool, device="cuda")
    got = c.run()
    assert all(torch.equal(want[n], got[n]) for n in want)
    # one key head expanded to all heads gives what sharing it gives
    qp, kp = index(c.q_ptr), index(c.k_ptr)
    wide = oeq.oeq_cross_attn_fwd(c.q, c.k.expand(-1, 3, -1), c.v.expand(-1, 3, -1), qp, kp)[0]
    assert rel_l2(host(wide), host(want["out"])) <= 2 * UNIT["bf16"]


def test_cross_attn_dropout_is_the_dropout_operators_mask():
    # uniform probabilities (q = 0) and one-hot values: the output is the mask itself
    Tk, H = 16, 2
    q = torch.zeros((3, H, 16), device="cuda")
    v = torch.eye(16, device="cuda")[:, None].expand(Tk, H, 16).contiguous()
    key = rng_state(77, 8)
    out, _ = oeq.oeq_cross_attn_fwd(q, v, v, index([0, 3]), index([0, Tk]), p_drop=0.4, rng=key)
    f = oeq.oeq_dropout_fwd(torch.full((3 * H, Tk), 1.0 / Tk, device="cuda"), 0.4, key)
    assert torch.allclose(out.view(3 * H, Tk), f, rtol=1e-5, atol=0)


def test_cross_attn_of_thousands_of_structures():
    # more than 64 x 64 structures: the search for a workgroup's structure takes three steps
    r = np.random.default_rng(13)
    n = 4500
    q_len, k_len = r.integers(0, 3, n), r.integers(0, 4, n)
    q_len[[0, -1]], k_len[[0, -1]] = 2, 3
    qp, kp = ptr(q_len), ptr(k_len)
    q = torch.from_numpy(r.normal(size=(qp[-1], 1, 8))).float().cuda()
    k = torch.from_numpy(r.normal(size=(kp[-1], 1, 8))).float().cuda()
    v = k.flip(0).contiguous()
    g = q.flip(0).contiguous()
    out, lse = oeq.oeq_cross_attn_fwd(q, k, v, index(qp), index(kp))
    got = oeq.oeq_cross_attn_bwd(q, k, v, index(qp), index(kp), out, lse, g)
    ref = readout.cross_attn(host(q), host(k), host(v), qp, kp, 8 ** -0.5, grad_out=host(g))
    assert rel_l2(host(out), ref["out"]) <= RTOL["f32"]
    for t, n in zip(got, ("grad_q", "grad_k", "grad_v")):
        assert rel_l2(host(t), ref[n]) <= RTOL["f32"], n


@pytest.mark.parametrize("lengths", [([5], [40]), ([200], [40])])
def test_cross_attn_offsets_past_32_bits(lengths):
    # states 2^26 elements apart: the last of 40 is 2.6e9 elements (5 GB) into the buffer
    r = np.random.default_rng(14)
    (nq,), (nk,) = lengths
    stride = 1 << 26
    buffer = torch.empty(stride * (nk - 1) + 64, dtype=torch.bfloat16, device="cuda")
    k, v = (buffer.as_strided((nk, 1, 16), (stride, 16, 1), at) for at in (0, 16))
    for t in (k, v):
        t.copy_(torch.from_numpy(r.normal(size=(nk, 1, 16))))
    q = torch.from_numpy(r.normal(size=(nq, 1, 16))).to("cuda", torch.bfloat16)
    args = (index([0, nq]), index([0, nk]))
    far = oeq.oeq_cross_attn_fwd(q, k, v, *args)
    near = oeq.oeq_cross_attn_fwd(q, k.contiguous(), v.contiguous(), *args)
    assert all(torch.equal(a, b) for a, b in zip(far, near))
    got = oeq.oeq_cross_attn_bwd(q, k, v, *args, *far, q)
    want = oeq.oeq_cross_attn_bwd(q, k.contiguous(), v.contiguous(), *args, *near, q)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_cross_attn_of_nothing():
    e = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    # no structures; no query rows; no states
    out, lse = oeq.oeq_cross_attn_fwd(e(0, 2, 8), e(0, 2, 8), e(0, 2, 8), index([0]), index([0]))
    assert out.shape == (0, 2, 8) and lse.shape == (0, 2)
    k = torch.ones((4, 2, 8), device="cuda")
    out, lse = oeq.oeq_cross_attn_fwd(e(0, 2, 8), k, k, index([0, 0]), index([0, 4]))
    gq, gk, gv = oeq.oeq_cross_attn_bwd(e(0, 2, 8), k, k, index([0, 0]), index([0, 4]), out, lse, e(0, 2, 8))
    assert gq.shape == (0, 2, 8) and torch.all(gk == 0) and torch.all(gv == 0)
    q = torch.ones((3, 2, 8), device="cuda")
    out, lse = oeq.oeq_cross_attn_fwd(q, e(0, 2, 8), e(0, 2, 8), index([0, 3]), index([0, 0]))
    assert torch.all(out == 0) and torch.all(lse == -math.inf)
    gq, gk, gv = oeq.oeq_cross_attn_bwd(q, e(0, 2, 8), e(0, 2, 8), index([0, 3]), index([0, 0]), out, lse, q)
    assert torch.all(gq == 0) and gk.shape == (0, 2, 8)


def test_cross_attn_cuts_row_pointers_to_the_rows():
    q = torch.ones((4, 1, 8), device="cuda")
    out = torch.full_like(q, 3.0)
    oeq.oeq_cross_attn_fwd(q, q, q, index([0, 2, 500]), index([-3, 2, 900]), out=out)
    assert torch.all(out[:2] == 1)


def test_cross_attn_on_another_stream_and_in_a_graph():
    c = Case("odd_lengths", "bf16", seed=11, masked=0.1)
    big = Case("long_states", "bf16", seed=12)  # splits and their workspace
    key = rng_state(5, 50)
    want = [c.run(0.1, key), big.run(0.1, key)]
    torch.cuda.synchronize()
    ptrs = [(index(x.q_ptr), index(x.k_ptr)) for x in (c, big)]

    def step():
        got = []
        for x, (qp, kp) in zip((c, big), ptrs):
            kw = dict(scale=x.scale, key_mask=x.mask, p_drop=0.1, rng=key)
            out, lse = oeq.oeq_cross_attn_fwd(x.q, x.k, x.v, qp, kp, **kw)
            g = oeq.oeq_cross_attn_bwd(x.q, x.k, x.v, qp, kp, out, lse, x.g, **kw)
            got.append(dict(zip(("out", "lse", "grad_q", "grad_k", "grad_v"), (out, lse, *g))))
        return got

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a[n], b[n]) for a, b in zip(want, got) for n in a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(3):
        key[1] = 50 + i
        graph.replay()
        torch.cuda.synchronize()
        copies = [{n: t.clone() for n, t in x.items()} for x in held]
        eager = step()
        assert all(torch.equal(a[n], b[n]) for a, b in zip(copies, eager) for n in a)
        torch.cuda.synchronize()


def test_cross_attn_refusals():
    q, k = torch.ones((4, 4, 16), device="cuda"), torch.ones((6, 2, 16), device="cuda")
    qp, kp = index([0, 4]), index([0, 6])

    def fwd(q=q, k=k, v=None, qp=qp, kp=kp, **kw):
        return oeq.oeq_cross_attn_fwd(q, k, k if v is None else v, qp, kp, **kw)

    fwd()
    wide = torch.ones((4, 4, 136), device="cuda")
    for bad, status in ((dict(k=torch.ones((6, 3, 16), device="cuda")), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
                        (dict(scale=float("nan")), 1), (dict(p_drop=1.0), 1), (dict(p_drop=-0.5), 1),
                        (dict(p_drop=0.1), 1), (dict(q=wide, k=wide, kp=index([0, 4])), 2),
                        (dict(q=q[..., :12].contiguous(), k=k[..., :12].contiguous()), 2),
                        (dict(qp=index([0]), kp=index([0])), 1)):
        with pytest.raises(oeq.OeqError) as e:
            fwd(**bad)
        assert e.value.status == status, bad
    # operands that are not 16-byte aligned
    off = torch.ones(6 * 2 * 16 + 1, device="cuda")[1:].view(6, 2, 16)
    with pytest.raises(oeq.OeqError) as e:
        fwd(k=off)
    assert e.value.status == 1
    odd = torch.ones((6, 2, 18), device="cuda")[..., :16]
    with pytest.raises(oeq.OeqError) as e:
        fwd(k=odd)
    assert e.value.status == 1
    for bad in (dict(k=k.half()), dict(q=q.double()), dict(qp=qp.long()), dict(key_mask=torch.ones(6, device="cuda")),
                dict(q=q.cpu())):
        with pytest.raises(TypeError):
            fwd(**bad)
    for bad in (dict(v=k[:3]), dict(qp=index([0, 2, 4])), dict(key_mask=torch.ones(5, dtype=torch.uint8, device="cuda")),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            fwd(**bad)
    long = torch.ones((4000, 1, 16), device="cuda")
    with pytest.raises(oeq.OeqError) as e:
        fwd(q=long[:1], k=long, qp=index([0, 1]), kp=index([0, 4000]),
            workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    out, lse = fwd()
    with pytest.raises(ValueError):
        oeq.oeq_cross_attn_bwd(q, k, k, qp, kp, out, lse, out[:2])
    with pytest.raises(ValueError):
        oeq.oeq_cross_attn_bwd(q, k, k, qp, kp, out, lse[:2], out)
