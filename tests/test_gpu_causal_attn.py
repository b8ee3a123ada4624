"""Causal attention on the GPU against the fp64 oracle.

Bounds, relative L2 per output tensor on the same (rounded) inputs, with u the unit roundoff of a 16-bit
type (2^-11 for fp16, 2^-8 for bf16) and the suite's 1e-5 for fp32 arithmetic: out 2 u + 1e-5 (the
probabilities are rounded once for their product, the result once); gradients 2 u + 1e-5 (the saved
out within delta, the result; probabilities and score gradients enter as two terms); lse is fp32: 1e-5.
"""
import math

import numpy as np
import pytest

from helpers import RTOL, rel_l2
from oracle import decoder

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
oeq = pytest.importorskip("cg_tensor_product_amd")

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}

# query rows and states of each sequence, heads, key heads, head dimension
CASES = {
    "tokens": ([1, 1, 1], [5, 17, 1], 4, 2, 16),
    "token_over_many": ([1, 1], [3000, 33], 8, 1, 64),
    "prompts": ([33, 1, 129, 70], None, 2, 2, 32),
    "one_tile": ([32, 32], None, 2, 1, 64),
    "shared_heads": ([65, 31], None, 8, 2, 40),
    "odd_share": ([50, 7], None, 6, 2, 24),
    "past_tiles": ([130, 257], None, 1, 1, 128),
    "chunk": ([40, 3], [200, 65], 4, 1, 128),
    "empty_sides": ([0, 3, 0, 5, 2], [4, 0, 0, 70, 3], 2, 2, 32),
    "more_queries": ([40, 10, 200], [30, 9, 33], 2, 1, 48),
    "many_sequences": ([1 + i % 7 for i in range(70)], None, 2, 2, 8),
    "dim_80": ([100, 37], None, 4, 2, 80),
    "dim_104": ([140], [150], 2, 1, 104),
    "long": ([700], None, 1, 1, 32),
    "tokens_of_wide_heads": ([1, 2], [300, 20], 2, 1, 128),
    "ragged": ([900, 3, 40, 260], None, 2, 1, 64),
    "long_chunk": ([90], [1500], 2, 1, 96),
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
        self.q_len, k_len, self.H, self.Hk, self.D = CASES[name]
        self.k_len = self.q_len if k_len is None else k_len
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
        out, lse = oeq.oeq_causal_attn_fwd(self.q, self.k, self.v, qp, kp, **kw)
        gq, gk, gv = oeq.oeq_causal_attn_bwd(self.q, self.k, self.v, qp, kp, out, lse, self.g, need=need, **kw)
        return {"out": out, "lse": lse, "grad_q": gq, "grad_k": gk, "grad_v": gv}

    def reference(self, p=0.0, rng=None):
        return decoder.causal_attn(host(self.q), host(self.k), host(self.v), self.q_ptr, self.k_ptr, self.scale,
                                   None if self.mask is None else host(self.mask), None, p, rng, host(self.g))

    def check(self, got, ref):
        u = UNIT[self.kind]
        lse = host(got["lse"])
        seen = np.isfinite(ref["lse"])
        assert np.array_equal(np.isfinite(lse), seen) and np.all(lse[~seen] == -np.inf)
        assert rel_l2(lse[seen], ref["lse"][seen]) <= RTOL["f32"]
        assert np.all(host(got["out"])[~seen] == 0) and np.all(host(got["grad_q"])[~seen] == 0)
        for name in ("out", "grad_q", "grad_k", "grad_v"):
            assert got[name].dtype == TYPES[self.kind]
            a, b = host(got[name]), ref[name]
            # sequences of one state have no score gradients: 0 up to the rounding of the dot product p dp
            e = rel_l2(a, b) if np.abs(b).max(initial=0.0) > 1e-6 else float(np.abs(a).max(initial=0.0))
            assert e <= 2 * u + RTOL["f32"], (name, e)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("masked", [0.0, 0.3])
@pytest.mark.parametrize("name", list(CASES))
def test_causal_attn(name, masked, kind):
    c = Case(name, kind, masked=masked)
    c.check(c.run(), c.reference())


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("name", list(CASES))
def test_causal_attn_with_dropout(name, kind):
    c = Case(name, kind, seed=1, masked=0.2)
    seed, offset, p = 0x123456789ABCDEF, (7 << 32) + 3, 0.25
    c.check(c.run(p, rng_state(seed, offset)), c.reference(p, (seed, offset)))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("name", ["prompts", "long_chunk", "tokens"])
def test_causal_attn_of_large_scores(name, kind):
    # scores of a few hundred: without the maximum taken out every exponential would overflow
    c = Case(name, kind, seed=2, scale=20.0)
    got, ref = c.run(), c.reference()
    # a score of size S carries rounding 2^-23 S (its terms' sums), which the exponential takes
    # as a relative error of the probabilities
    size = float(np.abs(ref["lse"][np.isfinite(ref["lse"])]).max())
    extra = size * 2.0 ** -21
    assert rel_l2(host(got["lse"]), ref["lse"]) <= RTOL["f32"]
    for n in ("out", "grad_v"):
        assert rel_l2(host(got[n]), ref[n]) <= 2 * UNIT[kind] + RTOL["f32"] + extra


@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("name", ["prompts", "shared_heads", "chunk", "more_queries", "token_over_many"])
def test_masked_states_have_no_part(name, p):
    c = Case(name, "bf16", seed=3, masked=0.4)
    rng = rng_state(1, 1) if p else None
    clean = c.run(p, rng)
    c.k, c.v = c.k.clone(), c.v.clone()
    hidden = c.mask == 0
    c.k[hidden] = float("nan")
    c.v[hidden] = float("inf")
    dirty = c.run(p, rng)
    for n in clean:
        assert torch.equal(clean[n], dirty[n]), n
    assert torch.all(dirty["grad_k"][hidden] == 0) and torch.all(dirty["grad_v"][hidden] == 0)


def close(a, b, kind, what):
    """The walks with care add the same products in another way: equal up to a rounding of the result."""
    assert torch.equal(a.isfinite(), b.isfinite()), what
    assert rel_l2(host(a), host(b)) <= UNIT[kind] + RTOL["f32"], what


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("name", ["prompts", "shared_heads", "past_tiles", "chunk", "dim_80", "odd_share"])
def test_later_states_have_no_part(name, kind, p, bad):
    # the last three states of the first sequence hold what must not reach the queries before them
    c = Case(name, kind, seed=4)
    rng = rng_state(1, 2) if p else None
    clean = c.run(p, rng)
    end, n = c.k_ptr[1], c.q_len[0]
    c.k, c.v = c.k.clone(), c.v.clone()
    c.v[end - 3:end, :, 1] = bad
    c.k[end - 2:end, :, 3] = bad
    dirty = c.run(p, rng)
    free = torch.ones(c.q.shape[0], dtype=torch.bool)
    free[n - 3:n] = False
    for key in ("out", "grad_q"):
        close(dirty[key][free], clean[key][free], kind, key)
        assert not dirty[key][n - 3:n].float().isfinite().all()
    other = slice(end, None)
    for key in ("grad_k", "grad_v"):
        close(dirty[key][other], clean[key][other], kind, key)


@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("name", ["prompts", "shared_heads", "past_tiles", "chunk", "dim_80", "odd_share"])
def test_earlier_rows_have_no_part_in_later_keys(name, kind, p):
    # a row whose gradient or query is not finite reaches the keys it sees, not those after it
    c = Case(name, kind, seed=5)
    rng = rng_state(3, 2) if p else None
    clean = c.run(p, rng)
    row = c.q_len[0] // 2
    last = row + c.k_len[0] - c.q_len[0]  # the last state that it sees
    c.g = c.g.clone()
    c.g[row, :, 2] = float("nan")
    dirty = c.run(p, rng)
    assert torch.equal(dirty["out"], clean["out"])
    free = torch.ones(c.q.shape[0], dtype=torch.bool)
    free[row] = False
    close(dirty["grad_q"][free], clean["grad_q"][free], kind, "grad_q")
    for key in ("grad_k", "grad_v"):
        close(dirty[key][last + 1:], clean[key][last + 1:], kind, key)
        assert not dirty[key][:last + 1].float().isfinite().all()
    c.g = Case(name, kind, seed=5).g
    c.q = c.q.clone()
    c.q[row, :, 2] = float("inf")
    dirty = c.run(p, rng)
    for key in ("out", "grad_q"):
        close(dirty[key][free], clean[key][free], kind, key)
    for key in ("grad_k", "grad_v"):
        close(dirty[key][last + 1:], clean[key][last + 1:], kind, key)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("name", ["tokens", "prompts", "chunk", "long_chunk", "shared_heads"])
def test_spare_rows_of_a_cache(name, kind):
    c = Case(name, kind, seed=6)
    want = c.run()
    spare = [7, 130, 0, 64][:len(c.k_len)]
    held = ptr([n + s for n, s in zip(c.k_len, spare)])
    k, v = (torch.full((held[-1], c.Hk, c.D), float("nan"), device="cuda").to(TYPES[kind]) for _ in range(2))
    for b, n in enumerate(c.k_len):
        k[held[b]:held[b] + n] = c.k[c.k_ptr[b]:c.k_ptr[b + 1]]
        v[held[b]:held[b] + n] = c.v[c.k_ptr[b]:c.k_ptr[b + 1]]
    out, lse = oeq.oeq_causal_attn_fwd(c.q, k, v, index(c.q_ptr), index(held), scale=c.scale, k_len=index(c.k_len))
    # other splits may be taken for longer rows, so equal up to a rounding of the result
    close(out, want["out"], kind, "out")
    assert rel_l2(host(lse), host(want["lse"])) <= RTOL["f32"]
    ref = c.reference()
    assert rel_l2(host(out), ref["out"]) <= 2 * UNIT[kind] + RTOL["f32"]


def test_lengths_of_a_cache_are_cut_to_its_rows():
    c = Case("chunk", "f32", seed=7)
    whole = c.run()
    args = (c.q, c.k, c.v, index(c.q_ptr), index(c.k_ptr))
    out, lse = oeq.oeq_causal_attn_fwd(*args, scale=c.scale, k_len=index([1 << 30, 65]))
    assert torch.equal(out, whole["out"]) and torch.equal(lse, whole["lse"])
    out, lse = oeq.oeq_causal_attn_fwd(*args, scale=c.scale, k_len=index([0, -5]))
    assert torch.all(out == 0) and torch.all(lse == -float("inf"))


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("name", ["prompts", "long", "long_chunk", "shared_heads"])
def test_repeats_bitwise_and_gradients_alone(name, kind):
    c = Case(name, kind, seed=8)
    first, again = c.run(), c.run()
    for n in first:
        assert torch.equal(first[n], again[n]), n
    for need in (("q",), ("k",), ("v",)):
        alone = c.run(need=need)
        for n in ("q", "k", "v"):
            if n in need:
                assert torch.equal(alone["grad_" + n], first["grad_" + n])
            else:
                assert alone["grad_" + n] is None


@pytest.mark.parametrize("kind", list(TYPES))
def test_a_single_token_equals_the_cross_attention(kind):
    c = Case("token_over_many", kind, seed=9)
    got = c.run()
    out, lse = oeq.oeq_cross_attn_fwd(c.q, c.k, c.v, index(c.q_ptr), index(c.k_ptr), scale=c.scale)
    close(got["out"], out, kind, "out")
    assert rel_l2(host(got["lse"]), host(lse)) <= RTOL["f32"]


@pytest.mark.parametrize("kind", list(TYPES))
def test_one_fused_projection(kind):
    # q, k and v as views of one tensor, one row pointer for both sides
    r = np.random.default_rng(10)
    qkv = torch.from_numpy(r.normal(size=(170, 8, 64))).to("cuda", TYPES[kind])
    p = index([0, 100, 170])
    views = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    out, lse = oeq.oeq_causal_attn_fwd(*views, p, p)
    dense = oeq.oeq_causal_attn_fwd(*(t.contiguous() for t in views), p, p)
    assert torch.equal(out, dense[0]) and torch.equal(lse, dense[1])
    g = torch.from_numpy(r.normal(size=(170, 4, 64))).to("cuda", TYPES[kind])
    a = oeq.oeq_causal_attn_bwd(*views, p, p, out, lse, g)
    b = oeq.oeq_causal_attn_bwd(*(t.contiguous() for t in views), p, p, out, lse, g)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("kind", list(TYPES))
def test_rows_that_no_sequence_holds_are_left_alone(kind):
    c = Case("prompts", kind, seed=11)
    want = c.run()
    n = c.q.shape[0]
    pad = lambda t: torch.cat([t[:0].new_full((5, *t.shape[1:]), 3.0), t, t.new_full((40, *t.shape[1:]), 3.0)])  # noqa: E731
    q, k, v, g = (pad(t) for t in (c.q, c.k, c.v, c.g))
    p = index([a + 5 for a in c.q_ptr])
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    oeq.oeq_causal_attn_fwd(q, k, v, p, p, scale=c.scale, out=out, lse=lse)
    grads = tuple(torch.full_like(t, 7.0) for t in (q, k, k))
    oeq.oeq_causal_attn_bwd(q, k, v, p, p, out, lse, g, scale=c.scale, grads=grads)
    for got, ref in zip((out, lse, *grads), (want[x] for x in ("out", "lse", "grad_q", "grad_k", "grad_v"))):
        assert torch.all(got[:5] == 7) and torch.all(got[n + 5:] == 7)
        close(got[5:n + 5], ref, kind, "rows")


@pytest.mark.parametrize("kind", list(TYPES))
def test_on_a_side_stream_and_in_a_graph(kind):
    c = Case("long_chunk", kind, seed=12)
    qp, kp = index(c.q_ptr), index(c.k_ptr)

    def step():
        out, lse = oeq.oeq_causal_attn_fwd(c.q, c.k, c.v, qp, kp)
        return (out, lse, *oeq.oeq_causal_attn_bwd(c.q, c.k, c.v, qp, kp, out, lse, c.g))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(3):
        other = Case("long_chunk", kind, seed=20 + seed)
        c.q.copy_(other.q)
        c.k.copy_(other.k)
        c.g.copy_(other.g)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("q_len,k_len", [([40, 7], [90, 30]), ([3], [5000]), ([1500], [1500])])
def test_in_the_callers_workspace(q_len, k_len, kind):
    r = np.random.default_rng(2)
    q, g = (torch.from_numpy(r.normal(size=(sum(q_len), 4, 32))).to("cuda", kind) for _ in range(2))
    k, v = (torch.from_numpy(r.normal(size=(sum(k_len), 2, 32))).to("cuda", kind) for _ in range(2))
    args = (q, k, v, index(ptr(q_len)), index(ptr(k_len)))
    sizes = oeq.oeq_causal_attn_workspace_size(q.shape, k.shape, len(q_len), kind)
    wholes = [torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes]
    want = oeq.oeq_causal_attn_fwd(*args)
    got = oeq.oeq_causal_attn_fwd(*args, workspace=wholes[0][:sizes[0]])
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    wants = oeq.oeq_causal_attn_bwd(*args, *want, g)
    gots = oeq.oeq_causal_attn_bwd(*args, *want, g, workspace=wholes[1][:sizes[1]])
    assert all(torch.equal(a, b) for a, b in zip(wants, gots))
    for n, whole in zip(sizes, wholes):
        assert torch.all(whole[n:] == 0x5A)


@pytest.mark.parametrize("size", [1e-4, 1e4])
@pytest.mark.parametrize("name", ["prompts", "long", "shared_heads"])
def test_fp16_gradients_of_other_sizes(name, size):
    # score gradients that leave fp16's range at either end
    c = Case(name, "f16", seed=13)
    c.g = (c.g.float() * size).half()
    got, ref = c.run(), c.reference()
    for key in ("grad_q", "grad_k", "grad_v"):
        a, b = host(got[key]), ref[key]
        # a result past 65504 has no finite fp16 value: it rounds to infinity from 65520 on (of sums of 1e4 x
        # |v| some are), where an error of 2 u = 64 may decide
        big = np.abs(b) > 65504 + 128
        assert np.array_equal(a[big], np.sign(b[big]) * np.inf)
        near = ~big & (np.abs(b) > 65504 - 128)
        a, b = a[~big & ~near], b[~big & ~near]
        # results below fp16's normal numbers are multiples of 2^-24
        assert np.linalg.norm(a - b) <= (2 * UNIT["f16"] + 1e-5) * np.linalg.norm(b) + 2.0 ** -25 * math.sqrt(a.size)


def test_fp16_gradients_of_rows_that_differ_widely():
    # a walk meets rows a million times larger than those its scale was taken from
    c = Case("long", "f16", seed=14)
    c.g = c.g.float()
    c.g[:350] *= 1e-4
    c.g[350:] *= 100.0
    c.g = c.g.half()
    got, ref = c.run(), c.reference()
    for key in ("grad_q", "grad_k", "grad_v"):
        assert rel_l2(host(got[key]), ref[key]) <= 2 * UNIT["f16"] + RTOL["f32"], key


def test_gradients_are_differences_of_the_forward():
    c = Case("shared_heads", "f32", seed=15)
    got = c.run()
    qp, kp = index(c.q_ptr), index(c.k_ptr)

    def value(q, k, v):
        return float((oeq.oeq_causal_attn_fwd(q, k, v, qp, kp, scale=c.scale)[0].double() * c.g.double()).sum())

    args = [c.q, c.k.contiguous(), c.v.contiguous()]
    for i, name in enumerate(("grad_q", "grad_k", "grad_v")):
        d = torch.randn_like(args[i])
        d /= d.norm()
        # truncation of order 1e-4 of the gradient, rounding 10^4 x 2^-23 / 2e-2
        ends = [value(*(t + s * d if j == i else t for j, t in enumerate(args))) for s in (1e-2, -1e-2)]
        change = (ends[0] - ends[1]) / 2e-2
        assert abs(change - float((got[name].double() * d.double()).sum())) <= 1e-2 * float(got[name].norm()) + 6e-2


@pytest.mark.parametrize("q_ptr,k_ptr", [([0, 90, 20, 130], [0, 90, 20, 130]), ([0, 400, 130], [0, -5, 130]),
                                         ([0, 1 << 30, 1 << 30], [0, 64, 130]), ([130, 130, 0], [0, 0, 130])])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_row_pointers_that_are_not_row_pointers_stay_in_the_tensors(kind, q_ptr, k_ptr):
    # the results mean nothing, but guard rows around every tensor stay as they are and the calls end
    whole = torch.full((5, 330, 2, 32), 0.5, device="cuda").to(TYPES[kind])
    q, k, v, g, out = (t[100:230] for t in whole)
    grads = tuple(torch.full((330, 2, 32), 0.5, device="cuda").to(TYPES[kind]) for _ in range(3))
    lse = torch.full((330, 2), 0.5, device="cuda")
    args = (q, k, v, index(q_ptr), index(k_ptr))
    oeq.oeq_causal_attn_fwd(*args, out=out, lse=lse[100:230])
    oeq.oeq_causal_attn_bwd(*args, out, lse[100:230], g, grads=tuple(t[100:230] for t in grads))
    torch.cuda.synchronize()
    for t in (*whole, *grads, lse):
        assert torch.all(t[:100] == 0.5) and torch.all(t[230:] == 0.5)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_a_cache_past_32_bit_offsets(kind):
    # 2.2 G elements of keys; the second sequence stands at their end
    n, used = (1 << 32) // (2 * 512) + 70000, 300
    k, v = (torch.zeros((n, 4, 128), dtype=TYPES[kind], device="cuda") for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(TYPES[kind])  # noqa: E731
    k[n - 400:n - 100], v[n - 400:n - 100] = rand(used, 4, 128), rand(used, 4, 128)
    v[n - 100:] = float("nan")  # spare rows
    q = rand(5, 8, 128)
    out, lse = oeq.oeq_causal_attn_fwd(q, k, v, index([0, 2, 5]), index([0, n - 400, n]), k_len=index([7, used]))
    small = oeq.oeq_causal_attn_fwd(q[2:], k[n - 400:n - 100].clone(), v[n - 400:n - 100].clone(), index([0, 3]),
                                    index([0, used]))
    close(out[2:], small[0], kind, "out")
    assert rel_l2(host(lse[2:]), host(small[1])) <= RTOL["f32"]
    assert torch.all(out[:2] == 0)  # of seven states of zeros


def test_what_the_binding_refuses():
    c = Case("chunk", "f32")
    args = (c.q, c.k, c.v, index(c.q_ptr), index(c.k_ptr))
    for bad in (torch.tensor([1, 2]).cuda(), index([1, 2]).cpu()):
        with pytest.raises(TypeError):
            oeq.oeq_causal_attn_fwd(*args, k_len=bad)
    with pytest.raises(ValueError):
        oeq.oeq_causal_attn_fwd(*args, k_len=index([1, 2, 3]))
    with pytest.raises(ValueError):
        oeq.oeq_causal_attn_fwd(c.q, c.k, c.v, index(c.q_ptr), index([0, 5]))
    with pytest.raises(TypeError):
        oeq.oeq_causal_attn_fwd(c.q, c.k.half(), c.v, index(c.q_ptr), index(c.k_ptr))
    with pytest.raises(oeq.OeqError):
        oeq.oeq_causal_attn_fwd(*args, p_drop=0.1)
