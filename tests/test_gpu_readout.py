"""The readout operators on the GPU against the fp64 oracle: group norm and dropout (cross
attention has a file of its own).

Bounds, relative L2 per output tensor against the oracle on the same (rounded) inputs: the
suite's fp32 bound of 1e-5 for fp32 arithmetic, plus one unit roundoff of the output's type
(2^-11 for fp16, 2^-8 for bf16: each element is rounded once).  Gradients to weight and bias,
means and reciprocal deviations are fp32 whatever the input's type.
"""
import numpy as np
import pytest

from helpers import RTOL, rel_l2
from oracle import readout

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
oeq = pytest.importorskip("cg_tensor_product_amd")

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def bound(kind):
    return RTOL["f32"] + UNIT[kind]


def host(t):
    return t.detach().double().cpu().numpy()


def rand(rng, shape, kind, scale=1.0, shift=0.0):
    return torch.from_numpy(rng.normal(shift, scale, shape)).to("cuda", TYPES[kind])


def index(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# group norm
# ---------------------------------------------------------------------------

# row pointer, channels, groups
GROUPS = {
    "one_value": ([0, 1], 1, 1),
    "one_row": ([0, 1], 64, 8),
    "empty_structures": ([0, 0, 5, 5, 5, 12, 12], 24, 3),
    "odd_channels": ([0, 3, 50, 57], 30, 3),
    "one_channel_groups": ([0, 17, 40], 70, 70),
    "three_channel_groups": ([0, 9, 11, 100], 51, 17),
    "wide_group": ([0, 33, 40], 130, 1),
    "widest_group": ([0, 5, 6], 2048, 1),
    "uneven_slabs": ([0, 21], 176, 11),
    "several_splits": ([0, 1500], 48, 6),
    "ragged_splits": ([0, 3, 3, 1400, 1401, 2300], 40, 4),
    "many_structures": (list(range(0, 301, 3)), 16, 2),
    "wide_group_splits": ([0, 700], 520, 2),
}


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("name", list(GROUPS))
def test_group_norm(name, act, kind):
    ptr, C, G = GROUPS[name]
    rng = np.random.default_rng(100 + len(name))
    T = ptr[-1]
    x, g = rand(rng, (T, C), kind, 1.5, 0.5), rand(rng, (T, C), kind)
    w, b = rand(rng, (C,), "f32", 0.3, 1.0), rand(rng, (C,), "f32", 0.3)
    p = index(ptr)
    out, mean, rstd = oeq.oeq_group_norm_fwd(x, p, G, w, b, act=act)
    gx, gw, gb = oeq.oeq_group_norm_bwd(x, p, G, mean, rstd, g, w, b, act=act)
    ref = readout.group_norm(host(x), ptr, G, host(w), host(b), act=act, grad_out=host(g))
    assert out.dtype == gx.dtype == x.dtype and mean.dtype == rstd.dtype == gw.dtype == gb.dtype == torch.float32
    assert rel_l2(host(mean), ref["mean"]) <= RTOL["f32"]
    assert rel_l2(host(rstd), ref["rstd"]) <= RTOL["f32"]
    assert rel_l2(host(out), ref["out"]) <= bound(kind)
    assert rel_l2(host(gb), ref["grad_bias"]) <= RTOL["f32"]
    if name != "one_value":
        assert rel_l2(host(gw), ref["grad_weight"]) <= RTOL["f32"]
        assert rel_l2(host(gx), ref["grad_x"]) <= bound(kind)
    else:  # a single value: xhat and its gradient are zero but for rounding
        assert np.abs(host(gx)).max() <= 1e-3 and np.abs(host(gw)).max() <= 1e-3


# structures cut into tiles of 64, 128, 256 and 512 rows: ends on a tile, one row past it and one
# short of it, a structure that has almost all the rows, over 64 structures, rows before the first
TILED = {
    "tiles_of_64": ([0, 64, 193, 320, 383, 1000, 1000], 24, 3),
    "tiles_of_128": ([0, 1, 129, 257, 40000], 12, 3),
    "tiles_of_256": ([0, 256, 256, 99000, 99257, 99512], 16, 2),
    "tiles_of_512": ([0, 512, 1025, 200000], 8, 1),
    "many_in_tiles": ([17 + 150 * i + (i * i) % 97 for i in range(131)], 40, 4),
}


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(TILED))
def test_group_norm_in_tiles(name, kind):
    ptr, C, G = TILED[name]
    rng = np.random.default_rng(700 + len(name))
    x, g = rand(rng, (ptr[-1], C), kind, 1.5, 0.5), rand(rng, (ptr[-1], C), kind)
    w, b = rand(rng, (C,), "f32", 0.3, 1.0), rand(rng, (C,), "f32", 0.3)
    p = index(ptr)
    out, mean, rstd = oeq.oeq_group_norm_fwd(x, p, G, w, b, act="silu")
    gx, gw, gb = oeq.oeq_group_norm_bwd(x, p, G, mean, rstd, g, w, b, act="silu")
    ref = readout.group_norm(host(x), ptr, G, host(w), host(b), act="silu", grad_out=host(g))
    rows = slice(ptr[0], ptr[-1])  # rows of no structure are not written
    assert rel_l2(host(mean), ref["mean"]) <= RTOL["f32"]
    assert rel_l2(host(rstd), ref["rstd"]) <= RTOL["f32"]
    assert rel_l2(host(out)[rows], ref["out"][rows]) <= bound(kind)
    assert rel_l2(host(gx)[rows], ref["grad_x"][rows]) <= bound(kind)
    assert rel_l2(host(gw), ref["grad_weight"]) <= RTOL["f32"]
    assert rel_l2(host(gb), ref["grad_bias"]) <= RTOL["f32"]


def test_group_norm_without_weight_and_bias():
    rng = np.random.default_rng(1)
    ptr = [0, 7, 30]
    x, g = rand(rng, (30, 32), "f32"), rand(rng, (30, 32), "f32")
    out, mean, rstd = oeq.oeq_group_norm_fwd(x, index(ptr), 4, act="silu")
    gx, gw, gb = oeq.oeq_group_norm_bwd(x, index(ptr), 4, mean, rstd, g, act="silu", need=("x",))
    assert gw is None and gb is None
    ref = readout.group_norm(host(x), ptr, 4, act="silu", grad_out=host(g))
    assert rel_l2(host(out), ref["out"]) <= RTOL["f32"]
    assert rel_l2(host(gx), ref["grad_x"]) <= RTOL["f32"]


@pytest.mark.parametrize("need", [("weight",), ("bias",), ("x", "bias"), ("weight", "bias"), ()])
@pytest.mark.parametrize("rows", [40, 900])
def test_group_norm_gradients_on_request(need, rows):
    rng = np.random.default_rng(2)
    x, g, w = rand(rng, (rows, 24), "f32"), rand(rng, (rows, 24), "f32"), rand(rng, (24,), "f32")
    p = index([0, rows])
    _, mean, rstd = oeq.oeq_group_norm_fwd(x, p, 3, w)
    every = oeq.oeq_group_norm_bwd(x, p, 3, mean, rstd, g, w)
    some = oeq.oeq_group_norm_bwd(x, p, 3, mean, rstd, g, w, need=need)
    for n, a, b in zip(("x", "weight", "bias"), every, some):
        assert (b is None) if n not in need else torch.equal(a, b)


@pytest.mark.parametrize("rows", [60, 2000])
def test_group_norm_reads_and_writes_strided_rows(rows):
    rng = np.random.default_rng(3)
    wide = rand(rng, (rows, 93), "bf16")
    x = wide[:, 5:45]  # rows neither 16-byte aligned nor a multiple of eight apart
    p, gwide = index([0, rows // 3, rows]), rand(rng, (rows, 61), "bf16")
    target = torch.full((rows, 50), 7.0, dtype=torch.bfloat16, device="cuda")
    out, mean, rstd = oeq.oeq_group_norm_fwd(x, p, 5, out=target[:, 3:43])
    dense = oeq.oeq_group_norm_fwd(x.contiguous(), p, 5)
    assert all(torch.equal(a, b) for a, b in zip((out, mean, rstd), dense))
    assert torch.all(target[:, :3] == 7) and torch.all(target[:, 43:] == 7)
    gx, _, _ = oeq.oeq_group_norm_bwd(x, p, 5, mean, rstd, gwide[:, 1:41])
    gd, _, _ = oeq.oeq_group_norm_bwd(x.contiguous(), p, 5, mean, rstd, gwide[:, 1:41].contiguous())
    assert torch.equal(gx, gd)


@pytest.mark.parametrize("rows", [100, 5000])
def test_group_norm_of_a_large_mean(rows):
    # x = 1000 + N(0, 1): each x carries a relative rounding of 2^-24, so 6e-5 of a deviation, in
    # the oracle's input too; the fp32 mean is off by at most half a unit (3e-5 of a deviation)
    rng = np.random.default_rng(4)
    x = rand(rng, (rows, 16), "f32", 1.0, 1000.0)
    out, _, rstd = oeq.oeq_group_norm_fwd(x, index([0, rows]), 2)
    ref = readout.group_norm(host(x), [0, rows], 2)
    assert rel_l2(host(rstd), ref["rstd"]) <= RTOL["f32"]
    assert rel_l2(host(out), ref["out"]) <= 6e-5


@pytest.mark.parametrize("rows", [30, 800])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_group_norm_keeps_bad_values_to_their_group(rows, bad):
    rng = np.random.default_rng(5)
    x = rand(rng, (2 * rows, 12), "f32")
    p = index([0, rows, 2 * rows])
    clean = oeq.oeq_group_norm_fwd(x, p, 3)[0]
    y = x.clone()
    y[rows + 3, 5] = bad  # second structure, second group
    got = oeq.oeq_group_norm_fwd(y, p, 3)[0]
    touched = torch.zeros_like(x, dtype=torch.bool)
    touched[rows:, 4:8] = True
    assert torch.equal(got[~touched], clean[~touched])
    assert torch.isnan(got[touched]).all()


def test_group_norm_of_nothing():
    x = torch.empty((0, 8), device="cuda")
    for ptr in ([0], [0, 0, 0]):
        B = len(ptr) - 1
        out, mean, rstd = oeq.oeq_group_norm_fwd(x, index(ptr), 2)
        assert out.shape == (0, 8) and mean.shape == (B, 2) and torch.all(mean == 0) and torch.all(rstd == 0)
        gx, gw, gb = oeq.oeq_group_norm_bwd(x, index(ptr), 2, mean, rstd, x)
        assert gx.shape == (0, 8) and torch.all(gw == 0) and torch.all(gb == 0)


def test_group_norm_is_bitwise_repeatable():
    rng = np.random.default_rng(6)
    x, g = rand(rng, (4000, 96), "f32"), rand(rng, (4000, 96), "f32")
    p = index([0, 1000, 4000])

    def once():
        out, mean, rstd = oeq.oeq_group_norm_fwd(x, p, 8, act="silu")
        return (out, mean, rstd, *oeq.oeq_group_norm_bwd(x, p, 8, mean, rstd, g, act="silu"))

    first = once()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, once()))


def test_group_norm_cuts_a_row_pointer_to_the_rows():
    x = torch.ones((10, 8), device="cuda")
    out, mean, _ = oeq.oeq_group_norm_fwd(x, index([0, 4, 1000]), 2, out=torch.zeros_like(x))
    assert torch.all(mean == 1) and torch.all(out == 0)


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------

SHAPES = [(1, 1), (1, 8), (3, 7), (5, 9), (64, 128), (17, 33), (300, 1), (2, 4001), (129, 257)]


def state(seed, offset):
    as_signed = lambda v: v - (1 << 64) if v >> 63 else v  # noqa: E731
    return torch.tensor([as_signed(seed), as_signed(offset)], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(shape, kind, residual):
    rng = np.random.default_rng(sum(shape))
    x, r = rand(rng, shape, kind), rand(rng, shape, kind) if residual else None
    seed, offset, p = 0xFEDCBA9876543210, (1 << 63) + 12345, 0.3
    out = oeq.oeq_dropout_fwd(x, p, state(seed, offset), residual=r)
    f = readout.dropout_factors(seed, offset, p, np.arange(shape[0]), shape[1])
    ref = host(x) * f + (host(r) if residual else 0.0)
    assert rel_l2(host(out), ref) <= bound(kind)
    dropped = torch.from_numpy(f == 0).cuda()
    assert torch.equal(out[dropped], (r if residual else torch.zeros_like(x))[dropped])
    g = rand(rng, shape, kind)
    gx = oeq.oeq_dropout_bwd(g, p, state(seed, offset))
    assert rel_l2(host(gx), host(g) * f) <= bound(kind)
    assert torch.all(gx[dropped] == 0)


@pytest.mark.parametrize("p", [0.0, 1e-9, 2.0 ** -16, 0.5, 0.99999, 1.0 - 2.0 ** -17])
def test_dropout_probabilities(p):
    x = torch.ones((50, 64), device="cuda")
    out = oeq.oeq_dropout_fwd(x, p, state(9, 4))
    f = readout.dropout_factors(9, 4, p, np.arange(50), 64)
    assert np.array_equal(host(out) == 0, f == 0)
    assert rel_l2(host(out), f) <= RTOL["f32"]


def test_dropout_strided_rows_and_in_place():
    rng = np.random.default_rng(8)
    wide = rand(rng, (40, 75), "f16")
    x = wide[:, 3:60]
    dense = oeq.oeq_dropout_fwd(x.contiguous(), 0.4, state(1, 2))
    target = torch.full((40, 80), 5.0, dtype=torch.float16, device="cuda")
    out = oeq.oeq_dropout_fwd(x, 0.4, state(1, 2), out=target[:, 9:66])
    assert torch.equal(out, dense)
    assert torch.all(target[:, :9] == 5) and torch.all(target[:, 66:] == 5)
    both = oeq.oeq_dropout_fwd(x.contiguous(), 0.4, state(1, 2), residual=out)
    again = oeq.oeq_dropout_fwd(x.contiguous(), 0.4, state(1, 2), residual=dense, out=dense)
    assert torch.equal(both, again) and again.data_ptr() == dense.data_ptr()


def test_dropout_drops_bad_values():
    x = torch.full((8, 64), float("nan"), device="cuda")
    out = oeq.oeq_dropout_fwd(x, 0.5, state(3, 3))
    f = readout.dropout_factors(3, 3, 0.5, np.arange(8), 64)
    assert np.array_equal(np.isnan(host(out)), f != 0)
    assert np.all(host(out)[f == 0] == 0)


def test_dropout_of_nothing():
    for shape in ((0, 8), (4, 0)):
        x = torch.empty(shape, device="cuda")
        assert oeq.oeq_dropout_fwd(x, 0.5, state(0, 0)).shape == shape
        assert oeq.oeq_dropout_bwd(x, 0.5, state(0, 0)).shape == shape


def test_offsets_past_32_bits():
    # rows 2^26 elements apart: the last of 40 is 2.6e9 elements into the buffer
    rng = np.random.default_rng(11)
    rows, stride = 40, 1 << 26
    x = torch.empty(stride * (rows - 1) + 32, dtype=torch.bfloat16, device="cuda").as_strided((rows, 32), (stride, 1))
    x.copy_(rand(rng, (rows, 32), "bf16"))
    near, p = x.contiguous(), index([0, 11, rows])
    far = oeq.oeq_group_norm_fwd(x, p, 4, act="silu")
    assert all(torch.equal(a, b) for a, b in zip(far, oeq.oeq_group_norm_fwd(near, p, 4, act="silu")))
    got = oeq.oeq_group_norm_bwd(x, p, 4, far[1], far[2], near, act="silu")
    want = oeq.oeq_group_norm_bwd(near, p, 4, far[1], far[2], near, act="silu")
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(oeq.oeq_dropout_fwd(x, 0.3, state(1, 1)), oeq.oeq_dropout_fwd(near, 0.3, state(1, 1)))


# ---------------------------------------------------------------------------
# both, as a program runs them
# ---------------------------------------------------------------------------

def test_runs_on_the_callers_stream():
    rng = np.random.default_rng(9)
    x, p = rand(rng, (3000, 64), "f32"), index([0, 3000])
    want = oeq.oeq_group_norm_fwd(x, p, 8)[0]
    drop = oeq.oeq_dropout_fwd(want, 0.2, state(5, 6))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = oeq.oeq_group_norm_fwd(x, p, 8)[0]
        got = oeq.oeq_dropout_fwd(got, 0.2, state(5, 6))
    side.synchronize()
    assert torch.equal(got, drop)


def test_replays_in_a_graph_with_an_advancing_offset():
    rng = np.random.default_rng(10)
    x, g = rand(rng, (900, 64), "f32"), rand(rng, (900, 64), "f32")
    p, key = index([0, 500, 900]), state(21, 100)

    def step():
        out, mean, rstd = oeq.oeq_group_norm_fwd(x, p, 8, act="silu")
        y = oeq.oeq_dropout_fwd(out, 0.25, key, residual=x)
        gd = oeq.oeq_dropout_bwd(g, 0.25, key)
        return (y, *oeq.oeq_group_norm_bwd(x, p, 8, mean, rstd, gd, act="silu"))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    masks = []
    for i in range(4):
        key[1] = 100 + i
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
        masks.append(got[0])
        torch.cuda.synchronize()
    assert not torch.equal(masks[0], masks[1])


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def test_group_norm_refusals():
    x, p = torch.ones((6, 8), device="cuda"), index([0, 6])
    w = torch.ones(8, device="cuda")
    for bad in (dict(n_groups=3), dict(n_groups=0), dict(eps=0.0), dict(eps=float("nan"))):
        with pytest.raises(oeq.OeqError) as e:
            oeq.oeq_group_norm_fwd(x, p, **{"n_groups": 2, **bad})
        assert e.value.status == 1
    with pytest.raises(oeq.OeqError) as e:
        oeq.oeq_group_norm_fwd(torch.ones((2, 4096), device="cuda"), index([0, 2]), 1)
    assert e.value.status == 2
    with pytest.raises(oeq.OeqError) as e:
        oeq.oeq_group_norm_fwd(x, index([0]), 2)
    assert e.value.status == 1
    for bad in (x.double(), x.cpu()):
        with pytest.raises(TypeError):
            oeq.oeq_group_norm_fwd(bad, p, 2)
    with pytest.raises(TypeError):
        oeq.oeq_group_norm_fwd(x, p.long(), 2)
    with pytest.raises(TypeError):
        oeq.oeq_group_norm_fwd(x, p, 2, weight=w.half())
    with pytest.raises(ValueError):
        oeq.oeq_group_norm_fwd(x, p, 2, weight=w[:4])
    with pytest.raises(ValueError):
        oeq.oeq_group_norm_fwd(x.t().contiguous().t(), p, 2)
    with pytest.raises(ValueError):
        oeq.oeq_group_norm_fwd(x[:1].expand(6, 8), p, 2)
    with pytest.raises(ValueError):
        oeq.oeq_group_norm_fwd(x, p, 2, act="gelu")
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    big = torch.ones((5000, 8), device="cuda")
    with pytest.raises(oeq.OeqError) as e:
        oeq.oeq_group_norm_fwd(big, index([0, 5000]), 2, workspace=small)
    assert e.value.status == 3
    _, mean, rstd = oeq.oeq_group_norm_fwd(x, p, 2)
    with pytest.raises(ValueError):
        oeq.oeq_group_norm_bwd(x, p, 2, mean, rstd, x[:, :4])
    with pytest.raises(TypeError):
        oeq.oeq_group_norm_bwd(x, p, 2, mean, rstd, x.half())
    with pytest.raises(ValueError):
        oeq.oeq_group_norm_bwd(x, p, 4, mean, rstd, x)


def test_dropout_refusals():
    x = torch.ones((6, 8), device="cuda")
    for p in (1.0, -0.1, float("nan"), 2.0):
        with pytest.raises(oeq.OeqError) as e:
            oeq.oeq_dropout_fwd(x, p, state(0, 0))
        assert e.value.status == 1
    with pytest.raises(TypeError):
        oeq.oeq_dropout_fwd(x, 0.1, torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError):
        oeq.oeq_dropout_fwd(x, 0.1, torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        oeq.oeq_dropout_fwd(x.double(), 0.1, state(0, 0))
    with pytest.raises(ValueError):
        oeq.oeq_dropout_fwd(x, 0.1, state(0, 0), residual=x[:3])
    with pytest.raises(ValueError):
        oeq.oeq_dropout_fwd(x[0], 0.1, state(0, 0))
    with pytest.raises(ValueError):
        oeq.oeq_dropout_bwd(x[:1].expand(6, 8), 0.1, state(0, 0))
