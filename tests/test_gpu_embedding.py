"""Embedding lookup and its gradient on the GPU against the fp64 oracle.

out is one fp32 product rounded once: exact for scale 1, else within u = eps / 2 of the type and
2^-24 of the product, relative to each element.  grad_table is an fp64 sum (an index's runs within
chunks of the sorted list rounded once to fp32, where a run is cut), times the scale, rounded to
fp32 and to the type: each element is within u + 2^-22 of the sum of its terms' magnitudes.
"""
import numpy as np
import pytest

from oracle import decoder

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
oeq = pytest.importorskip("cg_tensor_product_amd")

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

# table rows, columns, rows, skew of the index, share of absent indices
CASES = {
    "one": (1, 1, 1, 1.0, 0.0),
    "molecule": (89, 128, 56, 2.0, 0.0),
    "odd_columns": (7, 13, 300, 1.0, 0.1),
    "no_rows": (5, 24, 0, 1.0, 0.0),
    "no_rows_of_a_long_table": (300, 24, 0, 1.0, 0.0),
    "all_absent_of_a_long_table": (300, 24, 5000, 1.0, 1.0),
    "all_absent": (6, 16, 40, 1.0, 1.0),
    "one_row_table": (1, 40, 1000, 1.0, 0.0),
    "one_sorting_group": (700, 72, 4096, 2.0, 0.05),
    "past_four_a_thread": (255, 33, 4097, 1.0, 0.05),
    "most_of_one_group": (3000, 16, 16384, 2.0, 0.05),
    "past_one_group": (255, 33, 16385, 1.0, 0.05),
    "past_one_group_two_digits": (256, 9, 20000, 1.0, 0.05),
    "two_digits": (256, 8, 5000, 3.0, 0.0),
    "vocabulary": (32000, 520, 6000, 4.0, 0.05),
    "three_digits": (100000, 5, 9000, 3.0, 0.0),
    "few_common": (10, 256, 30000, 1.5, 0.0),
    "most_of_a_small_table": (16, 100, 2000, 1.0, 0.1),
    "next_small_table": (17, 100, 2000, 1.0, 0.1),
    "last_small_table": (32, 256, 900, 1.0, 0.1),
    "past_a_small_table": (33, 100, 2000, 1.0, 0.1),
    "small_table_of_wide_rows": (20, 264, 500, 1.0, 0.1),
    "small_table_wide": (6, 1100, 700, 2.0, 0.05),
    "counted_passes": (40, 16, 300000, 2.0, 0.01),
    "counted_two_digits": (1000, 8, 70000, 3.0, 0.01),
    "long": (3, 16, 300000, 1.0, 0.01),
    "wide": (50, 2051, 333, 1.0, 0.0),
}


def make(name, kind, index_type=torch.int64, seed=0):
    table, cols, rows, skew, absent = CASES[name]
    r = np.random.default_rng(seed + len(name))
    index = np.minimum((table * r.random(rows) ** skew).astype(np.int64), table - 1)
    index[r.random(rows) < absent] = -1
    t, g = (torch.from_numpy(r.normal(size=(n, cols))).to("cuda", TYPES[kind]) for n in (table, rows))
    return t, torch.from_numpy(index).to("cuda", index_type), g


def host(t):
    return t.detach().double().cpu().numpy()


def check_gradient(got, index, g, n_table, scale, kind):
    index = index.cpu().numpy()
    used = (index >= 0) & (index < n_table)
    want, size = np.zeros((2, n_table, g.shape[1]))
    np.add.at(want, index[used], scale * host(g)[used])
    np.add.at(size, index[used], np.abs(scale * host(g)[used]))
    bound = (torch.finfo(TYPES[kind]).eps / 2 + 2.0 ** -22) * size
    # fp16 rounds to multiples of 2^-24 near zero
    assert np.all(np.abs(host(got) - want) <= bound + (2.0 ** -25 if kind == "f16" else 0.0))


@pytest.mark.parametrize("index_type", [torch.int32, torch.int64])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("name", list(CASES))
def test_embedding(name, kind, index_type):
    table, index, g = make(name, kind, index_type)
    out = oeq.oeq_embedding_fwd(table, index)
    at = index.long().clamp(min=0)
    assert torch.equal(out, torch.where((index >= 0)[:, None], table[at], torch.zeros_like(table[:1])))
    for scale in (1.0, 11.3):
        got = oeq.oeq_embedding_bwd(index, g, table.shape[0], scale=scale)
        assert got.dtype == TYPES[kind] and got.shape == table.shape
        check_gradient(got, index, g, table.shape[0], float(np.float32(scale)), kind)
        # bitwise the same again
        assert torch.equal(got, oeq.oeq_embedding_bwd(index, g, table.shape[0], scale=scale))


@pytest.mark.parametrize("kind", list(TYPES))
def test_scaled_lookup_equals_the_oracle(kind):
    table, index, _ = make("odd_columns", kind)
    got = host(oeq.oeq_embedding_fwd(table, index, scale=3.7))
    want = decoder.embedding(host(table), index.cpu().numpy(), float(np.float32(3.7)))["out"]
    assert np.all(np.abs(got - want) <= (torch.finfo(TYPES[kind]).eps / 2 + 2.0 ** -23) * np.abs(want) + 2.0 ** -24)


def test_gradient_equals_the_oracle_and_differences():
    table, index, g = make("odd_columns", "f32")
    want = decoder.embedding(host(table), index.cpu().numpy(), 2.0, host(g))["grad_table"]
    got = oeq.oeq_embedding_bwd(index, g, table.shape[0], scale=2.0)
    assert np.allclose(host(got), want, rtol=0, atol=2.0 ** -20 * np.abs(want).max())
    # the lookup is linear in the table: a step of one in a direction is the gradient's component
    step = torch.randn_like(table)
    moved = oeq.oeq_embedding_fwd(table + step, index, scale=2.0).double() - oeq.oeq_embedding_fwd(table, index, scale=2.0)
    change = float((moved * g.double()).sum())
    # 300 rows x 13 sums of products of size 10, each element of the lookups 2^-22 off
    assert abs(change - float((got.double() * step.double()).sum())) <= 300 * 13 * 10 * 2.0 ** -22


@pytest.mark.parametrize("far", [7, 8, 1 << 20, -1, -(1 << 31), (1 << 31) - 1])
@pytest.mark.parametrize("index_type", [torch.int32, torch.int64])
def test_indices_outside_the_table(index_type, far):
    table = torch.randn(7, 24, device="cuda")
    index = torch.tensor([0, far, 6, far, 0], dtype=index_type, device="cuda")
    g = torch.randn(5, 24, device="cuda")
    out = oeq.oeq_embedding_fwd(table, index)
    assert torch.equal(out[[0, 2, 4]], table[[0, 6, 0]]) and torch.all(out[[1, 3]] == 0)
    got = oeq.oeq_embedding_bwd(index, g, 7)
    assert torch.all(got[1:6] == 0)
    check_gradient(got, index, g, 7, 1.0, "f32")
    if index_type is torch.int64:
        index[1] = (1 << 32) + 3  # not row 3
        assert torch.all(oeq.oeq_embedding_fwd(table, index)[1] == 0)


def test_absent_rows_take_no_gradient_whatever_they_hold():
    table, index, g = make("odd_columns", "bf16")
    clean = oeq.oeq_embedding_bwd(index, g, 7)
    g[index < 0] = float("nan")
    assert torch.equal(clean, oeq.oeq_embedding_bwd(index, g, 7))


@pytest.mark.parametrize("kind", list(TYPES))
def test_strided_operands(kind):
    table, index, g = make("odd_columns", kind)
    wide = torch.randn(7, 40, device="cuda").to(TYPES[kind])
    wide[:, 3:16] = table
    rows = torch.full((300, 31), 7.0, device="cuda").to(TYPES[kind])
    out = oeq.oeq_embedding_fwd(wide[:, 3:16], index, out=rows[:, 5:18])
    assert torch.equal(out, oeq.oeq_embedding_fwd(table, index))
    assert torch.all(rows[:, :5] == 7) and torch.all(rows[:, 18:] == 7)
    gs = torch.full((300, 29), 9.0, device="cuda").to(TYPES[kind])
    gs[:, 1:14] = g
    to = torch.full((7, 20), 7.0, device="cuda").to(TYPES[kind])
    oeq.oeq_embedding_bwd(index, gs[:, 1:14], 7, out=to[:, 2:15])
    assert torch.equal(to[:, 2:15], oeq.oeq_embedding_bwd(index, g, 7))
    assert torch.all(to[:, :2] == 7) and torch.all(to[:, 15:] == 7)


def test_on_a_side_stream_and_in_a_graph():
    table, index, g = make("past_one_group", "bf16")
    want = oeq.oeq_embedding_fwd(table, index), oeq.oeq_embedding_bwd(index, g, table.shape[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = oeq.oeq_embedding_fwd(table, index), oeq.oeq_embedding_bwd(index, g, table.shape[0])
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = oeq.oeq_embedding_fwd(table, index), oeq.oeq_embedding_bwd(index, g, table.shape[0])
    for seed in range(3):
        _, other, more = make("past_one_group", "bf16", seed=seed + 5)
        index.copy_(other)
        g.copy_(more)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], oeq.oeq_embedding_fwd(table, index))
        assert torch.equal(got[1], oeq.oeq_embedding_bwd(index, g, table.shape[0]))


@pytest.mark.parametrize("name", ["molecule", "past_one_group", "vocabulary", "few_common"])
def test_in_the_callers_workspace(name):
    table, index, g = make(name, "f32")
    n = oeq.oeq_embedding_workspace_size(table.shape[0], table.shape[1], index.shape[0])
    whole = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    got = oeq.oeq_embedding_bwd(index, g, table.shape[0], workspace=whole[:n])
    assert torch.equal(got, oeq.oeq_embedding_bwd(index, g, table.shape[0]))
    assert torch.all(whole[n:] == 0x5A)
    if n:
        with pytest.raises(oeq.OeqError):
            oeq.oeq_embedding_bwd(index, g, table.shape[0], workspace=whole[:n - 256])


def test_a_table_past_32_bit_offsets():
    # 2^21 + 3 rows of 1032 fp16 columns: 2.2 G elements
    n, cols = (1 << 21) + 3, 1032
    table = torch.zeros(n, cols, dtype=torch.float16, device="cuda")
    table[-1] = 3.0
    table[-2] = 2.0
    index = torch.tensor([n - 1, 0, n - 2, n - 1], device="cuda")
    out = oeq.oeq_embedding_fwd(table, index)
    assert out[:, 0].tolist() == [3.0, 0.0, 2.0, 3.0] and out[:, -1].tolist() == [3.0, 0.0, 2.0, 3.0]
    grad = oeq.oeq_embedding_bwd(index, out, n, out=table)
    assert grad[-3:, 5].tolist() == [0.0, 2.0, 6.0] and float(grad[:-2].abs().max()) == 0.0


def test_what_the_binding_refuses():
    table, index, g = make("odd_columns", "f32")
    for bad in (index.float(), index.cpu(), "x"):
        with pytest.raises(TypeError):
            oeq.oeq_embedding_fwd(table, bad)
    with pytest.raises(ValueError):
        oeq.oeq_embedding_fwd(table, index[::2])
    with pytest.raises(ValueError):
        oeq.oeq_embedding_bwd(index[:-1], g, 7)
    with pytest.raises(TypeError):
        oeq.oeq_embedding_fwd(table.double(), index)
    with pytest.raises(ValueError):
        oeq.oeq_embedding_fwd(table.t(), index)
    with pytest.raises(ValueError):
        oeq.oeq_embedding_bwd(index, g, 7, out=torch.empty(8, 13, device="cuda"))
