"""Group norm on the GPU where a structure's values are far apart or all the same, against the
fp64 oracle; bounds as for the operator's other tests."""
import numpy as np
import pytest

from helpers import RTOL, rel_l2
from oracle import readout

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
oeq = pytest.importorskip("cg_tensor_product_amd")


def host(t):
    return t.detach().double().cpu().numpy()


def index(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# row pointer, channels, groups: one structure that holds nearly all rows (one part, since the average
# is short), tiles of 64 and 512 rows, wide groups, parts of a few rows a thread
OUTLIERS = {
    "one_part": ([0, 7937, *range(7938, 8001)], 16, 2),
    "one_part_wide": ([0, 7937, *range(7938, 8001)], 200, 1),
    "one_part_widest": ([0, 900, *range(901, 910)], 2048, 1),
    "short": ([0, 90, 180], 24, 3),
    "tiles_of_64": ([0, 900, 1500], 24, 3),
    "tiles_of_512": ([0, 150000, 200000], 8, 1),
}


@pytest.mark.parametrize("where", [[0], [40], [0, 1, 2, 3], [-1]])
@pytest.mark.parametrize("name", list(OUTLIERS))
def test_group_norm_with_outliers(name, where):
    # rows a hundred deviations off, the structure's first ones among them: sums about such a row
    # would cancel in the variance.  A thread's sums of n squares carry sqrt(n) 2^-24 of their total
    # where nothing cancels, 1e-6 for the 250 rows a thread has at most: the suite's fp32 bound
    ptr, C, G = OUTLIERS[name]
    r = np.random.default_rng(3)
    a = r.normal(0, 1.5, (ptr[-1], C))
    for i in where:
        a[i if i >= 0 else ptr[1] - 1] += 150.0
    x, g = torch.from_numpy(a).float().cuda(), torch.from_numpy(r.normal(size=a.shape)).float().cuda()
    out, mean, rstd = oeq.oeq_group_norm_fwd(x, index(ptr), G, act="silu")
    gx, gw, gb = oeq.oeq_group_norm_bwd(x, index(ptr), G, mean, rstd, g, act="silu")
    ref = readout.group_norm(host(x), ptr, G, act="silu", grad_out=host(g))
    assert np.abs(host(rstd)[:1] / ref["rstd"][:1] - 1).max() <= RTOL["f32"]
    assert np.abs(host(mean)[:1] - ref["mean"][:1]).max() <= RTOL["f32"]
    assert rel_l2(host(out), ref["out"]) <= RTOL["f32"]
    assert rel_l2(host(gx), ref["grad_x"]) <= RTOL["f32"]


@pytest.mark.parametrize("rows", [120, 3000])
def test_group_norm_of_channels_with_means_of_their_own(rows):
    # one group whose channels lie 1000 apart, and rows that drift: between any two rows and any two
    # channels the values are far apart against their noise
    r = np.random.default_rng(5)
    a = r.normal(size=(rows, 16)) + 1000.0 * np.arange(16) + np.linspace(-300, 300, rows)[:, None]
    x = torch.from_numpy(a).float().cuda()
    out, mean, rstd = oeq.oeq_group_norm_fwd(x, index([0, rows]), 1)
    ref = readout.group_norm(host(x), [0, rows], 1)
    assert rel_l2(host(mean), ref["mean"]) <= RTOL["f32"]
    assert rel_l2(host(rstd), ref["rstd"]) <= RTOL["f32"]
    assert rel_l2(host(out), ref["out"]) <= RTOL["f32"]


@pytest.mark.parametrize("rows", [1, 50, 900])
@pytest.mark.parametrize("eps", [1e-5, 1e-30, 1.2e-38, 1e-40, 1e-44])
def test_group_norm_of_equal_values_with_a_tiny_eps(rows, eps):
    # no variance: rstd = 1 / sqrt(eps), finite for every fp32 eps above zero, and xhat = 0
    x = torch.full((rows, 8), 3.5, device="cuda")
    bias = torch.arange(8.0, device="cuda")
    out, mean, rstd = oeq.oeq_group_norm_fwd(x, index([0, rows]), 2, None, bias, eps=eps)
    want = 1.0 / np.sqrt(np.float64(np.float32(eps)))
    assert np.abs(host(rstd) / want - 1).max() <= RTOL["f32"]
    assert torch.all(mean == 3.5) and torch.equal(out, bias.expand_as(out))
    g = torch.from_numpy(np.random.default_rng(7).normal(size=(rows, 8))).float().cuda()
    gx, gw, gb = oeq.oeq_group_norm_bwd(x, index([0, rows]), 2, mean, rstd, g, None, bias)
    ref = readout.group_norm(host(x), [0, rows], 2, None, host(bias), eps=np.float64(np.float32(eps)), grad_out=host(g))
    assert rel_l2(host(gx), ref["grad_x"]) <= RTOL["f32"]
    assert torch.all(gw == 0) and rel_l2(host(gb), ref["grad_bias"]) <= RTOL["f32"]
