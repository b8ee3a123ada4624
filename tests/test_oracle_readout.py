"""Pins of the readout oracle: the generator's published answers, closed forms, and every
gradient against central differences."""
import numpy as np
import pytest

from oracle import readout

# Known answers of Philox4x32-10 (distributed with the generator's paper): counter, key, words
KNOWN = [
    ([0, 0, 0, 0], [0, 0], [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
]


@pytest.mark.parametrize("counter,key,words", KNOWN)
def test_philox_known_answers(counter, key, words):
    got = readout.philox4x32([np.array([c]) for c in counter], key)
    assert [int(w[0]) for w in got] == words


def test_dropout_factors_definition():
    seed, offset, p = (0x299F31D0 << 32) | 0xA4093822, (0x03707344 << 32) | 0x13198A2E, 0.3
    f = readout.dropout_factors(seed, offset, p, [0x85A308D3], 13)
    t = readout.drop_threshold(p)
    # columns 8..12 are block 1, whose words come from counter word 0 = 1
    words = readout.philox4x32([np.array([1]), np.array([0x85A308D3]), np.array([0x13198A2E]), np.array([0x03707344])],
                               [0xA4093822, 0x299F31D0])
    parts = [int(w[0]) >> s & 0xFFFF for w in words for s in (0, 16)]
    assert f.shape == (1, 13)
    assert np.array_equal(f[0, 8:] != 0, np.array(parts[:5]) >= t)
    assert set(np.unique(f)) <= {0.0, 65536.0 / (65536 - t)}


def test_dropout_factors_share_and_mean():
    f = readout.dropout_factors(7, 0, 0.25, np.arange(400), 1000)
    assert abs((f == 0).mean() - 0.25) < 4 * np.sqrt(0.25 * 0.75 / f.size)
    assert abs(f.mean() - 1) < 4 * np.sqrt(0.25 / 0.75 / f.size)
    assert np.all(readout.dropout_factors(7, 0, 0.0, np.arange(3), 20) == 1.0)


def _differences(f, x, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + eps
        hi = f()
        x[i] = keep - eps
        lo = f()
        x[i] = keep
        g[i] = (hi - lo) / (2 * eps)
    return g


@pytest.mark.parametrize("act", ["none", "silu"])
def test_group_norm_gradients_are_differences(act):
    r = np.random.default_rng(3)
    x, g = r.normal(1.0, 2.0, (9, 6)), r.normal(size=(9, 6))
    w, b = r.normal(size=6), r.normal(size=6)
    ptr = [0, 4, 4, 9]
    got = readout.group_norm(x, ptr, 2, w, b, act=act, grad_out=g)

    def loss():
        return (readout.group_norm(x, ptr, 2, w, b, act=act)["out"] * g).sum()

    for name, t in (("grad_x", x), ("grad_weight", w), ("grad_bias", b)):
        assert np.abs(got[name] - _differences(loss, t)).max() < 1e-7, name


def test_group_norm_normalises():
    r = np.random.default_rng(4)
    x = r.normal(50.0, 3.0, (40, 8))
    got = readout.group_norm(x, [0, 40, 40], 4, eps=1e-12)
    y = got["out"].reshape(40, 4, 2)
    assert np.abs(y.mean((0, 2))).max() < 1e-12
    assert np.abs(y.var((0, 2)) - 1).max() < 1e-9
    assert np.all(got["mean"][1] == 0) and np.all(got["rstd"][1] == 0)


@pytest.mark.parametrize("p", [0.0, 0.3])
def test_cross_attn_gradients_are_differences(p):
    r = np.random.default_rng(5)
    q_ptr, k_ptr = [0, 2, 2, 5], [0, 4, 5, 9]
    q, k, v = r.normal(size=(5, 4, 3)), r.normal(size=(9, 2, 3)), r.normal(size=(9, 2, 3))
    g = r.normal(size=q.shape)
    mask = np.array([1, 0, 1, 1, 1, 0, 1, 1, 1])
    kw = dict(scale=0.7, key_mask=mask, p_drop=p, rng=(11, 5))
    got = readout.cross_attn(q, k, v, q_ptr, k_ptr, grad_out=g, **kw)

    def loss():
        return (readout.cross_attn(q, k, v, q_ptr, k_ptr, **kw)["out"] * g).sum()

    for name, t in (("grad_q", q), ("grad_k", k), ("grad_v", v)):
        assert np.abs(got[name] - _differences(loss, t)).max() < 1e-7, name


def test_cross_attn_rows_that_see_nothing():
    r = np.random.default_rng(6)
    q, k = r.normal(size=(3, 1, 4)), r.normal(size=(4, 1, 4))
    k[2] = np.nan  # never read
    got = readout.cross_attn(q, k, k, [0, 1, 2, 3], [0, 0, 2, 4], 1.0, key_mask=[1, 1, 0, 0], grad_out=q)
    assert np.all(got["out"][[0, 2]] == 0) and np.all(got["lse"][[0, 2]] == -np.inf)
    assert all(np.isfinite(got[n]).all() for n in ("out", "grad_q", "grad_k", "grad_v"))
    assert np.all(got["grad_q"][[0, 2]] == 0) and np.all(got["grad_k"][2:] == 0)


def test_cross_attn_uniform_scores():
    v = np.arange(12.0).reshape(4, 1, 3)
    got = readout.cross_attn(np.zeros((2, 2, 3)), np.ones((4, 1, 3)), v, [0, 2], [0, 4], 1.0)
    assert np.allclose(got["out"], v.mean(0), atol=1e-14)
    assert np.allclose(got["lse"], np.log(4.0), atol=1e-14)
