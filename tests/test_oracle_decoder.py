"""Pins of the decoder operators' oracle: against torch's autograd in fp64 and against values written
out by hand."""
import numpy as np
import pytest

from oracle import decoder, readout

torch = pytest.importorskip("torch")


def test_embedding():
    r = np.random.default_rng(0)
    table, g = torch.from_numpy(r.normal(size=(6, 3))).requires_grad_(), r.normal(size=(9, 3))
    index = np.array([0, 5, 5, -1, 2, 6, 5, 0, 1 << 40])
    got = decoder.embedding(table.detach().numpy(), index, 1.5, g)
    real = torch.from_numpy((index >= 0) & (index < 6))
    out = 1.5 * table[torch.where(real, torch.from_numpy(index), torch.tensor(0))] * real[:, None]
    out.backward(torch.from_numpy(g))
    assert np.allclose(got["out"], out.detach().numpy(), rtol=1e-14)
    assert np.allclose(got["grad_table"], table.grad.numpy(), rtol=1e-14, atol=1e-15)
    assert np.all(got["grad_table"][3:5] == 0)


def test_e4m3_values():
    v = decoder.e4m3_values()
    assert len(v) == 127 and v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[-1] == 448 and v[-2] == 416
    assert np.all(np.diff(v) > 0)
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double().numpy()
    assert np.array_equal(v, codes)


def test_to_e4m3():
    x = np.concatenate([np.linspace(-460, 460, 4001), np.random.default_rng(1).normal(size=2000) * 0.02])
    want = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).float().double().numpy()
    assert np.array_equal(decoder.to_e4m3(np.float64(np.float32(x))), want)


@pytest.mark.parametrize("weighted", [False, True])
def test_rms_norm(weighted):
    r = np.random.default_rng(2)
    h = torch.from_numpy(r.normal(size=(5, 7))).requires_grad_()
    w = torch.from_numpy(1 + 0.1 * r.normal(size=7)).requires_grad_()
    g, gs = r.normal(size=(2, 5, 7))
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-3) * (w if weighted else 1)
    ((y * torch.from_numpy(g)).sum() + (h * torch.from_numpy(gs)).sum()).backward()
    got = decoder.rms_norm(h.detach().numpy(), w.detach().numpy() if weighted else None, 1e-3, g, gs)
    assert np.allclose(got["y"], y.detach().numpy(), rtol=1e-13)
    assert np.allclose(got["grad_x"], h.grad.numpy(), rtol=1e-12, atol=1e-14)
    if weighted:
        assert np.allclose(got["grad_weight"], w.grad.numpy(), rtol=1e-12)
    assert np.allclose(got["scale"] * 448, np.abs(got["y"]).max(1))


@pytest.mark.parametrize("p_drop", [0.0, 0.3])
def test_causal_attention(p_drop):
    r = np.random.default_rng(3)
    q_ptr, k_ptr, k_len = [0, 4, 4, 9, 12], [0, 4, 6, 16, 20], [4, 2, 8, 2]
    H, Hk, D = 4, 2, 5
    q, k, v = (torch.from_numpy(r.normal(size=s)).requires_grad_() for s in ((12, H, D), (20, Hk, D), (20, Hk, D)))
    mask, g = r.random(20) > 0.3, r.normal(size=(12, H, D))
    rng = (5, 77)
    got = decoder.causal_attn(*(t.detach().numpy() for t in (q, k, v)), q_ptr, k_ptr, 0.7, mask, k_len, p_drop, rng, g)
    outs = []
    for b in range(4):
        n, m = q_ptr[b + 1] - q_ptr[b], k_len[b]
        Q = q[q_ptr[b]:q_ptr[b + 1]].transpose(0, 1)
        K, V = (t[k_ptr[b]:k_ptr[b] + m].repeat_interleave(2, 1).transpose(0, 1) for t in (k, v))
        sees = torch.ones(n, m, dtype=torch.bool).tril(m - n) & torch.from_numpy(mask[k_ptr[b]:k_ptr[b] + m])
        S = (0.7 * Q @ K.transpose(1, 2)).masked_fill(~sees, -1e300)
        P = torch.softmax(S, 2) * sees
        if p_drop:
            rows = (np.arange(q_ptr[b], q_ptr[b + 1])[None, :] * H + np.arange(H)[:, None]).ravel()
            P = P * torch.from_numpy(readout.dropout_factors(*rng, p_drop, rows, m)).view(H, n, m)
        outs.append((P @ V).transpose(0, 1))
    out = torch.cat(outs)
    out.backward(torch.from_numpy(g))
    assert np.allclose(got["out"], out.detach().numpy(), rtol=1e-12, atol=1e-13)
    for name, t in (("grad_q", q), ("grad_k", k), ("grad_v", v)):
        assert np.allclose(got[name], t.grad.numpy(), rtol=1e-11, atol=1e-12), name
    # the third sequence's queries see 4 + i of its 8 states, the last one's first query sees none of 2
    assert np.all(np.isneginf(got["lse"][9])) and np.all(got["out"][9] == 0)
