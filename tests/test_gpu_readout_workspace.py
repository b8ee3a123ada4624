"""A caller's own workspace: of the size that the size query gives, the results are those without it and
nothing past it is written; what no kernel may be given is refused."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
oeq = pytest.importorskip("cg_tensor_product_amd")


def index(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def guarded(nbytes):
    """(workspace of nbytes, the whole buffer): a pattern lies past its end"""
    whole = torch.full((nbytes + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    return whole[:nbytes], whole


@pytest.mark.parametrize("ptr,channels,groups", [([0, 100, 230], 40, 4), ([0, 3, 5000], 48, 6)])
def test_group_norm_in_the_callers_workspace(ptr, channels, groups):
    r = np.random.default_rng(1)
    x, g = (torch.from_numpy(r.normal(size=(ptr[-1], channels))).float().cuda() for _ in range(2))
    p = index(ptr)
    sizes = oeq.oeq_group_norm_workspace_size(ptr[-1], len(ptr) - 1, channels, groups)
    spaces = [guarded(n) for n in sizes]
    want = oeq.oeq_group_norm_fwd(x, p, groups, act="silu")
    got = oeq.oeq_group_norm_fwd(x, p, groups, act="silu", workspace=spaces[0][0])
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    wants = oeq.oeq_group_norm_bwd(x, p, groups, *want[1:], g, act="silu")
    gots = oeq.oeq_group_norm_bwd(x, p, groups, *want[1:], g, act="silu", workspace=spaces[1][0])
    assert all(torch.equal(a, b) for a, b in zip(wants, gots))
    for n, (_, whole) in zip(sizes, spaces):
        assert torch.all(whole[n:] == 0x5A)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("q_len,k_len", [([40, 7], [9, 30]), ([3], [5000]), ([1500], [40])])
def test_cross_attn_in_the_callers_workspace(q_len, k_len, kind):
    r = np.random.default_rng(2)
    q, g = (torch.from_numpy(r.normal(size=(sum(q_len), 4, 32))).to("cuda", kind) for _ in range(2))
    k, v = (torch.from_numpy(r.normal(size=(sum(k_len), 2, 32))).to("cuda", kind) for _ in range(2))
    args = (q, k, v, index([0, *np.cumsum(q_len).tolist()]), index([0, *np.cumsum(k_len).tolist()]))
    sizes = oeq.oeq_cross_attn_workspace_size(q.shape, k.shape, len(q_len), kind)
    spaces = [guarded(n) for n in sizes]
    want = oeq.oeq_cross_attn_fwd(*args)
    got = oeq.oeq_cross_attn_fwd(*args, workspace=spaces[0][0])
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    wants = oeq.oeq_cross_attn_bwd(*args, *want, g)
    grads = tuple(torch.full_like(t, 7.0) for t in (q, k, k))
    gots = oeq.oeq_cross_attn_bwd(*args, *want, g, grads=grads, workspace=spaces[1][0])
    assert all(a is b for a, b in zip(grads, gots)) and all(torch.equal(a, b) for a, b in zip(wants, gots))
    for n, (_, whole) in zip(sizes, spaces):
        assert torch.all(whole[n:] == 0x5A)


def test_workspaces_that_are_refused():
    x, p = torch.ones((5000, 8), device="cuda"), index([0, 5000])
    need = oeq.oeq_group_norm_workspace_size(5000, 1, 8, 2)[0]
    with pytest.raises(TypeError):
        oeq.oeq_group_norm_fwd(x, p, 2, workspace=torch.empty(need, dtype=torch.uint8))  # on the host
    byte = torch.empty(1, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError):
        oeq.oeq_group_norm_fwd(x, p, 2, workspace=byte.expand(need))  # one byte, seen `need` times
    with pytest.raises(oeq.OeqError) as e:  # not 256-byte aligned
        oeq.oeq_group_norm_fwd(x, p, 2, workspace=torch.empty(need + 8, dtype=torch.uint8, device="cuda")[8:])
    assert e.value.status == 3
