"""Root-mean-square norm with the residual's addition on the GPU against the fp64 oracle.

With u = eps / 2 of the type: `sum` is the sum rounded once (exactly torch's); rstd is an fp32 value of
an fp32 sum of C squares, within (log2 C + 16) 2^-24 (pairs of eight-column pieces); y is three more
roundings in fp32 and one to the type: u + 2^-18 relative to each element.  grad_x is checked
relative to the row's largest magnitude of its terms: u + 2^-16; grad_weight relative to the sum of its
terms' magnitudes: 2^-18.  e4m3 rounds y / scale by at most 2^-4 of it (2^-10 below the normal numbers).
"""
import numpy as np
import pytest

from oracle import decoder

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
oeq = pytest.importorskip("cg_tensor_product_amd")

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = [(1, 1), (3, 7), (56, 64), (33, 100), (5, 128), (1000, 129), (16, 1024), (77, 520), (9, 2048), (4, 2049), (7, 4099),
         (3, 8200), (2, 16384), (2500, 72)]


def host(t):
    return t.detach().double().cpu().numpy()


def make(rows, cols, kind, seed=0, residual=True):
    r = np.random.default_rng(seed + rows + cols)
    rand = lambda *s, by=1.0: torch.from_numpy(r.normal(size=s) * by)  # noqa: E731
    x, res, g, gs = (rand(rows, cols, by=b).to("cuda", TYPES[kind]) for b in (1.0, 2.0, 1.0, 0.5))
    w = (1 + rand(cols, by=0.2)).float().cuda()
    return (x, res if residual else None, w, g, gs if residual else None)


def check_forward(y, rstd, total, w, kind, eps=1e-5):
    ref = decoder.rms_norm(host(total), None if w is None else host(w), eps)
    assert np.all(np.abs(host(rstd) - ref["rstd"]) <= 2.0 ** -18 * ref["rstd"])
    u = torch.finfo(TYPES[kind]).eps / 2
    tiny = 2.0 ** -25 if kind == "f16" else 0.0
    assert np.all(np.abs(host(y) - ref["y"]) <= (u + 2.0 ** -18) * np.abs(ref["y"]) + tiny)
    return ref


@pytest.mark.parametrize("residual", [True, False])
@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,cols", SIZES)
def test_rms_norm(rows, cols, kind, residual):
    x, res, w, g, gs = make(rows, cols, kind, residual=residual)
    y, rstd, total = oeq.oeq_rms_norm_fwd(x, w, residual=res)
    assert y.dtype == total.dtype == TYPES[kind]
    if residual:
        assert torch.equal(total, (x.float() + res.float()).to(TYPES[kind]))
    else:
        assert total is x
    check_forward(y, rstd, total, w, kind)
    gx, gw = oeq.oeq_rms_norm_bwd(total, rstd, g, w, grad_sum=gs)
    ref = decoder.rms_norm(host(total), host(w), 1e-5, host(g), None if gs is None else host(gs))
    terms = np.abs(host(g) * host(w)).max(1, keepdims=True) * ref["rstd"][:, None] * 8 + \
        (0 if gs is None else np.abs(host(gs)))
    u = torch.finfo(TYPES[kind]).eps / 2
    assert np.all(np.abs(host(gx) - ref["grad_x"]) <= u * np.abs(ref["grad_x"]) + 2.0 ** -16 * terms + 2.0 ** -25)
    size = np.abs(host(g) * host(total) * ref["rstd"][:, None]).sum(0)
    assert gw.dtype == torch.float32 and np.all(np.abs(host(gw) - ref["grad_weight"]) <= 2.0 ** -18 * size)
    again = oeq.oeq_rms_norm_bwd(total, rstd, g, w, grad_sum=gs)
    assert torch.equal(gx, again[0]) and torch.equal(gw, again[1])


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("rows,cols", SIZES)
def test_rms_norm_to_8_bits(rows, cols, kind):
    x, res, w, _, _ = make(rows, cols, kind, seed=1)
    q, scale, rstd, total = oeq.oeq_rms_norm_e4m3_fwd(x, w, residual=res)
    y, rstd_too, total_too = oeq.oeq_rms_norm_fwd(x, w, residual=res)
    assert q.dtype == torch.float8_e4m3fn and torch.equal(rstd, rstd_too) and torch.equal(total, total_too)
    ref = decoder.rms_norm(host(total), host(w))
    assert np.all(np.abs(host(scale) - ref["scale"]) <= 2.0 ** -18 * ref["scale"])
    over = ref["y"] / host(scale)[:, None]
    got = host(q.float())
    # the nearest value, or its neighbour where fp32's rounding of y / scale lies across the middle
    assert np.all(np.abs(got - over) <= np.abs(decoder.to_e4m3(over) - over) + 2.0 ** -17 * np.abs(over))
    assert np.all(np.abs(got - over) <= np.maximum(2.0 ** -4 * np.abs(over), 2.0 ** -10) * (1 + 2.0 ** -12))
    assert np.all(np.abs(got).max(1) == 448.0)  # the largest of a row takes the largest value


@pytest.mark.parametrize("kind", list(TYPES))
def test_rows_of_zeros(kind):
    x = torch.zeros(5, 72, device="cuda").to(TYPES[kind])
    y, rstd, _ = oeq.oeq_rms_norm_fwd(x)
    assert torch.all(y == 0) and np.allclose(host(rstd), 1e-5 ** -0.5, rtol=2.0 ** -18)
    q, scale, _, _ = oeq.oeq_rms_norm_e4m3_fwd(x)
    assert torch.all(q.float() == 0) and torch.all(scale > 0)


@pytest.mark.parametrize("cols", [40, 1000, 2900, 9000])
@pytest.mark.parametrize("size,eps", [(1e19, 1e-5), (3e30, 1e-5), (1e37, 1e-5), (1e-22, 1e-38), (3e-30, 1e-38), (1e-22, 1e-5)])
def test_squares_outside_fp32(size, eps, cols):
    r = np.random.default_rng(3)
    x = torch.from_numpy(r.normal(size=(6, cols)) * size).float().cuda()
    x[2] = torch.from_numpy(r.normal(size=cols))  # an ordinary row among them
    y, rstd, _ = oeq.oeq_rms_norm_fwd(x, eps=eps)
    check_forward(y, rstd, x, None, "f32", eps=float(np.float32(eps)))


def test_rows_that_are_not_finite_stay_their_own_matter():
    x = torch.randn(9, 200, device="cuda")
    clean, clean8 = oeq.oeq_rms_norm_fwd(x)[0], oeq.oeq_rms_norm_e4m3_fwd(x)[0]
    x[2, 7], x[5, 190] = float("nan"), float("inf")
    y, rstd, _ = oeq.oeq_rms_norm_fwd(x)
    q, scale, _, _ = oeq.oeq_rms_norm_e4m3_fwd(x)
    others = [0, 1, 3, 4, 6, 7, 8]
    assert torch.equal(y[others], clean[others])
    assert torch.equal(q[others].view(torch.uint8), clean8[others].view(torch.uint8))
    assert torch.all(y[2].isnan()) and torch.all(q[2].float().isnan()) and scale[2].isnan()
    assert y[5, 190].isnan() and q[5, 190].float().isnan()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("cols", [50, 1100])
def test_strided_and_in_place(cols, kind):
    x, res, w, g, gs = make(40, cols, kind)
    want = oeq.oeq_rms_norm_fwd(x, w, residual=res)
    wide = torch.full((40, 2 * cols + 3), 7.0, device="cuda").to(TYPES[kind])
    wide[:, 1:cols + 1] = x
    to = torch.full((40, cols + 9), 7.0, device="cuda").to(TYPES[kind])
    stream = res.clone()
    y, rstd, total = oeq.oeq_rms_norm_fwd(wide[:, 1:cols + 1], w, residual=stream, out=to[:, 2:cols + 2], sum=stream)
    assert total is stream and all(torch.equal(a, b) for a, b in zip((y, rstd, total), want))
    assert torch.all(to[:, :2] == 7) and torch.all(to[:, cols + 2:] == 7)
    mine = x.clone()
    assert torch.equal(oeq.oeq_rms_norm_fwd(mine, w, residual=res, sum=mine)[0], want[0]) and torch.equal(mine, want[2])
    q, scale, _, _ = oeq.oeq_rms_norm_e4m3_fwd(x, w, residual=res)
    bytes_ = torch.zeros((40, cols + 5), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    q2 = oeq.oeq_rms_norm_e4m3_fwd(x, w, residual=res, out=bytes_[:, 3:cols + 3])[0]
    assert torch.equal(q2.float(), q.float())
    assert torch.all(bytes_[:, :3].float() == 0) and torch.all(bytes_[:, cols + 3:].float() == 0)
    gx, gw = oeq.oeq_rms_norm_bwd(total, rstd, g, w, grad_sum=gs)
    in_place = gs.clone()
    got = oeq.oeq_rms_norm_bwd(total, rstd, g, w, grad_sum=in_place, out=in_place)
    assert torch.equal(in_place, gx) and torch.equal(got[1], gw)
    in_place = g.clone()
    oeq.oeq_rms_norm_bwd(total, rstd, in_place, w, grad_sum=gs, out=in_place, need=("x",))
    assert torch.equal(in_place, gx)


def test_gradients_asked_for_alone_and_no_rows():
    x, res, w, g, gs = make(70, 90, "f32")
    _, rstd, total = oeq.oeq_rms_norm_fwd(x, w, residual=res)
    gx, gw = oeq.oeq_rms_norm_bwd(total, rstd, g, w)
    a, b = oeq.oeq_rms_norm_bwd(total, rstd, g, w, need=("weight",)), oeq.oeq_rms_norm_bwd(total, rstd, g, w, need=("x",))
    assert a[0] is None and b[1] is None and torch.equal(a[1], gw) and torch.equal(b[0], gx)
    none = x[:0]
    y, rstd, total = oeq.oeq_rms_norm_fwd(none, w, residual=none)
    assert y.shape == total.shape == (0, 90)
    gx, gw = oeq.oeq_rms_norm_bwd(total, rstd, none, w)
    assert gx.shape == (0, 90) and torch.all(gw == 0)


def test_gradients_are_differences_of_the_forward():
    x, res, w, g, gs = make(6, 40, "f32")
    _, rstd, total = oeq.oeq_rms_norm_fwd(x, w, residual=res)
    gx, gw = oeq.oeq_rms_norm_bwd(total, rstd, g, w, grad_sum=gs)

    def value(x, w):
        y, _, total = oeq.oeq_rms_norm_fwd(x, w, residual=res)
        return float((y.double() * g.double()).sum() + (total.double() * gs.double()).sum())

    step = 1e-2  # truncation of order 1e-4 of the gradient, rounding 240 x 2^-23 / 1e-2
    for t, grad, at in ((x, gx, lambda v: value(v, w)), (w, gw, lambda v: value(x, v))):
        d = torch.randn_like(t)
        d /= d.norm()
        change = (at(t + step * d) - at(t - step * d)) / (2 * step)
        assert abs(change - float((grad.double() * d.double()).sum())) <= 1e-2 * float(grad.norm()) + 1e-2


def test_on_a_side_stream_and_in_a_graph():
    x, res, w, g, gs = make(300, 600, "bf16")

    def step():
        y, rstd, total = oeq.oeq_rms_norm_fwd(x, w, residual=res)
        q, scale, _, _ = oeq.oeq_rms_norm_e4m3_fwd(x, w, residual=res)
        gx, gw = oeq.oeq_rms_norm_bwd(total, rstd, g, w, grad_sum=gs)
        return y, rstd, total, q.view(torch.uint8), scale, gx, gw

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
        for t, u in zip((x, res, w, g, gs), make(300, 600, "bf16", seed=seed + 9)):
            t.copy_(u)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_in_the_callers_workspace():
    x, res, w, g, _ = make(700, 300, "f32")
    _, rstd, total = oeq.oeq_rms_norm_fwd(x, w, residual=res)
    n = oeq.oeq_rms_norm_workspace_size(700, 300)
    whole = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    got, want = oeq.oeq_rms_norm_bwd(total, rstd, g, w, workspace=whole[:n]), oeq.oeq_rms_norm_bwd(total, rstd, g, w)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.all(whole[n:] == 0x5A)
    with pytest.raises(oeq.OeqError):
        oeq.oeq_rms_norm_bwd(total, rstd, g, w, workspace=whole[:n - 256])


def test_what_the_binding_refuses():
    x, res, w, g, _ = make(4, 24, "bf16")
    with pytest.raises(TypeError):
        oeq.oeq_rms_norm_fwd(x, w.bfloat16())
    with pytest.raises(TypeError):
        oeq.oeq_rms_norm_fwd(x, w, residual=res.float())
    with pytest.raises(ValueError):
        oeq.oeq_rms_norm_fwd(x, w, residual=res[:3])
    with pytest.raises(ValueError):
        oeq.oeq_rms_norm_fwd(x, w[:23])
    with pytest.raises(ValueError):
        oeq.oeq_rms_norm_fwd(x, w, sum=x)
    with pytest.raises(oeq.OeqError):
        oeq.oeq_rms_norm_fwd(x, w, eps=0.0)
    with pytest.raises(oeq.OeqError):
        oeq.oeq_rms_norm_fwd(torch.zeros(1, 16385, device="cuda"))
    with pytest.raises(TypeError):
        oeq.oeq_rms_norm_e4m3_fwd(x, w, out=torch.empty_like(x))
    with pytest.raises(TypeError):
        oeq.oeq_rms_norm_fwd(x.cpu())
