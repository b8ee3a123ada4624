"""The readout example: its gradients against differences of its own forward, and that it learns."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
oeq = pytest.importorskip("cg_tensor_product_amd")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
readout = pytest.importorskip("invariant_readout")


@pytest.mark.parametrize("p_drop", [0.0, 0.2])
def test_gradients_are_differences_of_the_forward(p_drop):
    plan = oeq.Plan(f"{readout.CHANNELS}x0e", 1, 1, "f32")
    batch, model = readout.make_batch(6, seed=3), readout.make_model(plan, seed=4)
    rng = torch.tensor([5, 6], device="cuda")
    weight = torch.linspace(-1, 1, 6, device="cuda")

    def value():
        return float((readout.forward(plan, model, batch, p_drop, rng)[0] * weight).double().sum())

    _, saved = readout.forward(plan, model, batch, p_drop, rng)
    grads, grad_pos = readout.backward(plan, model, batch, saved, weight, p_drop, rng)
    gen = torch.Generator().manual_seed(0)
    # central differences along one direction a tensor: with a step of 1e-2 in fp32 the truncation is
    # of order 1e-4 of the gradient's size, the rounding 1e-6 / 1e-2; 1e-2 leaves both room
    for name, t, g in [(n, model[n], grads[n]) for n in model] + [("pos", batch["pos"], grad_pos)]:
        direction = torch.randn(t.shape, generator=gen).to("cuda")
        direction /= direction.norm()
        keep, eps = t.clone(), 1e-2
        t.copy_(keep + eps * direction)
        hi = value()
        t.copy_(keep - eps * direction)
        lo = value()
        t.copy_(keep)
        want = float((g.double() * direction.double()).sum())
        assert abs((hi - lo) / (2 * eps) - want) <= 1e-2 * float(g.norm()) + 1e-4, name


def test_it_learns():
    losses = readout.train(steps=60)
    assert sum(losses[-5:]) < 0.3 * sum(losses[:5])
