"""The decoder example, a run of the decoder operators together: its gradients against differences of its own
forward, its steps with a cache against the whole forward, and that it runs."""
import math
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
oeq = pytest.importorskip("cg_tensor_product_amd")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
decoder = pytest.importorskip("structure_decoder")


def test_gradients_are_differences_of_the_forward():
    batch, model = decoder.make_batch(7, seed=3), decoder.make_model(seed=4)
    gen = torch.Generator().manual_seed(0)
    weight = torch.randn(batch["tokens"].shape[0], decoder.SPECIES, generator=gen).cuda()

    def value():
        return float((decoder.forward(model, batch)[0] * weight).double().sum())

    grads = decoder.backward(model, batch, decoder.forward(model, batch)[1], weight)
    assert set(grads) == set(model)
    # central differences along one direction a tensor: with a step of 1e-2 in fp32 the truncation is
    # of order 1e-4 of the gradient's size, the rounding (scores of about 250 values) 1e-5 / 1e-2
    for name, t in model.items():
        direction = torch.randn(t.shape, generator=gen).to("cuda")
        direction /= direction.norm()
        keep, eps = t.clone(), 1e-2
        t.copy_(keep + eps * direction)
        hi = value()
        t.copy_(keep - eps * direction)
        lo = value()
        t.copy_(keep)
        want = float((grads[name].double() * direction.double()).sum())
        assert abs((hi - lo) / (2 * eps) - want) <= 1e-2 * float(grads[name].norm()) + 2e-2, name


def test_steps_with_a_cache_equal_the_whole_forward():
    batch, model = decoder.make_batch(9, seed=5), decoder.make_model(seed=6)
    whole, ptr = decoder.forward(model, batch)[0], batch["ptr"].tolist()
    cache = decoder.Cache(9, batch["longest"] + 5)
    states = decoder.atom_states(model, batch)[1:]
    for at in range(batch["longest"]):
        # a structure that has no such token writes some other one
        rows = torch.tensor([min(a + at, b - 1) for a, b in zip(ptr, ptr[1:])], device="cuda")
        scores = decoder.step(model, states, batch, cache, batch["tokens"][rows], at)
        there = torch.tensor([a + at < b for a, b in zip(ptr, ptr[1:])], device="cuda")
        want = whole[rows][there]
        # fp32 through both attentions and six dense products, in another order
        assert float((scores[there] - want).abs().max()) <= 2.0 ** -14 * (1 + float(want.abs().max()))


def test_it_trains_and_writes():
    model, batch, losses = decoder.train(steps=10)
    assert len(losses) == 10 and all(math.isfinite(v) for v in losses)
    written = decoder.generate(model, batch)
    assert written.shape == (24, batch["longest"]) and int(written.min()) >= 0 and int(written.max()) < decoder.SPECIES
