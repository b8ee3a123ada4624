"""A readout of whole structures on top of the convolution, trained end to end.

    species -> oeq_embedding_fwd -> node features -> oeq_tp_conv_fwd_pos -> the scalar block of the rows, in place
      -> oeq_group_norm_fwd (per structure, SiLU) -> keys and values (one dense product)
      -> oeq_cross_attn_fwd from a few learned query tokens to each structure's atoms
      -> oeq_dropout_fwd onto the tokens -> one number per structure

Structures of different sizes are stacked along the atoms.  The backward chains the library's
gradients in the opposite order; dense products are torch's.  Run on a GPU:

    python examples/invariant_readout.py
"""
from __future__ import annotations

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import cg_tensor_product_amd as oeq  # noqa: E402

SPECIES, CHANNELS, GROUPS, TOKENS, HEADS, DIM = 4, 32, 4, 3, 4, 16
NEIGHBOURS = 6


def make_batch(structures=24, seed=0, device="cuda"):
    """Stacked structures of 5 to 30 atoms, their graph, and a number to learn for each: the mean
    of a value per species."""
    gen = torch.Generator().manual_seed(seed)
    sizes = torch.randint(5, 31, (structures,), generator=gen)
    ptr = torch.cat([torch.zeros(1, dtype=torch.long), sizes.cumsum(0)])
    n = int(ptr[-1])
    of = torch.repeat_interleave(torch.arange(structures), sizes)
    step = torch.randint(1, 1 << 20, (n, NEIGHBOURS), generator=gen)
    src = ptr[of][:, None] + (torch.arange(n)[:, None] - ptr[of][:, None] + 1 + step % (sizes[of][:, None] - 1)) % \
        sizes[of][:, None]  # any other atom of the same structure
    species = torch.randint(0, SPECIES, (n,), generator=gen)
    value = torch.tensor([-1.0, -0.2, 0.4, 1.5])[species]
    target = torch.zeros(structures).index_add_(0, of, value) / sizes
    as_int = dict(dtype=torch.int32, device=device)
    return {"ptr": ptr.to(**as_int), "rowptr": torch.arange(0, n * NEIGHBOURS + 1, NEIGHBOURS).to(**as_int),
            "src": src.reshape(-1).to(**as_int), "pos": torch.randn(n, 3, generator=gen).to(device),
            "species": species.to(device), "target": target.to(device),
            "token_ptr": (torch.arange(structures + 1) * TOKENS).to(**as_int),
            # added to (seed, offset): the tokens' dropout draws from another seed than the attention's
            "other_seed": torch.tensor([1, 0], device=device)}


def make_model(plan, seed=1, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s, scale: (torch.randn(*s, generator=gen) * scale).to(device)  # noqa: E731
    width = HEADS * DIM
    return {"embed": rand(SPECIES, CHANNELS, scale=1.0), "edge": rand(1, plan.n_paths, plan.U, scale=NEIGHBOURS ** -0.5),
            "norm_weight": torch.ones(CHANNELS, device=device), "norm_bias": torch.zeros(CHANNELS, device=device),
            "kv": rand(CHANNELS, 2 * width, scale=CHANNELS ** -0.5), "tokens": rand(TOKENS, width, scale=1.0),
            "head": rand(width, scale=width ** -0.5)}


def forward(plan, model, batch, p_drop, rng):
    """Predictions [structures] and what the backward needs."""
    s = {}
    structures = batch["target"].shape[0]
    s["x"] = oeq.oeq_embedding_fwd(model["embed"], batch["species"])
    s["W"] = model["edge"].expand(batch["src"].shape[0], -1, -1).contiguous()
    s["rows"] = oeq.oeq_tp_conv_fwd_pos(plan, batch["rowptr"], batch["src"], s["x"], batch["pos"], s["W"])
    # the first block of a row is its CHANNELS scalars: normalised where they are
    s["normed"], s["mean"], s["rstd"] = oeq.oeq_group_norm_fwd(s["rows"][:, :CHANNELS], batch["ptr"], GROUPS,
                                                              model["norm_weight"], model["norm_bias"], act="silu")
    kv = (s["normed"] @ model["kv"]).view(-1, 2, HEADS, DIM)
    s["k"], s["v"] = kv[:, 0], kv[:, 1]
    s["q"] = model["tokens"].view(TOKENS, HEADS, DIM).repeat(structures, 1, 1)
    s["out"], s["lse"] = oeq.oeq_cross_attn_fwd(s["q"], s["k"], s["v"], batch["token_ptr"], batch["ptr"],
                                                p_drop=p_drop, rng=rng)
    s["mixed"] = oeq.oeq_dropout_fwd(s["out"].view(-1, HEADS * DIM), p_drop, rng + batch["other_seed"],
                                     residual=s["q"].view(-1, HEADS * DIM))
    return (s["mixed"] @ model["head"]).view(structures, TOKENS).mean(1), s



def backward(plan, model, batch, s, grad, p_drop, rng):
    """Gradients of sum(grad * predictions) for every parameter, and to the atoms' positions."""
    structures, width = grad.shape[0], HEADS * DIM
    g = {}
    per_token = (grad / TOKENS).repeat_interleave(TOKENS)
    g["head"] = per_token @ s["mixed"]
    grad_mixed = per_token[:, None] * model["head"]
    grad_out = oeq.oeq_dropout_bwd(grad_mixed, p_drop, rng + batch["other_seed"]).view(-1, HEADS, DIM)
    gq, gk, gv = oeq.oeq_cross_attn_bwd(s["q"], s["k"], s["v"], batch["token_ptr"], batch["ptr"], s["out"], s["lse"],
                                        grad_out, p_drop=p_drop, rng=rng)
    g["tokens"] = (gq.view(-1, width) + grad_mixed).view(structures, TOKENS, width).sum(0)
    grad_kv = torch.stack([gk, gv], 1).view(-1, 2 * width)
    g["kv"] = s["normed"].t() @ grad_kv
    grad_rows = torch.zeros_like(s["rows"])
    _, g["norm_weight"], g["norm_bias"] = oeq.oeq_group_norm_bwd(
        s["rows"][:, :CHANNELS], batch["ptr"], GROUPS, s["mean"], s["rstd"], grad_kv @ model["kv"].t(),
        model["norm_weight"], model["norm_bias"], act="silu", out=grad_rows[:, :CHANNELS])
    gx, g_pos, gW = oeq.oeq_tp_conv_bwd_pos(plan, batch["rowptr"], batch["src"], s["x"], batch["pos"], s["W"],
                                            grad_rows)
    g["embed"] = oeq.oeq_embedding_bwd(batch["species"], gx, SPECIES)
    g["edge"] = gW.sum(0, keepdim=True)
    return g, g_pos


def train(steps=60, p_drop=0.1, lr=1e-2, report=None):
    """Losses of each step."""
    plan = oeq.Plan(f"{CHANNELS}x0e", 1, 1, "f32")
    batch, model = make_batch(), make_model(plan)
    params = [p.requires_grad_() for p in model.values()]
    optimiser = torch.optim.Adam(params, lr=lr)
    rng = torch.tensor([2024, 0], device="cuda")  # seed, offset
    losses = []
    for step in range(steps):
        with torch.no_grad():
            got, saved = forward(plan, model, batch, p_drop, rng)
            error = got - batch["target"]
            grads, _ = backward(plan, model, batch, saved, 2 * error / error.numel(), p_drop, rng)
            for name, p in model.items():
                p.grad = grads[name]
            rng[1] += 1  # the next step draws other masks
        optimiser.step()
        losses.append(float(error.square().mean()))
        if report and step % 10 == 0:
            report(f"step {step:3d}  loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    train(report=print)
