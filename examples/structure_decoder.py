"""A decoder that writes the species of each structure's atoms in order, one token after another.

    tokens -> oeq_embedding_fwd -> x
      -> oeq_rms_norm_fwd -> queries, keys, values (one dense product) -> oeq_causal_attn_fwd
      -> oeq_rms_norm_fwd onto the residual stream -> oeq_cross_attn_fwd to the structure's atoms
      -> oeq_rms_norm_fwd onto the residual stream -> one score per species

Sequences of different lengths are packed along the tokens, structures along the atoms.  The backward
chains the library's gradients in the opposite order; dense products are torch's.  `generate` writes
token by token, with a cache of keys and values that has rows to spare.  Run on a GPU:

    python examples/structure_decoder.py
"""
from __future__ import annotations

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import cg_tensor_product_amd as oeq  # noqa: E402

SPECIES, CHANNELS, HEADS, KV_HEADS, DIM = 5, 64, 4, 2, 16
BEGIN = SPECIES  # the token before the first atom
SCALE = CHANNELS ** 0.5


def make_batch(structures=24, seed=0, device="cuda"):
    """Stacked structures of 3 to 12 atoms; the tokens to write are their species in order."""
    gen = torch.Generator().manual_seed(seed)
    sizes = torch.randint(3, 13, (structures,), generator=gen)
    ptr = torch.cat([torch.zeros(1, dtype=torch.long), sizes.cumsum(0)])
    species = torch.randint(0, SPECIES, (int(ptr[-1]),), generator=gen)
    target = torch.cat([species[a:b].sort().values for a, b in zip(ptr, ptr[1:])])
    tokens = target.roll(1)
    tokens[ptr[:-1]] = BEGIN
    return {"ptr": ptr.to(device, torch.int32), "species": species.to(device), "tokens": tokens.to(device),
            "target": target.to(device), "longest": int(sizes.max())}


def make_model(seed=1, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    rand = lambda *s: (torch.randn(*s, generator=gen) * s[0] ** -0.5).to(device)  # noqa: E731
    width, kv = HEADS * DIM, KV_HEADS * DIM
    m = {"token": rand(SPECIES + 1, CHANNELS), "atom": rand(SPECIES, CHANNELS), "qkv": rand(CHANNELS, width + 2 * kv),
         "self_out": rand(width, CHANNELS), "q": rand(CHANNELS, width), "kv": rand(CHANNELS, 2 * kv),
         "cross_out": rand(width, CHANNELS), "head": rand(CHANNELS, SPECIES)}
    for i in range(3):
        m[f"norm{i}"] = torch.ones(CHANNELS, device=device)
    return m


def atom_states(model, batch):
    """(rows of the atoms, keys, values) of the cross attention."""
    atoms = oeq.oeq_embedding_fwd(model["atom"], batch["species"], scale=SCALE)
    kv = (atoms @ model["kv"]).view(-1, 2, KV_HEADS, DIM)
    return atoms, kv[:, 0], kv[:, 1]


def split_heads(qkv):
    qkv = qkv.view(-1, HEADS + 2 * KV_HEADS, DIM)
    return qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]


def forward(model, batch):
    """Scores [tokens, species] and what the backward needs."""
    s, p = {}, batch["ptr"]
    s["x"] = oeq.oeq_embedding_fwd(model["token"], batch["tokens"], scale=SCALE)
    s["n0"], s["r0"], _ = oeq.oeq_rms_norm_fwd(s["x"], model["norm0"])
    s["q"], s["k"], s["v"] = split_heads(s["n0"] @ model["qkv"])
    s["a"], s["lse"] = oeq.oeq_causal_attn_fwd(s["q"], s["k"], s["v"], p, p)
    s["n1"], s["r1"], s["h1"] = oeq.oeq_rms_norm_fwd(s["a"].flatten(1) @ model["self_out"], model["norm1"],
                                                     residual=s["x"])
    s["q2"] = (s["n1"] @ model["q"]).view(-1, HEADS, DIM)
    s["atoms"], s["k2"], s["v2"] = atom_states(model, batch)
    s["c"], s["lse2"] = oeq.oeq_cross_attn_fwd(s["q2"], s["k2"], s["v2"], p, p)
    s["n2"], s["r2"], s["h2"] = oeq.oeq_rms_norm_fwd(s["c"].flatten(1) @ model["cross_out"], model["norm2"],
                                                     residual=s["h1"])
    return s["n2"] @ model["head"], s


def backward(model, batch, s, grad):
    """Gradients of sum(grad * scores) for every parameter."""
    g, p = {}, batch["ptr"]
    g["head"] = s["n2"].t() @ grad
    gh, g["norm2"] = oeq.oeq_rms_norm_bwd(s["h2"], s["r2"], grad @ model["head"].t(), model["norm2"])
    g["cross_out"] = s["c"].flatten(1).t() @ gh
    gq2, gk2, gv2 = oeq.oeq_cross_attn_bwd(s["q2"], s["k2"], s["v2"], p, p, s["c"], s["lse2"],
                                           (gh @ model["cross_out"].t()).view(-1, HEADS, DIM))
    gkv = torch.stack([gk2, gv2], 1).flatten(1)
    g["kv"] = s["atoms"].t() @ gkv
    g["atom"] = oeq.oeq_embedding_bwd(batch["species"], gkv @ model["kv"].t(), SPECIES, scale=SCALE)
    g["q"] = s["n1"].t() @ gq2.flatten(1)
    gh, g["norm1"] = oeq.oeq_rms_norm_bwd(s["h1"], s["r1"], gq2.flatten(1) @ model["q"].t(), model["norm1"], grad_sum=gh)
    g["self_out"] = s["a"].flatten(1).t() @ gh
    gq, gk, gv = oeq.oeq_causal_attn_bwd(s["q"], s["k"], s["v"], p, p, s["a"], s["lse"],
                                         (gh @ model["self_out"].t()).view(-1, HEADS, DIM))
    gqkv = torch.cat([gq, gk, gv], 1).flatten(1)
    g["qkv"] = s["n0"].t() @ gqkv
    gx, g["norm0"] = oeq.oeq_rms_norm_bwd(s["x"], s["r0"], gqkv @ model["qkv"].t(), model["norm0"], grad_sum=gh)
    g["token"] = oeq.oeq_embedding_bwd(batch["tokens"], gx, SPECIES + 1, scale=SCALE)
    return g


class Cache:
    """Keys and values of each structure's tokens, `rows` rows a structure, `used` of them in use."""

    def __init__(self, structures, rows, device="cuda"):
        self.k, self.v = torch.zeros((2, structures, rows, KV_HEADS, DIM), device=device).unbind(0)
        as_int = dict(dtype=torch.int32, device=device)
        self.k_ptr = torch.arange(0, structures * rows + 1, rows, **as_int)
        self.q_ptr = torch.arange(structures + 1, **as_int)
        self.used = torch.zeros(structures, **as_int)


def step(model, states, batch, cache, tokens, at):
    """Scores [structures, species] after one more token of each structure, the at-th."""
    x = oeq.oeq_embedding_fwd(model["token"], tokens, scale=SCALE)
    q, k, v = split_heads(oeq.oeq_rms_norm_fwd(x, model["norm0"])[0] @ model["qkv"])
    cache.k[:, at], cache.v[:, at] = k, v
    cache.used += 1
    a, _ = oeq.oeq_causal_attn_fwd(q, cache.k.flatten(0, 1), cache.v.flatten(0, 1), cache.q_ptr, cache.k_ptr,
                                   k_len=cache.used)
    n1, _, h1 = oeq.oeq_rms_norm_fwd(a.flatten(1) @ model["self_out"], model["norm1"], residual=x)
    c, _ = oeq.oeq_cross_attn_fwd((n1 @ model["q"]).view(-1, HEADS, DIM), *states, cache.q_ptr, batch["ptr"])
    n2, _, _ = oeq.oeq_rms_norm_fwd(c.flatten(1) @ model["cross_out"], model["norm2"], residual=h1)
    return n2 @ model["head"]


@torch.no_grad()
def generate(model, batch, steps=None):
    """The most likely tokens [structures, steps], each after those before it."""
    structures = batch["ptr"].shape[0] - 1
    steps = steps or batch["longest"]
    cache = Cache(structures, steps + 3, batch["ptr"].device)
    states = atom_states(model, batch)[1:]
    tokens, out = torch.full((structures,), BEGIN, device=batch["ptr"].device), []
    for at in range(steps):
        tokens = step(model, states, batch, cache, tokens, at).argmax(1)
        out.append(tokens)
    return torch.stack(out, 1)


def train(steps=200, lr=5e-3, report=None):
    """(model, batch, mean loss of each step)"""
    batch, model = make_batch(), make_model()
    optimiser = torch.optim.Adam([p.requires_grad_() for p in model.values()], lr=lr)
    losses = []
    for i in range(steps):
        with torch.no_grad():
            scores, saved = forward(model, batch)
            log_p = scores.log_softmax(1)
            grad = log_p.exp()
            grad[torch.arange(grad.shape[0]), batch["target"]] -= 1
            grads = backward(model, batch, saved, grad / grad.shape[0])
            for name, p in model.items():
                p.grad = grads[name]
            losses.append(-float(log_p.gather(1, batch["target"][:, None]).mean()))
        optimiser.step()
        if report and i % 25 == 0:
            report(f"step {i:3d}  loss {losses[-1]:.4f}")
    return model, batch, losses


if __name__ == "__main__":
    model, batch, _ = train(report=print)
    written, ptr = generate(model, batch), batch["ptr"].tolist()
    right = sum(int((written[b, :n - a] == batch["target"][a:n]).sum()) for b, (a, n) in enumerate(zip(ptr, ptr[1:])))
    print(f"{right} of {ptr[-1]} atoms written right")
