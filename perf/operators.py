"""Measured cases of the readout operators: group norm with an activation over the
atoms of each structure, dropout from a counter-based generator, and cross attention
from query tokens to the atoms of their structure.

Atoms (and query tokens) of all structures are stacked along the rows, and a CSR row
pointer per side says which rows belong to which structure, as the receiver CSR of the
convolution does.  `run` computes either the plain form (elementary torch operations in
32 bits, rounded once at the end) or, where `own` is set, the library's operators.
"""
from __future__ import annotations

import functools
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5

# What a case costs at most: group norm and dropout elements, attention scores (query rows x
# heads x longest sequence) of a forward and of a training pass.
MOST_ELEMENTS = 280_000 * 256
MOST_SCORES = {"fwd": 2 * 16 * 2048 * 5000, "train": 8 * 8 * 1024 * 2048}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # ---- group norm --------------------------------------------------------------------
        # one molecule's invariant features at inference: only latency counts
        {"name": "gn_fwd_molecule_f32", "op": "gn", "mode": "fwd", "type": "f32", "structures": 1, "rows": 21,
         "channels": 64, "groups": 8, "act": "silu", "width": 64},
        # a training batch of 64 structures, 5,000 atoms in all: the 128 scalars of node rows
        # 128x0e+128x1o (512 wide), read in place
        {"name": "gn_train_batch_f32", "op": "gn", "mode": "train", "type": "f32", "structures": 64, "rows": 5000,
         "channels": 128, "groups": 8, "act": "silu", "width": 512},
        # one large box of atoms (a molecular-dynamics frame), an odd number of rows
        {"name": "gn_fwd_box_f32", "op": "gn", "mode": "fwd", "type": "f32", "structures": 1, "rows": 100003,
         "channels": 128, "groups": 16, "act": "none", "width": 128},
        # edge embeddings (280,000 edges) of 32 structures in training, 256 channels
        {"name": "gn_train_edges_bf16", "op": "gn", "mode": "train", "type": "bf16", "structures": 32,
         "rows": 280000, "channels": 256, "groups": 32, "act": "silu", "width": 256},
        # ---- dropout -----------------------------------------------------------------------
        # the pooled tokens of a few structures: latency
        {"name": "drop_fwd_tokens_bf16", "op": "drop", "mode": "fwd", "type": "bf16", "rows": 64, "cols": 128,
         "p": 0.1, "residual": True},
        # whole node rows of the 5,000-atom graph (128x0e+128x1o+128x2e), with the residual stream
        {"name": "drop_train_nodes_f32", "op": "drop", "mode": "train", "type": "f32", "rows": 5000, "cols": 1152,
         "p": 0.1, "residual": True},
        # per-edge features in training
        {"name": "drop_train_edges_bf16", "op": "drop", "mode": "train", "type": "bf16", "rows": 280000,
         "cols": 256, "p": 0.25, "residual": False},
        # ---- cross attention -----------------------------------------------------------------
        # a readout token of one molecule: latency
        {"name": "attn_fwd_molecule_f32", "op": "attn", "mode": "fwd", "type": "f32", "structures": 1, "q_most": 1,
         "k_most": 56, "ragged": False, "heads": 4, "kv_heads": 4, "dim": 32, "p": 0.0, "masked": 0.0},
        # serving: one new token for each of 16 requests, each over its own structure's states
        {"name": "attn_fwd_token_bf16", "op": "attn", "mode": "fwd", "type": "bf16", "structures": 16, "q_most": 1,
         "k_most": 5000, "ragged": True, "heads": 16, "kv_heads": 4, "dim": 64, "p": 0.0, "masked": 0.1},
        # training of a readout with 32 latent tokens on 64 small structures
        {"name": "attn_train_batch_f32", "op": "attn", "mode": "train", "type": "f32", "structures": 64,
         "q_most": 32, "k_most": 200, "ragged": True, "heads": 8, "kv_heads": 8, "dim": 32, "p": 0.1, "masked": 0.0},
        # training of a decoder over structure states, with masked states and shared key heads
        {"name": "attn_train_decoder_bf16", "op": "attn", "mode": "train", "type": "bf16", "structures": 8,
         "q_most": 1024, "k_most": 2048, "ragged": True, "heads": 8, "kv_heads": 4, "dim": 64, "p": 0.1,
         "masked": 0.1},
        # a long prompt over 5,000 atoms at inference
        {"name": "attn_fwd_prompt_f16", "op": "attn", "mode": "fwd", "type": "f16", "structures": 2, "q_most": 2048,
         "k_most": 5000, "ragged": False, "heads": 16, "kv_heads": 4, "dim": 128, "p": 0.0, "masked": 0.0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gn", "drop", "attn", "attn"])
    mode = rng.choice(["fwd", "train"])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op == "gn":
        group = rng.choice([1, 3, 4, 8, 10, 16, 32])
        groups = rng.choice([g for g in (1, 2, 4, 6, 8, 16, 32) if 16 <= g * group <= 512])
        channels = group * groups
        rows = _log(rng, 8, MOST_ELEMENTS // max(256, channels))
        return {"op": op, "mode": mode, "type": kind, "structures": _log(rng, 1, min(256, rows)), "rows": rows,
                "channels": channels, "groups": groups, "act": rng.choice(["none", "silu"]),
                "width": channels * rng.choice([1, 1, 4])}
    if op == "drop":
        cols = _log(rng, 17, 1152)
        return {"op": op, "mode": mode, "type": kind, "rows": _log(rng, 8, MOST_ELEMENTS // max(256, cols)),
                "cols": cols, "p": rng.choice([0.05, 0.1, 0.25, 0.5]), "residual": rng.choice([True, False])}
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 1, 2, 4])
    dim = rng.choice([16, 24, 32, 40, 64, 80, 128])
    structures = _log(rng, 1, 64)
    # as many rows a side as fit what a case may cost
    per = MOST_SCORES[mode] * 64 // (structures * heads * max(dim, 64))
    q_most = rng.choice([1, _log(rng, 2, 2048)]) if mode == "fwd" else _log(rng, 1, 1024)
    k_most = _log(rng, 8, max(8, min(16384, per // q_most)))
    return {"op": op, "mode": mode, "type": kind, "structures": structures, "q_most": q_most, "k_most": k_most,
            "ragged": rng.choice([True, False]), "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "p": rng.choice([0.0, 0.1]) if mode == "train" else 0.0, "masked": rng.choice([0.0, 0.1])}


def _shares(count, total, salt):
    """Row pointer [count + 1] of `total` rows in `count` structures of uneven sizes."""
    r = random.Random(salt)
    cuts = sorted(r.randint(0, total) for _ in range(count - 1))
    return [0, *cuts, total]


def _lengths(case):
    """Query and key lengths of each structure: a fourth of the longest to the longest where
    the case is ragged; the first structure has the longest."""
    n, out = case["structures"], []
    for side in ("q_most", "k_most"):
        most = case[side]
        r = random.Random("%s %d %d" % (side, n, most))
        out.append([most] + [r.randint((most + 3) // 4, most) if case["ragged"] else most for _ in range(n - 1)])
    return out


def _ptr(lengths):
    out = [0]
    for v in lengths:
        out.append(out[-1] + v)
    return out


def work(case):
    size, train = SIZES[case["type"]], case["mode"] == "train"
    if case["op"] == "gn":
        n = case["rows"] * case["channels"]
        stats = 8 * case["structures"] * case["groups"] + 8 * case["channels"]
        ptr = 4 * (case["structures"] + 1)
        # forward: x in, y out.  Backward: x and the output's gradient in, the gradient of x out
        # (and the weights', with the saved statistics in)
        return {"bytes": n * size * (5 if train else 2) + (ptr + stats) * (2 if train else 1)
                + (8 * case["channels"] if train else 0), "flops": n * (30 if train else 10)}
    if case["op"] == "drop":
        n = case["rows"] * case["cols"]
        return {"bytes": n * size * (2 + case["residual"] + (2 if train else 0)) + 16 * (2 if train else 1),
                "flops": n * (4 if train else 2)}
    q_len, k_len = _lengths(case)
    tq, tk, h, hk, d = sum(q_len), sum(k_len), case["heads"], case["kv_heads"], case["dim"]
    rows, states, side = tq * h * d * size, tk * hk * d * size, 4 * tq * h
    small = 8 * (case["structures"] + 1) + (tk if case["masked"] else 0)
    scores = h * sum(a * b for a, b in zip(q_len, k_len)) * (1 - case["masked"])
    # forward: q, k, v in, out and the rows' log sums out; two products.  Backward: q, k, v, out,
    # its gradient and the log sums in, three gradients out; five products
    return {"bytes": 2 * rows + 2 * states + side + small + ((4 * rows + 4 * states + side + small) if train else 0),
            "flops": scores * d * 2 * (7 if train else 2)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = TYPES[case["type"]]
    train = case["mode"] == "train"

    def normal(*shape, scale=1.0, shift=0.0, dtype=dt):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).add_(shift).to(dtype)

    def index(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    s = {"case": dict(case)}
    if case["op"] == "gn":
        t, c = case["rows"], case["channels"]
        # node rows hold the normalised channels first, and what else a row holds after them
        s["x"] = normal(t, case["width"], scale=1.5, shift=0.25)[:, :c]
        s["weight"] = normal(c, scale=0.2, shift=1.0, dtype=torch.float32)
        s["bias"] = normal(c, scale=0.2, dtype=torch.float32)
        s["ptr"] = index(_shares(case["structures"], t, "%d %d" % (case["structures"], t)))
        s["grad"] = normal(t, c) if train else None
        return s
    s["rng"] = torch.tensor([int(seed) * 0x9E3779B97F4A7C1 + 12345 & (1 << 62) - 1, int(seed) + 1], dtype=torch.int64,
                            device="cuda")
    if case["op"] == "drop":
        s["x"] = normal(case["rows"], case["cols"])
        s["residual"] = normal(case["rows"], case["cols"]) if case["residual"] else None
        s["grad"] = normal(case["rows"], case["cols"]) if train else None
        return s
    q_len, k_len = _lengths(case)
    tq, tk, h, hk, d = sum(q_len), sum(k_len), case["heads"], case["kv_heads"], case["dim"]
    s["q"] = normal(tq, h, d, scale=1.5)
    kv = normal(tk, 2, hk, d)  # keys and values come out of one projection
    s["k"], s["v"] = kv[:, 0], kv[:, 1]
    s["q_ptr"], s["k_ptr"] = index(_ptr(q_len)), index(_ptr(k_len))
    s["mask"] = None
    if case["masked"]:
        s["mask"] = (torch.rand(tk, generator=gen, device="cuda") >= case["masked"]).to(torch.uint8)
    s["scale"] = 1.0 / math.sqrt(d)
    s["q_most"], s["k_most"] = max(q_len), max(k_len)
    s["grad"] = normal(tq, h, d) if train else None
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"gn": _own_gn, "drop": _own_drop, "attn": _own_attn}[op](state)
    return {"gn": _plain_gn, "drop": _plain_drop, "attn": _plain_attn}[op](state)


def _own_gn(s):
    import cg_tensor_product_amd as oeq
    c = s["case"]
    y, mean, rstd = oeq.oeq_group_norm_fwd(s["x"], s["ptr"], c["groups"], s["weight"], s["bias"], eps=EPS,
                                           act=c["act"])
    out = {"y": y, "mean": mean, "rstd": rstd}
    if s["grad"] is not None:
        out["grad_x"], out["grad_weight"], out["grad_bias"] = oeq.oeq_group_norm_bwd(
            s["x"], s["ptr"], c["groups"], mean, rstd, s["grad"], s["weight"], s["bias"], act=c["act"])
    return out


def _own_drop(s):
    import cg_tensor_product_amd as oeq
    p = s["case"]["p"]
    out = {"y": oeq.oeq_dropout_fwd(s["x"], p, s["rng"], residual=s["residual"])}
    if s["grad"] is not None:
        out["grad_x"] = oeq.oeq_dropout_bwd(s["grad"], p, s["rng"])
    return out


def _own_attn(s):
    import cg_tensor_product_amd as oeq
    kw = {"scale": s["scale"], "key_mask": s["mask"], "p_drop": s["case"]["p"],
          "rng": s["rng"] if s["case"]["p"] else None}
    out, lse = oeq.oeq_cross_attn_fwd(s["q"], s["k"], s["v"], s["q_ptr"], s["k_ptr"], **kw)
    got = {"out": out, "lse": lse}
    if s["grad"] is not None:
        got["grad_q"], got["grad_k"], got["grad_v"] = oeq.oeq_cross_attn_bwd(
            s["q"], s["k"], s["v"], s["q_ptr"], s["k_ptr"], out, lse, s["grad"], **kw)
    return got


# ---- plain forms -------------------------------------------------------------

def _plain_gn(s):
    c = s["case"]
    dt, n, g = s["x"].dtype, c["structures"], c["groups"]
    ptr = s["ptr"].long()
    rows = ptr[1:] - ptr[:-1]
    of = torch.repeat_interleave(torch.arange(n, device=ptr.device), rows, output_size=c["rows"])
    x = s["x"].float().reshape(c["rows"], g, -1)
    count = (rows * x.shape[2]).float().clamp(min=1)[:, None]

    member = (of == torch.arange(n, device=of.device)[:, None]).float()

    def total(v):  # sums over the rows of each structure
        return member @ v

    mean = total(x.sum(2)) / count
    centred = x - mean[of][:, :, None]
    var = total(centred.square().sum(2)) / count
    rstd = torch.where(rows[:, None] > 0, torch.rsqrt(var + EPS), torch.zeros_like(var))
    hat = centred * rstd[of][:, :, None]
    w, b = s["weight"].view(1, g, -1), s["bias"].view(1, g, -1)
    z = hat * w + b
    silu = c["act"] == "silu"
    gate = torch.sigmoid(z) if silu else None
    out = {"y": (z * gate if silu else z).reshape(c["rows"], -1).to(dt), "mean": mean, "rstd": rstd}
    if s["grad"] is not None:
        dz = s["grad"].float().reshape(x.shape)
        if silu:
            dz = dz * gate * (1 + z * (1 - gate))
        out["grad_weight"] = (dz * hat).sum(0).reshape(-1)
        out["grad_bias"] = dz.sum(0).reshape(-1)
        dhat = dz * w
        m1 = total(dhat.sum(2)) / count
        m2 = total((dhat * hat).sum(2)) / count
        gx = rstd[of][:, :, None] * (dhat - m1[of][:, :, None] - hat * m2[of][:, :, None])
        out["grad_x"] = gx.reshape(c["rows"], -1).to(dt)
    return out


M32 = 0xFFFFFFFF


def _mul_hi_lo(a, m):
    """High and low words of the product of 32-bit words held in int64 (the product wraps to
    the right 64 bits)."""
    p = a * m
    return (p >> 32) & M32, p & M32


def _philox_round(state, i):
    """One round of Philox4x32 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
    easy as 1, 2, 3", SC 2011)."""
    c0, c1, c2, c3, k0, k1 = state
    h0, l0 = _mul_hi_lo(c0, 0xD2511F53)
    h1, l1 = _mul_hi_lo(c2, 0xCD9E8D57)
    return h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0, (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32


def _plain_factors(rng, p, row, cols):
    """Factors [*row.shape, cols]: 0 where dropped, 1 / (share kept) elsewhere.  Eight columns
    take the eight 16-bit parts of one Philox4x32-10 block with counter (column / 8, row,
    offset) and key seed; a part below the threshold drops its column."""
    block = torch.arange((cols + 7) // 8, device=row.device)
    seed, offset = rng[0], rng[1]
    c0, c1 = torch.broadcast_tensors(block, row[..., None])
    state = (c0, c1, torch.full_like(c0, 0) + (offset & M32), torch.full_like(c0, 0) + ((offset >> 32) & M32),
             seed & M32, (seed >> 32) & M32)
    words = functools.reduce(_philox_round, range(10), state)[:4]
    parts = torch.stack([part for w in words for part in (w & 0xFFFF, w >> 16)], -1).flatten(-2)[..., :cols]
    t = min(65535, int(p * 65536 + 0.5))
    return (parts >= t).float() * (65536.0 / (65536 - t))


def _plain_drop(s):
    c, x = s["case"], s["x"]
    f = _plain_factors(s["rng"], c["p"], torch.arange(c["rows"], device=x.device), c["cols"])
    y = x.float() * f
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(x.dtype)}
    if s["grad"] is not None:
        out["grad_x"] = (s["grad"].float() * f).to(x.dtype)
    return out


def _plain_attn(s):
    c, dt, dev = s["case"], s["q"].dtype, s["q"].device
    h, hk, d = c["heads"], c["kv_heads"], c["dim"]
    b, g, lq, lk = c["structures"], h // hk, s["q_most"], s["k_most"]
    q_ptr, k_ptr = s["q_ptr"].long(), s["k_ptr"].long()
    # pad both sides to the longest: [structures, longest] row numbers and which of them are real
    q_at, k_at = q_ptr[:-1, None] + torch.arange(lq, device=dev), k_ptr[:-1, None] + torch.arange(lk, device=dev)
    q_real, k_real = q_at < q_ptr[1:, None], k_at < k_ptr[1:, None]
    q_at, k_at = q_at.clamp(max=s["q"].shape[0] - 1), k_at.clamp(max=s["k"].shape[0] - 1)
    seen = k_real if s["mask"] is None else k_real & (s["mask"][k_at] != 0)

    def padded(t, at, real):  # [structures, kv heads, rows (with the shared heads), dim] in 32 bits
        t = t[at].float().masked_fill(~real[:, :, None, None], 0.0)
        return t.view(b, at.shape[1], hk, -1, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)

    q, k, v = padded(s["q"], q_at, q_real), padded(s["k"], k_at, seen), padded(s["v"], k_at, seen)
    scores = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"])
    scores.masked_fill_(~seen[:, None, None, :], -math.inf)
    top = scores.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    prob = scores.sub_(top).exp_()
    total = prob.sum(3, keepdim=True)
    prob = prob.div_(total.clamp(min=1e-37))
    lse = (total.log() + top).view(b, h, lq).transpose(1, 2)[q_real]
    factors = None
    if c["p"]:
        row = (q_at[:, None, :] * h + torch.arange(h, device=dev)[None, :, None]).reshape(b, hk, g * lq)
        factors = _plain_factors(s["rng"], c["p"], row, lk)

    def stacked(t, heads, real):  # back to the real rows of all structures, in the inputs' type
        rows = real.shape[1]
        return t.reshape(b, heads, rows, d).transpose(1, 2)[real].to(dt)

    kept = prob if factors is None else prob * factors
    out = torch.matmul(kept, v)
    got = {"out": stacked(out, h, q_real), "lse": lse}
    if s["grad"] is not None:
        go = padded(s["grad"], q_at, q_real)
        gv = torch.matmul(kept.transpose(2, 3), go)
        gp = torch.matmul(go, v.transpose(2, 3))
        if factors is not None:
            gp = gp.mul_(factors)
        gs = gp.sub_((go * out).sum(3, keepdim=True)).mul_(prob).mul_(s["scale"])
        got["grad_q"] = stacked(torch.matmul(gs, k), h, q_real)
        got["grad_k"] = stacked(torch.matmul(gs.transpose(2, 3), q), hk, k_real)
        got["grad_v"] = stacked(gv, hk, k_real)
    return got


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64

    def factors(row, cols):
        """The dropout factors of the rows numbered `row`, with every 32-bit product formed from
        16-bit halves."""
        key, off = int(s["rng"][0]), int(s["rng"][1])
        t = min(65535, int(case["p"] * 65536 + 0.5))
        nb = (cols + 7) // 8
        c = [torch.arange(nb, device="cuda").repeat(row.numel(), 1), row[:, None].repeat(1, nb),
             torch.full((row.numel(), nb), off & M32, device="cuda"),
             torch.full((row.numel(), nb), off >> 32, device="cuda")]
        k = [key & M32, key >> 32 & M32]

        def times(a, m):
            al, ah, ml, mh = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
            low, mid = al * ml, ah * ml
            cross = al * mh + (mid & 0xFFFF) + (low >> 16)
            return ah * mh + (mid >> 16) + (cross >> 16), (cross & 0xFFFF) << 16 | low & 0xFFFF

        for i in range(10):
            a, b = times(c[0], 0xD2511F53), times(c[2], 0xCD9E8D57)
            c = [b[0] ^ c[1] ^ (k[0] + i * 0x9E3779B9 & M32), b[1], a[0] ^ c[3] ^ (k[1] + i * 0xBB67AE85 & M32), a[1]]
        keep = torch.zeros(row.numel(), nb, 8, dtype=f8, device="cuda")
        for j in range(8):
            keep[:, :, j] = ((c[j // 2] >> 16 * (j % 2)) & 0xFFFF) >= t
        return keep.view(row.numel(), -1)[:, :cols] * (65536.0 / (65536 - t))

    if case["op"] == "gn":
        g, c = case["groups"], case["channels"]
        ptr = s["ptr"].tolist()
        w, b = s["weight"].to(f8), s["bias"].to(f8)
        y = torch.empty(case["rows"], c, dtype=f8, device="cuda")
        mean = torch.zeros(case["structures"], g, dtype=f8, device="cuda")
        rstd = torch.zeros_like(mean)
        gx, gw, gb = torch.empty_like(y), torch.zeros_like(w), torch.zeros_like(b)
        for i, (lo, hi) in enumerate(zip(ptr, ptr[1:])):
            if lo == hi:
                continue
            x = s["x"][lo:hi].to(f8).view(hi - lo, g, c // g)
            mean[i] = x.mean((0, 2))
            rstd[i] = ((x - mean[i][:, None]).square().mean((0, 2)) + EPS) ** -0.5
            hat = ((x - mean[i][:, None]) * rstd[i][:, None]).view(hi - lo, c)
            z = hat * w + b
            gate = 1 / (1 + torch.exp(-z)) if case["act"] == "silu" else torch.ones_like(z)
            y[lo:hi] = z * gate
            if s["grad"] is None:
                continue
            slope = gate + z * gate * (1 - gate)  # of z * gate; where there is no gate it is 1
            dz = s["grad"][lo:hi].to(f8) * slope
            gw += (dz * hat).sum(0)
            gb += dz.sum(0)
            dh, hg = (dz * w).view(hi - lo, g, -1), hat.view(hi - lo, g, -1)
            inner = dh - dh.mean((0, 2), keepdim=True) - hg * (dh * hg).mean((0, 2), keepdim=True)
            gx[lo:hi] = (inner * rstd[i][:, None]).view(hi - lo, c)
        out = {"y": y, "mean": mean, "rstd": rstd}
        return out if s["grad"] is None else {**out, "grad_x": gx, "grad_weight": gw, "grad_bias": gb}

    if case["op"] == "drop":
        f = factors(torch.arange(case["rows"], device="cuda"), case["cols"])
        y = s["x"].to(f8) * f + (0 if s["residual"] is None else s["residual"].to(f8))
        return {"y": y} if s["grad"] is None else {"y": y, "grad_x": s["grad"].to(f8) * f}

    h, share, p = case["heads"], case["heads"] // case["kv_heads"], case["p"]
    q_ptr, k_ptr = s["q_ptr"].tolist(), s["k_ptr"].tolist()
    got = {"out": torch.zeros(s["q"].shape, dtype=f8, device="cuda"),
           "lse": torch.full(s["q"].shape[:2], -math.inf, dtype=f8, device="cuda")}
    if s["grad"] is not None:
        got.update({n: torch.zeros(s[n[-1]].shape, dtype=f8, device="cuda") for n in ("grad_q", "grad_k", "grad_v")})
    for a0, a1, b0, b1 in zip(q_ptr, q_ptr[1:], k_ptr, k_ptr[1:]):
        at = torch.arange(b0, b1, device="cuda")
        at = at if s["mask"] is None else at[s["mask"][b0:b1] != 0]  # the states that are seen
        if a0 == a1 or not at.numel():
            continue
        for j in range(h):
            q, k, v = s["q"][a0:a1, j].to(f8), s["k"][at, j // share].to(f8), s["v"][at, j // share].to(f8)
            z = q @ k.T * s["scale"]
            got["lse"][a0:a1, j] = torch.logsumexp(z, 1)
            prob = torch.exp(z - got["lse"][a0:a1, j, None])
            f = factors(torch.arange(a0, a1, device="cuda") * h + j, b1 - b0)[:, at - b0] if p else 1.0
            got["out"][a0:a1, j] = (prob * f) @ v
            if s["grad"] is None:
                continue
            go = s["grad"][a0:a1, j].to(f8)
            gp = go @ v.T * f
            gz = prob * (gp - (gp * prob).sum(1, keepdim=True)) * s["scale"]
            got["grad_q"][a0:a1, j] = gz @ k
            got["grad_k"].index_put_((at, torch.full_like(at, j // share)), gz.T @ q, accumulate=True)
            got["grad_v"].index_put_((at, torch.full_like(at, j // share)), (prob * f).T @ go, accumulate=True)
    return got
