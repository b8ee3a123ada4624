"""Measured cases of a decoder's operators on structures: embedding lookup with its gradient by
sorted tokens, root-mean-square norm with the residual's addition (also to 8 bits with a scale a
row), and causal attention over packed sequences.

Atoms or tokens are stacked along the rows; a CSR row pointer says which rows belong to which
sequence.  `run` computes either the plain form (elementary torch operations in 32 bits or more,
rounded once at the end) or, where `own` is set, the library's operators.
"""
from __future__ import annotations

import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5
E4M3_MOST = 448.0

# What a case costs at most: elements looked up or normalised, table elements, and attention
# scores (query rows x heads x longest sequence of states) of a forward and of a training pass.
MOST_ELEMENTS = 280_000 * 256
MOST_TABLE = 32_000 * 1024
MOST_SCORES = {"fwd": 2 * 16 * 4096 * 4096, "train": 8 * 8 * 2048 * 2048}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # ---- embedding ---------------------------------------------------------------------
        # the species of one molecule's atoms at inference: only latency counts
        {"name": "emb_fwd_molecule_f32", "op": "emb", "mode": "fwd", "type": "f32", "table": 89, "rows": 56,
         "channels": 128, "skew": 2.0, "scaled": False, "absent": 0.0, "index": "i64"},
        # a training batch of 5,000 atoms, a few common species
        {"name": "emb_train_atoms_f32", "op": "emb", "mode": "train", "type": "f32", "table": 89, "rows": 5000,
         "channels": 128, "skew": 4.0, "scaled": False, "absent": 0.0, "index": "i64"},
        # the species of the senders of 280,000 edges: few rows, each with tens of thousands of uses
        {"name": "emb_train_edges_bf16", "op": "emb", "mode": "train", "type": "bf16", "table": 10, "rows": 280000,
         "channels": 256, "skew": 1.5, "scaled": False, "absent": 0.0, "index": "i32"},
        # a decoder's tokens in training, with padding
        {"name": "emb_train_tokens_bf16", "op": "emb", "mode": "train", "type": "bf16", "table": 32000, "rows": 16384,
         "channels": 1024, "skew": 4.0, "scaled": True, "absent": 0.05, "index": "i64"},
        # ---- rms norm ------------------------------------------------------------------------
        # one new token of 16 requests, to 8 bits for the next product: latency
        {"name": "rms_fwd_token_e4m3", "op": "rms", "mode": "fwd", "type": "bf16", "rows": 16, "channels": 1024,
         "residual": True, "out": "e4m3"},
        # a decoder's tokens in training
        {"name": "rms_train_tokens_bf16", "op": "rms", "mode": "train", "type": "bf16", "rows": 16384,
         "channels": 1024, "residual": True, "out": "same"},
        # a long prompt of a wide model, to 8 bits
        {"name": "rms_fwd_prompt_e4m3", "op": "rms", "mode": "fwd", "type": "bf16", "rows": 8191, "channels": 4096,
         "residual": True, "out": "e4m3"},
        # ---- causal attention ------------------------------------------------------------------
        # serving: one new token for each of 16 requests, each over its own cache
        {"name": "causal_fwd_token_bf16", "op": "causal", "mode": "fwd", "type": "bf16", "sequences": 16, "q_most": 1,
         "past_most": 5000, "spare": 120, "ragged": True, "heads": 16, "kv_heads": 4, "dim": 64, "p": 0.0,
         "masked": 0.0},
        # training on many short sequences
        {"name": "causal_train_batch_f32", "op": "causal", "mode": "train", "type": "f32", "sequences": 64,
         "q_most": 200, "past_most": 0, "spare": 0, "ragged": True, "heads": 8, "kv_heads": 8, "dim": 32, "p": 0.1,
         "masked": 0.0},
        # training of a decoder, packed sequences of different lengths with shared key heads
        {"name": "causal_train_decoder_bf16", "op": "causal", "mode": "train", "type": "bf16", "sequences": 8,
         "q_most": 2048, "past_most": 0, "spare": 0, "ragged": True, "heads": 8, "kv_heads": 4, "dim": 64, "p": 0.0,
         "masked": 0.0},
        # a chunk of a prompt over what the cache holds already
        {"name": "causal_fwd_chunk_bf16", "op": "causal", "mode": "fwd", "type": "bf16", "sequences": 2, "q_most": 500,
         "past_most": 6000, "spare": 100, "ragged": False, "heads": 16, "kv_heads": 2, "dim": 128, "p": 0.0,
         "masked": 0.1},
        # two whole prompts at inference
        {"name": "causal_fwd_prompt_f16", "op": "causal", "mode": "fwd", "type": "f16", "sequences": 2,
         "q_most": 4096, "past_most": 0, "spare": 0, "ragged": False, "heads": 16, "kv_heads": 4, "dim": 128,
         "p": 0.0, "masked": 0.0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["emb", "rms", "causal", "causal"])
    mode = rng.choice(["fwd", "train"])
    kind = rng.choice(["f32", "f16", "bf16"])
    if op == "emb":
        channels = _log(rng, 5, 2048)
        return {"op": op, "mode": mode, "type": kind, "table": _log(rng, 2, MOST_TABLE // max(channels, 320)),
                "rows": _log(rng, 8, MOST_ELEMENTS // max(channels, 256)), "channels": channels,
                "skew": rng.choice([1.0, 2.0, 4.0]), "scaled": rng.choice([True, False]),
                "absent": rng.choice([0.0, 0.05]), "index": rng.choice(["i32", "i64"])}
    if op == "rms":
        channels = _log(rng, 17, 8192)
        return {"op": op, "mode": mode, "type": kind, "rows": _log(rng, 8, MOST_ELEMENTS // max(channels, 256) // 2),
                "channels": channels, "residual": rng.choice([True, True, False]),
                "out": rng.choice(["same", "e4m3"]) if mode == "fwd" else "same"}
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 1, 2, 4])
    dim = rng.choice([16, 24, 32, 40, 64, 80, 128])
    sequences = _log(rng, 1, 64)
    # as many rows a side as fit what a case may cost
    per = MOST_SCORES[mode] * 64 // (sequences * heads * max(dim, 64))
    if mode == "train":
        q_most, past_most, spare = _log(rng, 8, min(2048, math.isqrt(per))), 0, 0
    else:
        q_most = rng.choice([1, _log(rng, 2, min(4096, math.isqrt(per)))])
        most = min(16384, per // q_most) - q_most
        past_most = rng.choice([0, _log(rng, 1, most)]) if most > 1 else 0
        spare = rng.choice([0, 37]) if past_most else 0
    return {"op": op, "mode": mode, "type": kind, "sequences": sequences, "q_most": q_most, "past_most": past_most,
            "spare": spare, "ragged": rng.choice([True, False]), "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "p": rng.choice([0.0, 0.1]) if mode == "train" else 0.0, "masked": rng.choice([0.0, 0.1])}


def _lengths(case):
    """New tokens of each sequence and the states it has before them: a fourth of the most to
    the most where the case is ragged; the first sequence has the most."""
    n, out = case["sequences"], []
    for side in ("q_most", "past_most"):
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
    if case["op"] == "emb":
        n, c = case["rows"], case["channels"]
        used, index = min(n, case["table"]), n * (8 if case["index"] == "i64" else 4)
        # forward: the index and the rows in use in, the looked-up rows out.  Backward: index and
        # gradient in, the table's gradient out
        return {"bytes": index + (used + n) * c * size + ((index + (n + case["table"]) * c * size) if train else 0),
                "flops": n * c * (2 if train else 1)}
    if case["op"] == "rms":
        n, c = case["rows"] * case["channels"], case["channels"]
        res, one = case["residual"], 1 if case["out"] == "e4m3" else size
        # forward: x (and residual) in, the norm (and the sum) out.  Backward: the sum, both
        # gradients that arrive in, the gradient of x out
        return {"bytes": n * size * (1 + 2 * res) + n * one + 4 * c + 4 * case["rows"]
                + ((n * size * (3 + res) + 8 * c + 4 * case["rows"]) if train else 0), "flops": n * (15 if train else 5)}
    q_len, past = _lengths(case)
    k_len = [a + b for a, b in zip(q_len, past)]
    tq, tk, h, hk, d = sum(q_len), sum(k_len), case["heads"], case["kv_heads"], case["dim"]
    rows, states, side = tq * h * d * size, tk * hk * d * size, 4 * tq * h
    small = 8 * (case["sequences"] + 1) + (tk if case["masked"] else 0)
    pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(q_len, past)) * h * (1 - case["masked"])
    # forward: q, k, v in, out and the rows' log sums out; two products.  Backward: q, k, v, out,
    # its gradient and the log sums in, three gradients out; five products
    return {"bytes": 2 * rows + 2 * states + side + small + ((4 * rows + 4 * states + side + small) if train else 0),
            "flops": pairs * d * 2 * (7 if train else 2)}


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

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda", dtype=torch.float64)

    s = {"case": dict(case)}
    if case["op"] == "emb":
        n, v, c = case["rows"], case["table"], case["channels"]
        s["table"] = normal(v, c)
        # common species and tokens come first; what is absent (padding) has the index -1
        index = (v * uniform(n) ** case["skew"]).long().clamp(max=v - 1)
        index = torch.where(uniform(n) < case["absent"], torch.full_like(index, -1), index)
        s["index"] = index.to(torch.int64 if case["index"] == "i64" else torch.int32)
        s["scale"] = math.sqrt(c) if case["scaled"] else 1.0
        s["grad"] = normal(n, c) if train else None
        return s
    if case["op"] == "rms":
        n, c = case["rows"], case["channels"]
        s["x"] = normal(n, c)
        s["residual"] = normal(n, c, scale=2.0) if case["residual"] else None
        s["weight"] = normal(c, scale=0.2, shift=1.0, dtype=torch.float32)
        s["grad"] = normal(n, c) if train else None
        s["grad_sum"] = normal(n, c) if train and case["residual"] else None
        return s

    def index(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    q_len, past = _lengths(case)
    k_len = [a + b for a, b in zip(q_len, past)]
    held = [v + case["spare"] for v in k_len]
    tq, tk, h, hk, d = sum(q_len), sum(held), case["heads"], case["kv_heads"], case["dim"]
    s["q_ptr"], s["k_ptr"] = index(_ptr(q_len)), index(_ptr(held))
    s["k_len"] = index(k_len) if case["spare"] else None
    if case["past_most"]:
        s["q"] = normal(tq, h, d, scale=1.5)
        kv = normal(tk, 2, hk, d)  # a cache of keys and values
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
    else:
        qkv = normal(tq, h + 2 * hk, d)  # out of one projection
        s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
    s["mask"] = (uniform(tk) >= case["masked"]).to(torch.uint8) if case["masked"] else None
    s["rng"] = torch.tensor([int(seed) * 0x9E3779B97F4A7C1 + 12345 & (1 << 62) - 1, int(seed) + 1], dtype=torch.int64,
                            device="cuda")
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
        return {"emb": _own_emb, "rms": _own_rms, "causal": _own_causal}[op](state)
    return {"emb": _plain_emb, "rms": _plain_rms, "causal": _plain_causal}[op](state)


def _own_emb(s):
    import cg_tensor_product_amd as oeq
    out = {"out": oeq.oeq_embedding_fwd(s["table"], s["index"], scale=s["scale"])}
    if s["grad"] is not None:
        out["grad_table"] = oeq.oeq_embedding_bwd(s["index"], s["grad"], s["case"]["table"], scale=s["scale"])
    return out


def _own_rms(s):
    import cg_tensor_product_amd as oeq
    if s["case"]["out"] == "e4m3":
        y, scale, rstd, total = oeq.oeq_rms_norm_e4m3_fwd(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        out = {"y": y, "scale": scale, "rstd": rstd}
    else:
        y, rstd, total = oeq.oeq_rms_norm_fwd(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        out = {"y": y, "rstd": rstd}
    if s["residual"] is not None:
        out["sum"] = total
    if s["grad"] is not None:
        out["grad_x"], out["grad_weight"] = oeq.oeq_rms_norm_bwd(total, rstd, s["grad"], s["weight"],
                                                                 grad_sum=s["grad_sum"])
    return out


def _own_causal(s):
    import cg_tensor_product_amd as oeq
    kw = {"scale": s["scale"], "key_mask": s["mask"], "p_drop": s["case"]["p"],
          "rng": s["rng"] if s["case"]["p"] else None}
    out, lse = oeq.oeq_causal_attn_fwd(s["q"], s["k"], s["v"], s["q_ptr"], s["k_ptr"], k_len=s["k_len"], **kw)
    got = {"out": out, "lse": lse}
    if s["grad"] is not None:
        got["grad_q"], got["grad_k"], got["grad_v"] = oeq.oeq_causal_attn_bwd(
            s["q"], s["k"], s["v"], s["q_ptr"], s["k_ptr"], out, lse, s["grad"], **kw)
    return got


# ---- plain forms -------------------------------------------------------------

def _plain_emb(s):
    c, dt = s["case"], s["table"].dtype
    index = s["index"].long()
    real = (index >= 0) & (index < c["table"])
    at = torch.where(real, index, torch.zeros_like(index))
    rows = s["table"][at].float() * s["scale"]
    out = {"out": rows.masked_fill(~real[:, None], 0.0).to(dt)}
    if s["grad"] is not None:
        # by sorted tokens: differences of the sorted rows' running sums where a token ends, in 64
        # bits, since rows are used up to tens of thousands of times (absent ones sort to the end)
        token = torch.where(real, index, torch.full_like(index, c["table"]))
        order = torch.argsort(token, stable=True)
        sums = torch.cumsum(s["grad"][order].t().contiguous().double(), 1)
        sums = torch.cat([sums.new_zeros(c["channels"], 1), sums], 1)
        uses = torch.zeros(c["table"] + 1, dtype=torch.int64, device=token.device)
        end = uses.index_add_(0, token, torch.ones_like(token)).cumsum(0)[:-1]
        first = torch.cat([end.new_zeros(1), end[:-1]])
        out["grad_table"] = (sums[:, end] - sums[:, first]).mul_(s["scale"]).t().to(dt).contiguous()
    return out


def _plain_rms(s):
    dt = s["x"].dtype
    # the sum is the residual stream: held in the inputs' type, and normalised as it is held
    total = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(dt)
    h = total.float()
    rstd = torch.rsqrt(h.square().mean(1) + EPS)
    hat = h * rstd[:, None]
    y = hat * s["weight"]
    if s["case"]["out"] == "e4m3":
        scale = y.abs().amax(1).clamp(min=2.0 ** -100) / E4M3_MOST
        out = {"y": (y / scale[:, None]).clamp(-E4M3_MOST, E4M3_MOST).to(torch.float8_e4m3fn), "scale": scale,
               "rstd": rstd}
    else:
        out = {"y": y.to(dt), "rstd": rstd}
    if s["residual"] is not None:
        out["sum"] = total
    if s["grad"] is not None:
        g = s["grad"].float()
        dhat = g * s["weight"]
        gx = rstd[:, None] * (dhat - hat * (dhat * hat).mean(1, keepdim=True))
        if s["grad_sum"] is not None:
            gx = gx + s["grad_sum"].float()
        out["grad_x"] = gx.to(dt)
        out["grad_weight"] = (g * hat).sum(0, dtype=torch.float64).float()
    return out


M32 = 0xFFFFFFFF


def _philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
    SC 2011) of 32-bit words held in int64, whose products wrap to the right 64 bits."""
    for i in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & M32 ^ c1 ^ (k0 + i * 0x9E3779B9 & M32), b & M32,
                          (a >> 32) & M32 ^ c3 ^ (k1 + i * 0xBB67AE85 & M32), a & M32)
    return c0, c1, c2, c3


def _plain_factors(rng, p, row, cols):
    """Dropout factors [*row.shape, cols]: 0 where dropped, 1 / (share kept) elsewhere.  Eight
    columns take the eight 16-bit parts of the block with counter (column / 8, row, offset) and
    key seed; a part below the threshold drops its column."""
    block = torch.arange((cols + 7) // 8, device=row.device)
    seed, offset = rng[0], rng[1]
    c0, c1 = torch.broadcast_tensors(block, row[..., None])
    words = _philox(c0, c1, torch.full_like(c0, 0) + (offset & M32), torch.full_like(c0, 0) + ((offset >> 32) & M32),
                    seed & M32, (seed >> 32) & M32)
    parts = torch.stack([part for w in words for part in (w & 0xFFFF, w >> 16)], -1).flatten(-2)[..., :cols]
    t = min(65535, int(p * 65536 + 0.5))
    return (parts >= t).float() * (65536.0 / (65536 - t))


def _plain_causal(s):
    c, dt, dev = s["case"], s["q"].dtype, s["q"].device
    h, hk, d = c["heads"], c["kv_heads"], c["dim"]
    b, g, lq, lk = c["sequences"], h // hk, s["q_most"], s["k_most"]
    q_ptr, k_ptr = s["q_ptr"].long(), s["k_ptr"].long()
    q_len, k_len = q_ptr[1:] - q_ptr[:-1], k_ptr[1:] - k_ptr[:-1] if s["k_len"] is None else s["k_len"].long()
    # pad both sides to the longest: [sequences, longest] row numbers and which of them are real
    q_no, k_no = torch.arange(lq, device=dev), torch.arange(lk, device=dev)
    q_real, k_real = q_no < q_len[:, None], k_no < k_len[:, None]
    q_at = (q_ptr[:-1, None] + q_no).clamp(max=s["q"].shape[0] - 1)
    k_at = (k_ptr[:-1, None] + k_no).clamp(max=s["k"].shape[0] - 1)
    there = k_real if s["mask"] is None else k_real & (s["mask"][k_at] != 0)
    # the last query sees all states, the one before it all but the last, and so on
    sees = k_no <= (q_no[None, :, None] + (k_len - q_len)[:, None, None])
    sees = (sees & there[:, None, :]).repeat(1, g, 1)[:, None]  # [sequences, 1, heads that share x queries, states]

    def padded(t, at, real):  # [sequences, kv heads, rows (with the shared heads), dim] in 32 bits
        t = t[at].float().masked_fill(~real[:, :, None, None], 0.0)
        return t.view(b, at.shape[1], hk, -1, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)

    q, k, v = padded(s["q"], q_at, q_real), padded(s["k"], k_at, there), padded(s["v"], k_at, there)
    scores = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"])
    scores.masked_fill_(~sees, -math.inf)
    top = scores.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    prob = scores.sub_(top).exp_()
    total = prob.sum(3, keepdim=True)
    prob = prob.div_(total.clamp(min=1e-37))
    lse = (total.log() + top).view(b, h, lq).transpose(1, 2)[q_real]
    factors = None
    if c["p"]:
        row = ((q_ptr[:-1, None] + q_no)[:, None, :] * h + torch.arange(h, device=dev)[None, :, None]).reshape(b, hk, -1)
        factors = _plain_factors(s["rng"], c["p"], row, lk)

    def stacked(t, heads, real):  # back to the real rows of all sequences, in the inputs' type
        return t.reshape(b, heads, real.shape[1], d).transpose(1, 2)[real].to(dt)

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
    if case["op"] == "emb":
        out = torch.zeros(case["rows"], case["channels"], dtype=f8, device="cuda")
        used = torch.nonzero(s["index"] >= 0)[:, 0]
        tokens = s["index"][used].long()
        out[used] = s["table"].to(f8)[tokens] * s["scale"]
        if s["grad"] is None:
            return {"out": out}
        grad = torch.zeros(case["table"], case["channels"], dtype=f8, device="cuda")
        grad.index_add_(0, tokens, s["grad"][used].to(f8), alpha=s["scale"])
        return {"out": out, "grad_table": grad}

    if case["op"] == "rms":
        x = s["x"].to(f8)
        total = x if s["residual"] is None else (x + s["residual"].to(f8)).to(s["x"].dtype).to(f8)
        rstd = ((total ** 2).sum(1) / case["channels"] + EPS) ** -0.5
        w = s["weight"].to(f8)
        out = {"rstd": rstd}
        y = total * rstd[:, None] * w
        if case["out"] == "e4m3":
            out["scale"] = torch.maximum(y.amax(1), -y.amin(1)) / E4M3_MOST
            out["y"] = y / out["scale"][:, None]
        else:
            out["y"] = y
        if s["residual"] is not None:
            out["sum"] = total
        if s["grad"] is not None:
            g = s["grad"].to(f8)
            inner = (g * w * total).sum(1, keepdim=True) / case["channels"]
            gx = (g * w - total * inner * rstd[:, None] ** 2) * rstd[:, None]
            out["grad_x"] = gx if s["grad_sum"] is None else gx + s["grad_sum"].to(f8)
            out["grad_weight"] = torch.einsum("nc,nc,n->c", g, total, rstd)
        return out

    h, share, p = case["heads"], case["heads"] // case["kv_heads"], case["p"]
    q_ptr, k_ptr = s["q_ptr"].tolist(), s["k_ptr"].tolist()
    ends = k_ptr[1:] if s["k_len"] is None else [a + n for a, n in zip(k_ptr, s["k_len"].tolist())]

    def factors(row, cols):
        """The dropout factors of the rows numbered `row`, with every 32-bit product formed from
        16-bit halves."""
        key, off = int(s["rng"][0]), int(s["rng"][1])
        t = min(65535, int(p * 65536 + 0.5))
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

    got = {"out": torch.zeros(s["q"].shape, dtype=f8, device="cuda"),
           "lse": torch.full(s["q"].shape[:2], -math.inf, dtype=f8, device="cuda")}
    if s["grad"] is not None:
        got.update({n: torch.zeros(s[n[-1]].shape, dtype=f8, device="cuda") for n in ("grad_q", "grad_k", "grad_v")})
    for a0, a1, b0, b1 in zip(q_ptr, q_ptr[1:], k_ptr, ends):
        hidden = torch.ones(a1 - a0, b1 - b0, device="cuda").triu((b1 - b0) - (a1 - a0) + 1) != 0
        if s["mask"] is not None:
            hidden |= s["mask"][b0:b1] == 0
        for j in range(h):
            q, k, v = s["q"][a0:a1, j].to(f8), s["k"][b0:b1, j // share].to(f8), s["v"][b0:b1, j // share].to(f8)
            z = (q @ k.T * s["scale"]).masked_fill_(hidden, -math.inf)
            got["lse"][a0:a1, j] = torch.logsumexp(z, 1)
            prob = torch.exp(z - got["lse"][a0:a1, j, None]).nan_to_num_(0.0)  # a row that sees nothing: -inf + inf
            f = factors(torch.arange(a0, a1, device="cuda") * h + j, b1 - b0) if p else 1.0
            got["out"][a0:a1, j] = (prob * f) @ v
            if s["grad"] is None:
                continue
            go = s["grad"][a0:a1, j].to(f8)
            gp = go @ v.T * f
            gz = prob * (gp - (gp * prob).sum(1, keepdim=True)) * s["scale"]
            got["grad_q"][a0:a1, j] = gz @ k
            got["grad_k"][b0:b1, j // share] += gz.T @ q
            got["grad_v"][b0:b1, j // share] += (prob * f).T @ go
    return got
