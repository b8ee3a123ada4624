"""The readout operators in plain fp64 numpy: group norm with an activation over the rows of
each structure, dropout from a counter-based generator, and cross attention over ragged
structures, each with its gradients.

Written from the formulas, structure by structure and head by head, independently of the
library.  Inputs of any float type are taken at their values in fp64; nothing is rounded.
"""
from __future__ import annotations

import numpy as np

# ---------------------------------------------------------------------------
# generator and dropout
# ---------------------------------------------------------------------------

_M = (0xD2511F53, 0xCD9E8D57)
_W = (0x9E3779B9, 0xBB67AE85)


def philox4x32(counter, key, rounds: int = 10):
    """Philox4x32 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
    SC 2011): counter is four and key two arrays of 32-bit words; returns four uint64 arrays of
    32-bit words."""
    low = np.uint64(0xFFFFFFFF)
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [int(v) for v in key]
    for _ in range(rounds):
        a, b = c[0] * np.uint64(_M[0]), c[2] * np.uint64(_M[1])
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + _W[0]) & 0xFFFFFFFF, (k[1] + _W[1]) & 0xFFFFFFFF]
    return c


def drop_threshold(p: float) -> int:
    return min(65535, int(np.floor(65536 * p + 0.5)))


def dropout_factors(seed: int, offset: int, p: float, rows, n_cols: int):
    """Factor of each (row, column): 0 where dropped, else the reciprocal of the share kept."""
    rows = np.asarray(rows, dtype=np.uint64)
    n_blocks = -(-n_cols // 8)
    block = np.broadcast_to(np.arange(n_blocks, dtype=np.uint64), (rows.size, n_blocks))
    row = np.broadcast_to(rows[:, None], block.shape)
    full = lambda v: np.full(block.shape, v, dtype=np.uint64)  # noqa: E731
    seed, offset = seed & (1 << 64) - 1, offset & (1 << 64) - 1
    words = philox4x32((block, row, full(offset & 0xFFFFFFFF), full(offset >> 32)),
                       (seed & 0xFFFFFFFF, seed >> 32))
    parts = np.empty(block.shape + (8,), dtype=np.int64)
    for j in range(4):
        parts[..., 2 * j] = words[j] & np.uint64(0xFFFF)
        parts[..., 2 * j + 1] = words[j] >> np.uint64(16)
    t = drop_threshold(p)
    keep = parts.reshape(rows.size, 8 * n_blocks)[:, :n_cols] >= t
    return keep * (65536.0 / (65536 - t))


# ---------------------------------------------------------------------------
# group norm
# ---------------------------------------------------------------------------

def _act(z, act):
    """(value, slope)"""
    if act == "none":
        return z, np.ones_like(z)
    gate = 1.0 / (1.0 + np.exp(-z))
    return z * gate, gate * (1.0 + z * (1.0 - gate))


def group_norm(x, ptr, groups, weight=None, bias=None, eps=1e-5, act="none", grad_out=None):
    """dict with out, mean, rstd and, where grad_out is given, grad_x, grad_weight, grad_bias."""
    x = np.asarray(x, dtype=np.float64)
    T, C = x.shape
    w = np.ones(C) if weight is None else np.asarray(weight, dtype=np.float64)
    b = np.zeros(C) if bias is None else np.asarray(bias, dtype=np.float64)
    B = len(ptr) - 1
    r = {"out": np.zeros((T, C)), "mean": np.zeros((B, groups)), "rstd": np.zeros((B, groups))}
    if grad_out is not None:
        g = np.asarray(grad_out, dtype=np.float64)
        r.update(grad_x=np.zeros((T, C)), grad_weight=np.zeros(C), grad_bias=np.zeros(C))
    for s in range(B):
        rows = slice(int(ptr[s]), int(ptr[s + 1]))
        if rows.start == rows.stop:
            continue
        for k in range(groups):
            ch = slice(k * C // groups, (k + 1) * C // groups)
            v = x[rows, ch]
            mean = v.mean()
            rstd = 1.0 / np.sqrt(np.mean((v - mean) ** 2) + eps)
            hat = (v - mean) * rstd
            r["mean"][s, k], r["rstd"][s, k] = mean, rstd
            r["out"][rows, ch], slope = _act(hat * w[ch] + b[ch], act)
            if grad_out is not None:
                dz = g[rows, ch] * slope
                r["grad_weight"][ch] += (dz * hat).sum(0)
                r["grad_bias"][ch] += dz.sum(0)
                dh = dz * w[ch]
                r["grad_x"][rows, ch] = rstd * (dh - dh.mean() - hat * (dh * hat).mean())
    return r


# ---------------------------------------------------------------------------
# cross attention
# ---------------------------------------------------------------------------

def cross_attn(q, k, v, q_ptr, k_ptr, scale, key_mask=None, p_drop=0.0, rng=None, grad_out=None):
    """dict with out [Tq, H, D] and lse [Tq, H] (-inf and a zero row where nothing is seen) and,
    where grad_out is given, grad_q, grad_k, grad_v.  key_mask [Tk]: nonzero = seen.
    rng = (seed, offset); the dropout row of (query row i, head h) is i H + h, its column the
    key's number within its structure.  Masked keys and values are never read."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    Tq, H, D = q.shape
    share = H // k.shape[1]
    r = {"out": np.zeros((Tq, H, D)), "lse": np.full((Tq, H), -np.inf)}
    if grad_out is not None:
        g = np.asarray(grad_out, dtype=np.float64)
        r.update(grad_q=np.zeros(q.shape), grad_k=np.zeros(k.shape), grad_v=np.zeros(v.shape))
    for s in range(len(q_ptr) - 1):
        qr = np.arange(int(q_ptr[s]), int(q_ptr[s + 1]))
        k0, k1 = int(k_ptr[s]), int(k_ptr[s + 1])
        kr = np.arange(k0, k1)
        if key_mask is not None:
            kr = kr[np.asarray(key_mask[k0:k1]) != 0]
        if qr.size == 0 or kr.size == 0:
            continue
        for h in range(H):
            Q, K, V = q[qr, h], k[kr, h // share], v[kr, h // share]
            S = scale * (Q @ K.T)
            top = S.max(1, keepdims=True)
            lse = top + np.log(np.exp(S - top).sum(1, keepdims=True))
            P = np.exp(S - lse)
            F = 1.0
            if p_drop > 0:
                F = dropout_factors(rng[0], rng[1], p_drop, qr * H + h, k1 - k0)[:, kr - k0]
            r["lse"][qr, h] = lse[:, 0]
            r["out"][qr, h] = (P * F) @ V
            if grad_out is not None:
                G = g[qr, h]
                dP = (G @ V.T) * F
                dS = P * (dP - (dP * P).sum(1, keepdims=True))
                r["grad_q"][qr, h] = scale * (dS @ K)
                r["grad_k"][kr, h // share] += scale * (dS.T @ Q)
                r["grad_v"][kr, h // share] += (P * F).T @ G
    return r
