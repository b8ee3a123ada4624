"""The decoder operators in plain fp64 numpy: embedding lookup and its gradient, root-mean-square norm
with the residual's addition (and its rounding to e4m3), and causal attention over packed sequences,
each with its gradients.

Written from the formulas, row by row or head by head, independently of the library.  Inputs of any
float type are taken at their values in fp64; nothing is rounded but where a function says so.
"""
from __future__ import annotations

import numpy as np

from .readout import dropout_factors


# ---------------------------------------------------------------------------
# embedding
# ---------------------------------------------------------------------------

def embedding(table, index, scale=1.0, grad_out=None):
    """dict with out and, where grad_out is given, grad_table; an index outside the table names no row."""
    table = np.asarray(table, dtype=np.float64)
    index = np.asarray(index)
    r = {"out": np.zeros((index.size, table.shape[1]))}
    if grad_out is not None:
        grad_out = np.asarray(grad_out, dtype=np.float64)
        r["grad_table"] = np.zeros(table.shape)
    for i, t in enumerate(index.tolist()):
        if 0 <= t < table.shape[0]:
            r["out"][i] = scale * table[t]
            if grad_out is not None:
                r["grad_table"][t] += scale * grad_out[i]
    return r


# ---------------------------------------------------------------------------
# rms norm
# ---------------------------------------------------------------------------

def e4m3_values():
    """The non-negative finite values of e4m3 (exponent bias 7, no infinities, 0x7F is NaN), in order."""
    v = []
    for code in range(0x7F):
        e, m = code >> 3, code & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


def to_e4m3(x):
    """x rounded to the nearest e4m3 value, ties to the even code; past 448 to 448."""
    v = e4m3_values()
    a = np.minimum(np.abs(np.asarray(x, dtype=np.float64)), 448.0)
    hi = np.clip(np.searchsorted(v, a), 1, len(v) - 1)
    lo = hi - 1
    up = (a - v[lo] > v[hi] - a) | ((a - v[lo] == v[hi] - a) & (hi % 2 == 0))
    return np.sign(x) * np.where(up, v[hi], v[lo])


def rms_norm(total, weight=None, eps=1e-5, grad_out=None, grad_sum=None):
    """dict with y, rstd, scale (of the 8-bit form) for rows `total` (the sum as the residual stream holds
    it) and, where grad_out is given, grad_x and grad_weight."""
    h = np.asarray(total, dtype=np.float64)
    w = np.ones(h.shape[1]) if weight is None else np.asarray(weight, dtype=np.float64)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    hat = h * rstd[:, None]
    y = hat * w
    most = np.abs(y).max(axis=1) if h.size else np.zeros(h.shape[0])
    r = {"y": y, "rstd": rstd, "scale": np.maximum(most, 2.0 ** -100) / 448.0}
    if grad_out is not None:
        g = np.asarray(grad_out, dtype=np.float64)
        dy = g * w
        r["grad_x"] = rstd[:, None] * (dy - hat * np.mean(dy * hat, axis=1, keepdims=True))
        if grad_sum is not None:
            r["grad_x"] = r["grad_x"] + np.asarray(grad_sum, dtype=np.float64)
        r["grad_weight"] = (g * hat).sum(axis=0)
    return r


# ---------------------------------------------------------------------------
# causal attention
# ---------------------------------------------------------------------------

def causal_attn(q, k, v, q_ptr, k_ptr, scale, key_mask=None, k_len=None, p_drop=0.0, rng=None, grad_out=None):
    """dict with out [Tq, H, D] and lse [Tq, H] (-inf and a zero row where nothing is seen) and,
    where grad_out is given, grad_q, grad_k, grad_v.  Query i of n in a sequence of m states sees the
    states j <= i + m - n that key_mask [Tk] leaves; a sequence's states are the first k_len of
    k_ptr's rows, or all.  Query by query: what a query does not see is never read."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    Tq, H, D = q.shape
    share = H // k.shape[1]
    r = {"out": np.zeros((Tq, H, D)), "lse": np.full((Tq, H), -np.inf)}
    if grad_out is not None:
        g = np.asarray(grad_out, dtype=np.float64)
        r.update(grad_q=np.zeros(q.shape), grad_k=np.zeros(k.shape), grad_v=np.zeros(v.shape))
    for s in range(len(q_ptr) - 1):
        q0, q1, k0, k1 = int(q_ptr[s]), int(q_ptr[s + 1]), int(k_ptr[s]), int(k_ptr[s + 1])
        if k_len is not None:
            k1 = k0 + max(0, min(int(k_len[s]), k1 - k0))
        for i in range(q0, q1):
            at = np.arange(k0, min(k1, k0 + (i - q0) + (k1 - k0) - (q1 - q0) + 1))
            if key_mask is not None and at.size:
                at = at[np.asarray(key_mask)[at] != 0]
            if not at.size:
                continue
            for h in range(H):
                K, V = k[at, h // share], v[at, h // share]
                S = scale * (K @ q[i, h])
                top = S.max()
                lse = top + np.log(np.exp(S - top).sum())
                P = np.exp(S - lse)
                F = 1.0
                if p_drop > 0:
                    F = dropout_factors(rng[0], rng[1], p_drop, [i * H + h], k1 - k0)[0, at - k0]
                r["lse"][i, h] = lse
                r["out"][i, h] = (P * F) @ V
                if grad_out is not None:
                    G = g[i, h]
                    dP = (V @ G) * F
                    dS = P * (dP - (dP * P).sum())
                    r["grad_q"][i, h] = scale * (dS @ K)
                    r["grad_k"][at, h // share] += scale * dS[:, None] * q[i, h]
                    r["grad_v"][at, h // share] += (P * F)[:, None] * G
    return r
