"""Float64 oracle of the operators over sequences (test infrastructure only).

The recurrences are those of seed_oracle.dense_step, a token at a time; the
backward pass is the chain rule through each token with every state kept;
the group norm is its formula.  Numpy only, no code shared with the GPU path.
"""
from __future__ import annotations

import numpy as np


def _token(rule, S, k, v, g, beta):
    """One update of [H, d_k, d_v] states: decayed state, miss, written, new."""
    kept = S * (g[:, :, None] if rule == "kda" else g[:, None, None])
    if rule == "mamba2":
        miss = u = v
    else:
        miss = v - np.einsum("hij,hi->hj", kept, k)
        u = beta[:, None] * miss
    return kept, miss, u, kept + k[:, :, None] * u[:, None, :]


def scan(rule, q, k, v, g, beta, S0, offsets):
    """o [T, H, d_v] (NaN outside the sequences) and the last states
    [n, H, d_k, d_v].  q, k [T, key_heads, d_k]; offsets: n + 1 integers."""
    T, H, d_v = v.shape
    per = H // q.shape[1]
    q, k = np.repeat(q, per, 1), np.repeat(k, per, 1)
    n = len(offsets) - 1
    S = np.zeros((n, H, q.shape[-1], d_v)) if S0 is None else S0.copy()
    o = np.full((T, H, d_v), np.nan)
    for s in range(n):
        for t in range(offsets[s], offsets[s + 1]):
            S[s] = _token(rule, S[s], k[t], v[t], g[t], None if beta is None else beta[t])[3]
            o[t] = np.einsum("hij,hi->hj", S[s], q[t])
    return o, S


def scan_backward(rule, q, k, v, g, beta, S0, offsets, do, dS):
    """Gradients (a dict: q, k, v, g, beta, S0) of sum(o do) + sum(S dS);
    NaN outside the sequences.  g and beta are inner products; g_scale and
    beta_scale are |x| |y| / sqrt(n) of their n terms, the size such a sum of
    unrelated terms has."""
    T, H, d_v = v.shape
    HK = q.shape[1]
    per = H // HK
    q, k = np.repeat(q, per, 1), np.repeat(k, per, 1)
    n = len(offsets) - 1
    d = {"q": np.full(q.shape, np.nan), "k": np.full(k.shape, np.nan), "v": np.full(v.shape, np.nan),
         "g": np.full(g.shape, np.nan)}
    if beta is not None:
        d["beta"] = np.full(beta.shape, np.nan)
    d["g_scale"] = np.full(g.shape, np.nan)
    d["beta_scale"] = np.full(g.shape[:2], np.nan)
    d["S0"] = np.zeros((n, H, q.shape[-1], d_v)) if dS is None else dS.copy()
    for s in range(n):
        S = np.zeros((H, q.shape[-1], d_v)) if S0 is None else S0[s].copy()
        states = []
        for t in range(offsets[s], offsets[s + 1]):
            states.append(S)
            S = _token(rule, S, k[t], v[t], g[t], None if beta is None else beta[t])[3]
        D = d["S0"][s]
        for t in range(offsets[s + 1] - 1, offsets[s] - 1, -1):
            before = states[t - offsets[s]]
            kept, miss, u, new = _token(rule, before, k[t], v[t], g[t], None if beta is None else beta[t])
            d["q"][t] = np.einsum("hij,hj->hi", new, do[t])
            D = D + q[t][:, :, None] * do[t][:, None, :]
            du = np.einsum("hij,hi->hj", D, k[t])
            dk = np.einsum("hij,hj->hi", D, u)
            if rule == "mamba2":
                d["v"][t] = du
            else:
                d["beta"][t] = (du * miss).sum(-1)
                d["beta_scale"][t] = np.sqrt((du ** 2).sum(-1) * (miss ** 2).sum(-1) / d_v)
                dmiss = beta[t][:, None] * du
                d["v"][t] = dmiss
                dk = dk - np.einsum("hij,hj->hi", kept, dmiss)
                D = D - k[t][:, :, None] * dmiss[:, None, :]
            d["k"][t] = dk
            dg = (D * before).sum(-1)
            d["g"][t] = dg if rule == "kda" else dg.sum(-1)
            over = (2,) if rule == "kda" else (1, 2)
            terms = d_v if rule == "kda" else d_v * q.shape[-1]
            d["g_scale"][t] = np.sqrt((D ** 2).sum(over) * (before ** 2).sum(over) / terms)
            D = D * (g[t][:, :, None] if rule == "kda" else g[t][:, None, None])
        d["S0"][s] = D
    for name in ("q", "k"):
        d[name] = d[name].reshape(T, HK, per, -1).sum(2)
    return d


def _act(name, x):
    s = 1.0 / (1.0 + np.exp(-x))
    if name is None:
        return x, np.ones_like(x)
    return (x * s, s * (1 + x * (1 - s))) if name == "silu" else (s, s * (1 - s))


def _slope_size(name, x):
    """The size of the terms of act's derivative: SiLU's, s + x s (1 - s),
    cancels around x = -1.28."""
    s = 1.0 / (1.0 + np.exp(-x))
    return s + np.abs(x) * s * (1 - s) if name == "silu" else np.abs(_act(name, x)[1])


def group_norm(x, gate, weight, bias, eps, centered, activation, gate_first, dy=None):
    """y, or with dy the gradients (a dict: x, gate, weight, bias) of sum(y dy).
    x [rows, groups, d]; weight and bias [d] or [groups, d] or None.  The
    gradient of h is a difference of terms of size rstd |dhat| max(1, hat^2);
    x_scale is that size, which the difference
    can fall far below; gate_scale has the same of act's derivative."""
    w = np.ones(x.shape[-1]) if weight is None else weight
    b = 0.0 if bias is None else bias
    h = x * _act(activation, gate)[0] if gate_first else x
    mean = h.mean(-1, keepdims=True) if centered else 0.0
    rstd = 1 / np.sqrt(((h - mean) ** 2).mean(-1, keepdims=True) + eps)
    hat = (h - mean) * rstd
    m = hat * w + b
    if gate is None:
        y, slope = _act(activation, m)
    elif gate_first:
        y, slope = m, 1.0
    else:
        a, da = _act(activation, gate)
        y, slope = m * a, a
    if dy is None:
        return y
    dm = dy * slope
    out = {}
    if gate is not None and not gate_first:
        out["gate"] = dy * m * da
        out["gate_scale"] = np.abs(dy) * (np.abs(hat * w) + np.abs(b)) * _slope_size(activation, gate)
    shared = (0, 1) if w.ndim == 1 and np.ndim(b) <= 1 else (0,)
    out["weight"], out["bias"] = (dm * hat).sum(shared), dm.sum(shared)
    dhat = dm * w
    dh = dhat - hat * (dhat * hat).mean(-1, keepdims=True)
    if centered:
        dh = dh - dhat.mean(-1, keepdims=True)
    dh = dh * rstd
    size = (rstd * np.abs(dhat)).max(-1, keepdims=True) * np.maximum(1.0, hat * hat).max(-1, keepdims=True)
    out["x_scale"] = np.broadcast_to(size, dh.shape)
    if gate_first:
        a, da = _act(activation, gate)
        out["gate_scale"] = size * np.abs(x) * _slope_size(activation, gate)
        out["x_scale"] = size * np.abs(a)
        out["gate"], dh = dh * x * da, dh * a
    out["x"] = dh
    return out
