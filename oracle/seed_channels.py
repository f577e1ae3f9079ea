"""Float64 oracle of the operators on channels (test infrastructure only).

The short convolution and the selective scan by their definitions, a token at
a time, the backward passes by the chain rule through each token.  Beside each
value stands how far an evaluation in fp32 may be off: every rounding is
followed through the formulas with the terms' magnitudes (u = 2^-24 each, the
hardware's exponential and reciprocal one unit in the last place, 2 u), so the
bounds hold for any order of the sums of the stated depth.  Numpy only, no
code shared with the GPU path.
"""
from __future__ import annotations

import numpy as np

u = 2.0 ** -24


def _sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


def _sigmoid_rel(x):
    """Relative error of 1 / (1 + 2^(-x log2 e)): the argument's rounding
    (and the constant's) 2 u |x|, exponential, sum and reciprocal."""
    return (2 * np.abs(x) + 5) * u


def _silu(x):
    s = _sigmoid(x)
    return x * s, np.abs(x * s) * (_sigmoid_rel(x) + u)


def _silu_slope(x):
    """s + x s (1 - s): its terms' sizes times their errors (1 - s is off by
    the error of s)."""
    s = _sigmoid(x)
    t = x * s * (1 - s)
    off = s * _sigmoid_rel(x)
    return s + t, off + np.abs(t) * (_sigmoid_rel(x) + 3 * u) + np.abs(x) * s * (off + u) + u * (s + np.abs(t))


# ---------------------------------------------------------------- the convolution

def conv(x, w, b, S0, silu, offsets, io_u=0.0):
    """(y, its bound, S): y [T, C] (NaN outside the sequences), S [n, K-1, C]."""
    T, C = x.shape
    K, n = w.shape[1], len(offsets) - 1
    y, off = np.full((T, C), np.nan), np.zeros((T, C))
    S = np.zeros((n, K - 1, C))
    for s in range(n):
        lo, hi = offsets[s], offsets[s + 1]
        line = np.concatenate((np.zeros((K - 1, C)) if S0 is None else S0[s], x[lo:hi]))
        S[s] = line[hi - lo:]
        pre, mass = _pre(line, w, b, hi - lo)
        y[lo:hi], off[lo:hi] = pre, (K + 1) * u * mass
        if silu:
            v, e = _silu(pre)
            y[lo:hi], off[lo:hi] = v, 1.1 * (K + 1) * u * mass + e      # |silu'| < 1.1
    return y, off + io_u * (np.abs(np.nan_to_num(y)) + off), S


def _pre(line, w, b, L):
    K = w.shape[1]
    bias = np.zeros(w.shape[0]) if b is None else b
    pre, mass = np.zeros((L, w.shape[0])) + bias, np.zeros((L, w.shape[0])) + np.abs(bias)
    for j in range(K):
        pre += line[j:j + L] * w[:, j]
        mass += np.abs(line[j:j + L] * w[:, j])
    return pre, mass


def conv_backward(x, w, b, S0, silu, offsets, dy, dS, depth, io_u=0.0):
    """{name: (gradient, bound)} of x, weight, bias, S0; `depth`: additions in
    a row of the weights' sums."""
    T, C = x.shape
    K, n = w.shape[1], len(offsets) - 1
    dx, dx_off = np.full((T, C), np.nan), np.zeros((T, C))
    dw, dw_off, dw_mass = np.zeros((C, K)), np.zeros((C, K)), np.zeros((C, K))
    db, db_off, db_mass = np.zeros(C), np.zeros(C), np.zeros(C)
    dS0, dS0_off = np.zeros((n, K - 1, C)), np.zeros((n, K - 1, C))
    for s in range(n):
        lo, hi = offsets[s], offsets[s + 1]
        L = hi - lo
        line = np.concatenate((np.zeros((K - 1, C)) if S0 is None else S0[s], x[lo:hi]))
        e, e_off = dy[lo:hi], np.zeros((L, C))
        if silu:
            pre, mass = _pre(line, w, b, L)
            slope, off = _silu_slope(pre)
            e_off = np.abs(e) * (off + 0.5 * (K + 1) * u * mass + u * np.abs(slope))     # |silu''| <= 1/2
            e = e * slope
        g, g_off, g_mass = (np.zeros((L + K - 1, C)) for _ in range(3))
        if dS is not None:
            g[L:] += dS[s]
            g_mass[L:] += np.abs(dS[s])
        for j in range(K):
            g[j:j + L] += e * w[:, j]
            g_off[j:j + L] += e_off * np.abs(w[:, j])
            g_mass[j:j + L] += np.abs(e * w[:, j])
            dw[:, j] += (e * line[j:j + L]).sum(0)
            dw_off[:, j] += (e_off * np.abs(line[j:j + L])).sum(0)
            dw_mass[:, j] += np.abs(e * line[j:j + L]).sum(0)
        db += e.sum(0)
        db_off += e_off.sum(0)
        db_mass += np.abs(e).sum(0)
        g_off += (K + 2) * u * g_mass
        g_off += io_u * (np.abs(g) + g_off)
        dx[lo:hi], dx_off[lo:hi] = g[K - 1:], g_off[K - 1:]
        dS0[s], dS0_off[s] = g[:K - 1], g_off[:K - 1]
    return {"x": (dx, dx_off), "weight": (dw, dw_off + (depth + 1) * u * dw_mass),
            "bias": (db, db_off + depth * u * db_mass), "S0": (dS0, dS0_off)}


# ---------------------------------------------------------------- the selective scan

def _steps(dt, dt_bias, softplus):
    """delta, its relative error, and the slope of softplus with its own."""
    v = dt if dt_bias is None else dt + dt_bias
    if not softplus:
        return v, np.full(v.shape, u), np.ones(v.shape), np.zeros(v.shape), v
    # v is rounded (|v| u through a logarithmic slope of at most 1), then the
    # exponential's argument (2 |v| u), and some 14 operations behind it
    return (np.logaddexp(v, 0), (3 * np.abs(v) + 14) * u, _sigmoid(v),
            _sigmoid_rel(v) + np.abs(v) * u, v)


def _group_rows(B, channels):
    """[T, G, N] as [T, channels, N]."""
    return np.repeat(B, channels // B.shape[1], 1)


def _forward(x, dt, A, B, dt_bias, softplus, S0, offsets):
    """Per sequence, lists over its tokens of h, magnitudes and errors."""
    delta, d_rel, slope, slope_rel, v = _steps(dt, dt_bias, softplus)
    channels, N = A.shape
    B = _group_rows(B, channels)
    runs = []
    for s in range(len(offsets) - 1):
        h = np.zeros((channels, N)) if S0 is None else S0[s].copy()
        M, E = np.abs(h), np.zeros((channels, N))
        tokens = []
        for t in range(offsets[s], offsets[s + 1]):
            d = delta[t][:, None]
            a = np.exp(d * A)
            a_rel = np.abs(d * A) * (d_rel[t][:, None] + 3 * u) + 2 * u
            put = d * x[t][:, None] * B[t]
            before = (h, M, E)
            h = a * h + put
            E = a * E + a * M * a_rel + np.abs(put) * (d_rel[t][:, None] + 2 * u)
            M = a * M + np.abs(put)
            E = E + u * M
            tokens.append((a, a_rel, before, (h, M, E)))
        runs.append((tokens, (h, M, E)))
    return delta, d_rel, slope, slope_rel, v, runs


def _read(C, h, M, E, N):
    """C.h, its magnitude and error (N products and sums)."""
    s, m = (C * h).sum(-1), np.abs(C * M).sum(-1)
    return s, m, (np.abs(C) * E).sum(-1) + (N + 1) * u * m


def select(x, dt, A, B, C, D, z, dt_bias, softplus, S0, offsets, io_u=0.0):
    """((y, bound), (S, bound)); y NaN outside the sequences."""
    T, channels = x.shape
    N, n = A.shape[1], len(offsets) - 1
    Cc = _group_rows(C, channels)
    *_, runs = _forward(x, dt, A, B, dt_bias, softplus, S0, offsets)
    y, off = np.full((T, channels), np.nan), np.zeros((T, channels))
    S, S_off = np.zeros((n, channels, N)), np.zeros((n, channels, N))
    for s in range(n):
        for t, (_, _, _, state) in zip(range(offsets[s], offsets[s + 1]), runs[s][0]):
            v, m, e = _read(Cc[t], *state, N)
            if D is not None:
                v, m = v + D * x[t], m + np.abs(D * x[t])
            e = e + 2 * u * m
            if z is not None:
                g, g_off = _silu(z[t])
                v, e = v * g, np.abs(g) * e + np.abs(v) * g_off + u * np.abs(v * g)
            y[t], off[t] = v, e
        S[s], _, S_off[s] = runs[s][1]
    return (y, off + io_u * (np.abs(np.nan_to_num(y)) + off)), (S, S_off)


def select_backward(x, dt, A, B, C, D, z, dt_bias, softplus, S0, offsets, dy, dS, depth, io_u=0.0):
    """{name: (gradient, bound)} of x, dt, A, B, C, D, z, dt_bias, S0 (NaN in
    rows outside the sequences); `depth`: additions in a row of the sums over
    tokens and of those over channels (one number: of both)."""
    over_tokens, over_channels = depth if isinstance(depth, tuple) else (depth, depth)
    T, channels = x.shape
    N, n, G = A.shape[1], len(offsets) - 1, B.shape[1]
    delta, d_rel, slope, slope_rel, v, runs = _forward(x, dt, A, B, dt_bias, softplus, S0, offsets)
    Bc, Cc = _group_rows(B, channels), _group_rows(C, channels)
    Dv = np.zeros(channels) if D is None else D

    def rows():
        return np.full((T, channels), np.nan), np.zeros((T, channels))

    dx, dx_off = rows()
    ddt, ddt_off = rows()
    dz, dz_off = rows()
    dB, dB_off = np.full((T, G, N), np.nan), np.zeros((T, G, N))
    dC, dC_off = np.full((T, G, N), np.nan), np.zeros((T, G, N))
    sums = {k: [np.zeros(shape) for _ in range(3)] for k, shape in
            (("A", (channels, N)), ("D", (channels,)), ("dt_bias", (channels,)))}   # value, error, magnitude
    dS0, dS0_off = np.zeros((n, channels, N)), np.zeros((n, channels, N))

    def add(name, value, error, mass):
        for a, b in zip(sums[name], (value, error, mass)):
            a += b

    def over(value):
        return value.reshape(G, channels // G, N).sum(1)

    for s in range(n):
        g = np.zeros((channels, N)) if dS is None else dS[s].copy()
        M, E = np.abs(g), np.zeros((channels, N))
        for t in range(offsets[s + 1] - 1, offsets[s] - 1, -1):
            a, a_rel, (h0, M0, E0), (h, Mh, Eh) = runs[s][0][t - offsets[s]]
            d, rel = delta[t][:, None], d_rel[t][:, None]
            ds, ds_off = dy[t], np.zeros(channels)
            if z is not None:
                gate, gate_off = _silu(z[t])
                ds, ds_off = dy[t] * gate, np.abs(dy[t]) * (gate_off + u * np.abs(gate))
                r, m, e = _read(Cc[t], h, Mh, Eh, N)
                r, m, e = r + Dv * x[t], m + np.abs(Dv * x[t]), e
                e = e + 2 * u * m
                sl, sl_off = _silu_slope(z[t])
                dz[t] = dy[t] * r * sl
                dz_off[t] = np.abs(dy[t]) * (e * np.abs(sl) + np.abs(r) * sl_off) + 3 * u * np.abs(dz[t])
            g = g + ds[:, None] * Cc[t]
            E = E + ds_off[:, None] * np.abs(Cc[t]) + u * np.abs(ds[:, None] * Cc[t])
            M = M + np.abs(ds[:, None] * Cc[t])
            E = E + u * M
            dC[t] = over(ds[:, None] * h)
            dC_off[t] = over(np.abs(ds)[:, None] * Eh + ds_off[:, None] * np.abs(h)
                             + (over_channels + 1) * u * np.abs(ds[:, None] * h))
            put = d * x[t][:, None]
            dB[t] = over(g * put)
            dB_off[t] = over(np.abs(put) * (E + M * (rel + (over_channels + 2) * u)))
            du, du_m, du_off = _read(Bc[t], g, M, E, N)
            rate, rate_m = g * a * h0, M * a * M0
            rate_off = a * (E * M0 + M * E0) + rate_m * (a_rel + 2 * u)
            size = np.abs(d)
            add("A", d * rate, size * rate_off + size * rate_m * (rel + u), size * rate_m)
            step = x[t] * du + (A * rate).sum(-1)
            step_m = np.abs(x[t]) * du_m + np.abs(A * rate_m).sum(-1)
            step_off = np.abs(x[t]) * du_off + (np.abs(A) * rate_off).sum(-1) + (N + 6) * u * step_m
            ddt[t] = step * slope[t]
            ddt_off[t] = slope[t] * (step_off + step_m * (slope_rel[t] + u))
            add("dt_bias", ddt[t], ddt_off[t], slope[t] * step_m)
            dx[t] = delta[t] * du + Dv * ds
            size = np.abs(delta[t])
            dx_off[t] = (size * (du_off + du_m * d_rel[t]) + np.abs(Dv) * ds_off
                         + 3 * u * (size * du_m + np.abs(Dv * ds)))
            add("D", ds * x[t], ds_off * np.abs(x[t]), np.abs(ds * x[t]))
            g, E, M = a * g, a * E + a * M * (a_rel + u), a * M
        dS0[s], dS0_off[s] = g, E

    def io(value, off):
        return value, off + io_u * (np.abs(np.nan_to_num(value)) + off)

    out = {k: (a, e + (over_tokens + 1) * u * m) for k, (a, e, m) in sums.items()}
    out.update(x=io(dx, dx_off), dt=io(ddt, ddt_off), z=io(dz, dz_off), B=io(dB, dB_off), C=io(dC, dC_off),
               S0=(dS0, dS0_off))
    return out
