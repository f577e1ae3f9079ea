"""The sequence oracle against the single-token oracle, central differences
and hand-made identities."""
import numpy as np
import pytest

import oracle
from oracle import seed_sequence as seq


def _inputs(rule, T, H, HK, d_k, d_v, n, rng):
    x = {"q": rng.standard_normal((T, HK, d_k)), "k": rng.standard_normal((T, HK, d_k)),
         "v": rng.standard_normal((T, H, d_v)),
         "g": rng.uniform(0.3, 1.0, (T, H, d_k) if rule == "kda" else (T, H)),
         "beta": None if rule == "mamba2" else rng.uniform(0, 1, (T, H)),
         "S0": rng.standard_normal((n, H, d_k, d_v))}
    x["k"] /= np.linalg.norm(x["k"], axis=-1, keepdims=True)
    return x


@pytest.mark.parametrize("rule", ["gdn", "kda", "mamba2"])
def test_scan_is_the_dense_step_repeated(rule):
    rng = np.random.default_rng(3)
    x = _inputs(rule, 7, 3, 3, 5, 4, 2, rng)
    offsets = [0, 5, 7]
    o, S = seq.scan(rule, **x, offsets=offsets)
    for s in range(2):
        St = x["S0"][s]
        for t in range(offsets[s], offsets[s + 1]):
            St, ot = oracle.dense_step(rule, St, x["q"][t], x["k"][t], x["v"][t], x["g"][t],
                                       None if x["beta"] is None else x["beta"][t])
            np.testing.assert_allclose(o[t], ot, rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(S[s], St, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("rule", ["gdn", "kda", "mamba2"])
@pytest.mark.parametrize("zero_gate", [False, True])
def test_scan_gradients_by_differences(rule, zero_gate):
    rng = np.random.default_rng(4)
    x = _inputs(rule, 8, 4, 2, 3, 2, 3, rng)
    if zero_gate:
        x["g"][2] = 0.0
        x["g"][6, 1] = 0.0
    offsets = [0, 4, 4, 8]
    do, dS = rng.standard_normal((8, 4, 2)), rng.standard_normal((3, 4, 3, 2))
    d = seq.scan_backward(rule, **x, offsets=offsets, do=do, dS=dS)

    def value(y):
        o, S = seq.scan(rule, **y, offsets=offsets)
        return (o * do).sum() + (S * dS).sum()

    for name, arr in x.items():
        if arr is None:
            continue
        for _ in range(6):
            at = tuple(rng.integers(0, m) for m in arr.shape)
            y = {k: None if v is None else v.copy() for k, v in x.items()}
            y[name][at] += 1e-6
            up = value(y)
            y[name][at] -= 2e-6
            diff = (up - value(y)) / 2e-6
            assert abs(diff - d[name][at]) < 1e-7 * (1 + abs(diff)), (name, at)


@pytest.mark.parametrize("gate", ["none", "after", "before"])
@pytest.mark.parametrize("activation", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("centered", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_norm_gradients_by_differences(gate, activation, centered, shared):
    rng = np.random.default_rng(5)
    shape = (4, 3, 6)
    w = (6,) if shared else (3, 6)
    x = {"x": rng.standard_normal(shape), "gate": None if gate == "none" else rng.standard_normal(shape),
         "weight": rng.standard_normal(w), "bias": rng.standard_normal(w)}
    dy = rng.standard_normal(shape)
    flags = {"eps": 1e-3, "centered": centered, "activation": activation, "gate_first": gate == "before"}
    d = seq.group_norm(**x, **flags, dy=dy)
    for name, arr in x.items():
        if arr is None:
            continue
        for _ in range(5):
            at = tuple(rng.integers(0, m) for m in arr.shape)
            y = {k: None if v is None else v.copy() for k, v in x.items()}
            y[name][at] += 1e-6
            up = (seq.group_norm(**y, **flags) * dy).sum()
            y[name][at] -= 2e-6
            diff = (up - (seq.group_norm(**y, **flags) * dy).sum()) / 2e-6
            assert abs(diff - d[name][at]) < 1e-6 * (1 + abs(diff)), (name, at)


def test_norm_statistics():
    x = np.arange(12.0).reshape(1, 2, 6)
    y = seq.group_norm(x, None, None, None, 0.0, True, None, False)
    np.testing.assert_allclose(y.mean(-1), 0, atol=1e-15)
    np.testing.assert_allclose((y * y).mean(-1), 1, rtol=1e-14)
