"""The oracle of the operators on channels against closed forms, torch's own
autograd through the definitions, and central differences."""
import numpy as np
import pytest
import torch

from oracle import seed_channels as och


def test_conv_by_hand():
    """Two taps on one channel: y_t = w0 x_{t-1} + w1 x_t, and what is kept."""
    x = np.array([[1.0], [2.0], [3.0], [5.0]])
    w = np.array([[10.0, 1.0]])
    y, off, S = och.conv(x, w, np.array([0.5]), np.array([[[7.0]], [[9.0]], [[4.0]]]), False, [0, 3, 3, 4])
    assert y[:, 0].tolist() == [71.5, 12.5, 23.5, 45.5]
    assert S[:, 0, 0].tolist() == [3.0, 9.0, 5.0]
    assert (off >= 0).all()


def test_short_sequences_pass_the_state_on():
    x = np.arange(1.0, 3.0)[:, None]
    S0 = np.array([[[-3.0], [-2.0], [-1.0]]])
    _, _, S = och.conv(x, np.ones((1, 4)), None, S0, False, [0, 2])
    assert S[0, :, 0].tolist() == [-1.0, 1.0, 2.0]


def test_select_decays_and_integrates():
    """One state: h_t = e^(-1/2) h + x / 2 from 2; a rate of zero adds up."""
    x, dt = np.ones((3, 2)), np.full((3, 2), 0.5)
    A = np.array([[-1.0], [0.0]])
    one = np.ones((3, 1, 1))
    S0 = np.full((1, 2, 1), 2.0)
    (y, _), (S, _) = och.select(x, dt, A, one, one, None, None, None, False, S0, [0, 3])
    a = np.exp(-0.5)
    h = 2.0
    for t in range(3):
        h = a * h + 0.5
        assert abs(y[t, 0] - h) < 1e-15 and abs(y[t, 1] - (2.5 + 0.5 * t)) < 1e-15
    assert np.allclose(S[0, :, 0], [h, 3.5])


def test_softplus_of_far_values():
    delta, *_ = och._steps(np.array([[-80.0, 0.0, 80.0]]), None, True)
    assert np.allclose(delta, [[np.exp(-80.0), np.log(2.0), 80.0]], rtol=1e-15)


def _make(seed=0, T=9, channels=6, G=2, N=3, n=3):
    rng = np.random.default_rng(seed)
    r = rng.standard_normal
    return {"x": r((T, channels)), "dt": r((T, channels)) - 1, "A": -np.exp(0.5 * r((channels, N))),
            "B": r((T, G, N)), "C": r((T, G, N)), "D": r(channels), "z": r((T, channels)),
            "dt_bias": 0.3 * r(channels), "S0": r((n, channels, N))}, r((T, channels)), r((n, channels, N))


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("leave", [(), ("D", "z", "dt_bias", "S0")])
def test_select_backward_is_autograd(softplus, leave):
    p, dy, dS = _make()
    if not softplus:
        p["dt"] = np.abs(p["dt"])
    for k in leave:
        p[k] = None
    offsets = [0, 4, 4, 9]
    got = och.select_backward(*(p[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")), softplus, p["S0"],
                              offsets, dy, dS, 4)
    t = {k: None if v is None else torch.tensor(v, requires_grad=True) for k, v in p.items()}
    total = torch.zeros((), dtype=torch.float64)
    for s in range(3):
        h = torch.zeros(6, 3, dtype=torch.float64) if t["S0"] is None else t["S0"][s]
        for i in range(offsets[s], offsets[s + 1]):
            v = t["dt"][i] if t["dt_bias"] is None else t["dt"][i] + t["dt_bias"]
            d = torch.nn.functional.softplus(v) if softplus else v
            h = torch.exp(d[:, None] * t["A"]) * h + (d * t["x"][i])[:, None] * t["B"][i].repeat_interleave(3, 0)
            y = (h * t["C"][i].repeat_interleave(3, 0)).sum(-1)
            if t["D"] is not None:
                y = y + t["D"] * t["x"][i]
            if t["z"] is not None:
                y = y * torch.nn.functional.silu(t["z"][i])
            total = total + (y * torch.tensor(dy[i])).sum()
        total = total + (h * torch.tensor(dS[s])).sum()
    total.backward()
    for k, v in t.items():
        if v is not None:
            assert np.allclose(got[k][0], v.grad.numpy(), rtol=1e-12, atol=1e-13), k


@pytest.mark.parametrize("silu", [True, False])
def test_conv_backward_is_autograd(silu):
    rng = np.random.default_rng(1)
    x, w, b, S0 = (rng.standard_normal(s) for s in ((9, 5), (5, 4), (5,), (3, 3, 5)))
    dy, dS = rng.standard_normal((9, 5)), rng.standard_normal((3, 3, 5))
    offsets = [0, 2, 2, 9]
    got = och.conv_backward(x, w, b, S0, silu, offsets, dy, dS, 4)
    t = [torch.tensor(v, requires_grad=True) for v in (x, w, b, S0)]
    total = torch.zeros((), dtype=torch.float64)
    for s in range(3):
        line = torch.cat((t[3][s], t[0][offsets[s]:offsets[s + 1]]))
        L = offsets[s + 1] - offsets[s]
        pre = sum(line[j:j + L] * t[1][:, j] for j in range(4)) + t[2]
        y = torch.nn.functional.silu(pre) if silu else pre
        total = total + (y * torch.tensor(dy[offsets[s]:offsets[s + 1]])).sum() + (line[L:] * torch.tensor(dS[s])).sum()
    total.backward()
    for k, v in zip(("x", "weight", "bias", "S0"), t):
        assert np.allclose(got[k][0], v.grad.numpy(), rtol=1e-12, atol=1e-13), k


def test_select_backward_is_a_difference():
    p, dy, dS = _make(3)
    offsets = [0, 4, 4, 9]
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")
    got = och.select_backward(*(p[k] for k in names), True, p["S0"], offsets, dy, dS, 4)
    rng = np.random.default_rng(4)
    along = {k: rng.standard_normal(v.shape) for k, v in p.items()}

    def loss(h):
        q = {k: v + h * along[k] for k, v in p.items()}
        (y, _), (S, _) = och.select(*(q[k] for k in names), True, q["S0"], offsets)
        return (y * dy).sum() + (S * dS).sum()

    want = (loss(1e-5) - loss(-1e-5)) / 2e-5
    have = sum((got[k][0] * along[k]).sum() for k in p)
    assert abs(have - want) < 1e-7 * max(1.0, abs(want))


def _round(x):
    return x.astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("seed", range(3))
def test_bounds_hold_for_fp32(seed):
    """The definitions evaluated in fp32 by torch stay within the bounds, and
    the bounds are no wider than some hundred roundings of the values' sizes."""
    p, _, _ = _make(seed, T=40, channels=8, G=2, N=5, n=1)
    p = {k: _round(v) for k, v in p.items()}
    (y, off), (S, S_off) = och.select(*(p[k] for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")), True,
                                      p["S0"], [0, 40])
    f = {k: torch.tensor(v, dtype=torch.float32) for k, v in p.items()}
    h = f["S0"][0]
    for i in range(40):
        d = torch.nn.functional.softplus(f["dt"][i] + f["dt_bias"])
        h = torch.exp(d[:, None] * f["A"]) * h + (d * f["x"][i])[:, None] * f["B"][i].repeat_interleave(4, 0)
        v = ((h * f["C"][i].repeat_interleave(4, 0)).sum(-1) + f["D"] * f["x"][i]) * torch.nn.functional.silu(f["z"][i])
        assert (np.abs(v.double().numpy() - y[i]) <= off[i]).all()
    assert (np.abs(h.double().numpy() - S[0]) <= S_off[0]).all()
    assert off.max() < 1e-4 * np.abs(y).max()
