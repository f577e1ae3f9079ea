"""The selective scan with rates that are not ordinary: of -infinity, which
leave nothing of a state (taken as the lowest fp32 number), against the
float64 oracle with that number, within its bounds."""
import numpy as np
import pytest
import torch

from gpu_util import f64, requires_gpu
from oracle import seed_channels as och
from sink_rank_recurrent_amd import channels
from test_gpu_selective_scan import FULL, NAMES, backward, depth, forward, make, outputs
from test_gpu_short_conv import check

pytestmark = [pytest.mark.gpu, requires_gpu]

LOWEST = float(torch.finfo(torch.float32).min)


def offsets_of(lens):
    return [0, *np.cumsum(lens).tolist()]


def on_device(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


def in_64_bits(p):
    h = {k: None if v is None else f64(v) for k, v in p.items()}
    h["A"] = np.maximum(h["A"], LOWEST)
    return h


def against_oracle(p, offsets, softplus=True):
    """float32: both passes through the kernels, every output within the bounds."""
    n, T, W = len(offsets) - 1, *p["x"].shape
    out = outputs(p, n)
    forward(p, out, softplus, on_device(offsets))
    backward(p, out, softplus, on_device(offsets))
    h = in_64_bits(p)
    args = [h[k] for k in NAMES]
    y, S = och.select(*args, softplus, h["S0"], offsets)
    check(out["y"], *y, "y")
    check(out["S"], *S, "S")
    want = och.select_backward(*args, softplus, h["S0"], offsets, h["dy"], h["dS"],
                               max(depth(offsets, W, p["B"].shape[1], T)))
    for k in (*NAMES, "S0"):
        if p[k] is not None:
            check(out["d" + k], *want[k], "d" + k)
    return out


@pytest.mark.parametrize("N", [5, 16, 20, 40])
@pytest.mark.parametrize("lens", [(9,), (1, 0, 8, 15), (300,), (130, 257)])
def test_rate_of_minus_infinity(lens, N):
    """Whole sequences and segments, of lengths on and off the tiles of 8."""
    offsets = offsets_of(lens)
    p = make(offsets[-1], 70, 1, N, len(lens), torch.float32, N)
    p["A"][3], p["A"][10:, N // 2] = -float("inf"), -float("inf")
    against_oracle(p, offsets)


@pytest.mark.parametrize("N", [5, 16])
def test_rate_of_minus_infinity_in_many_whole_sequences(N):
    lens = [(7 * i) % 23 for i in range(200)]
    offsets = offsets_of(lens)
    p = make(offsets[-1], 130, 1, N, len(lens), torch.float32, N + 1)
    p["A"][5:9] = -float("inf")
    against_oracle(p, offsets)


@pytest.mark.parametrize("N", [3, 16])
def test_rate_of_minus_infinity_in_a_step(N):
    """A step, and a scan of nine tokens against nine steps within the sum of
    their bounds."""
    p = make(9, 70, 1, N, 1, torch.float32, N, FULL)
    p["A"][3], p["A"][10:, N // 2] = -float("inf"), -float("inf")
    out = outputs(p, 1, back=False)
    forward(p, out, True, on_device([0, 9]))
    S, y = p["S0"].clone(), torch.empty_like(out["y"])
    for t in range(9):
        row = slice(t, t + 1)
        channels.seed_selective_step(*(p[k] if k == "A" else p[k][row] for k in NAMES[:5]), y[row], S, D=p["D"],
                                     z=p["z"][row], dt_bias=p["dt_bias"])
    h = in_64_bits(p)
    (want, off), (wS, S_off) = och.select(*(h[k] for k in NAMES), True, h["S0"], [0, 9])
    check(y, want, off, "y of steps")
    check(S, wS, S_off, "S of steps")
    check(out["y"], want, off, "y")
    check(out["S"], wS, S_off, "S")


def test_steps_of_zero_leave_such_a_state():
    """softplus off, steps of zero: the states stay as they are whatever the
    rate, in the scan and in a step."""
    p = make(20, 64, 1, 16, 1, torch.float32, 2, {"S0"})
    p["dt"][:, :32], p["A"][::2] = 0.0, -float("inf")
    out = outputs(p, 1, back=False)
    forward(p, out, False, on_device([0, 20]))
    assert torch.equal(out["S"][0, :32], p["S0"][0, :32])
    S, y = p["S0"].clone(), torch.empty(1, 64, device="cuda")
    channels.seed_selective_step(*(p[k] if k == "A" else p[k][:1] for k in NAMES[:5]), y, S, softplus=False)
    assert torch.equal(S[0, :32], p["S0"][0, :32]) and torch.isfinite(S).all()


def test_rate_that_is_no_number():
    p = make(20, 64, 1, 16, 1, torch.float32, 3)
    p["A"][7, 2] = float("nan")
    out = outputs(p, 1, back=False)
    forward(p, out, True, on_device([0, 20]))
    assert torch.isnan(out["S"][0, 7, 2]) and torch.isnan(out["y"][:, 7]).all()
    assert torch.isfinite(out["y"][:, :7]).all() and torch.isfinite(out["y"][:, 8:]).all()
    assert int(torch.isnan(out["S"]).sum()) == 1
