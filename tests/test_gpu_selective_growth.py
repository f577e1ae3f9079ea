"""The selective scan where states grow by more than fp32 holds over a segment
(rates and steps of the same sign) but are zero while they do: every value is
that of a walk token by token, within the float64 oracle's bounds."""
import numpy as np
import pytest
import torch

from gpu_util import requires_gpu
from oracle import seed_channels as och
from test_gpu_selective_rates import in_64_bits, offsets_of, on_device
from test_gpu_selective_scan import NAMES, backward, depth, forward, make, outputs
from test_gpu_short_conv import check

pytestmark = [pytest.mark.gpu, requires_gpu]

GROWS, GONE, BLOCKED = slice(8, 12), slice(20, 23), slice(30, 33)
HAVE = {"D", "z", "dt_bias", "S0"}


def grow(p, offsets):
    """In the channels GROWS every token multiplies a state by e^2, input comes
    in the last 15 tokens of a sequence and gradient in its first 15; in the
    channels GONE and BLOCKED that growth ends after 60 tokens, two tokens take
    e^100 or e^40 each away, and input, gradient and decay go on as usual."""
    for channels in (GROWS, GONE, BLOCKED):
        p["A"][channels] = 2.0
        p["dt_bias"][channels] = p["S0"][:, channels] = p["dS"][:, channels] = 0.0
    for lo, hi in zip(offsets, offsets[1:]):
        row = slice(lo, hi)
        p["dt"][row, GROWS] = 1.0
        p["x"][lo:hi - 15, GROWS] = 0.0
        p["dy"][lo + 15:hi, GROWS] = 0.0
        at = min(lo + 60, hi)
        for channels, step in ((GONE, -50.0), (BLOCKED, -20.0)):
            p["dt"][lo:at, channels], p["x"][lo:at, channels] = 1.0, 0.0
            p["dt"][at:at + 2, channels], p["dt"][at + 2:hi, channels] = step, -0.1
            p["dy"][lo:min(at + 2, hi), channels] = 0.0
    return p


def against_oracle(p, offsets):
    n, T, W = len(offsets) - 1, *p["x"].shape
    out = outputs(p, n)
    forward(p, out, False, on_device(offsets))
    backward(p, out, False, on_device(offsets))
    h = in_64_bits(p)
    args = [h[k] for k in NAMES]
    y, S = och.select(*args, False, h["S0"], offsets)
    check(out["y"], *y, "y")
    check(out["S"], *S, "S")
    want = och.select_backward(*args, False, h["S0"], offsets, h["dy"], h["dS"],
                               max(depth(offsets, W, p["B"].shape[1], T)))
    for k in (*NAMES, "S0"):
        if p[k] is None:
            continue
        value, off = want[k]
        if k in ("x", "dt", "S0"):
            # decays below 2^-126 are zero: e^-100 = 2^-144 is, so what the
            # tokens before GONE's two would get through them may be missing
            off = off.copy()
            if k == "S0":
                off[:, GONE] += np.abs(value[:, GONE])
            for lo, hi in zip(offsets, offsets[1:]) if k != "S0" else ():
                before = slice(lo, min(lo + 61, hi))
                off[before, GONE] += np.abs(value[before, GONE])
        check(out["d" + k], value, off, "d" + k)
    return out


@pytest.mark.parametrize("N", [5, 16, 20, 40])
@pytest.mark.parametrize("lens", [(400,), (30, 0, 300, 131)])
def test_growth_of_zeros(lens, N):
    offsets = offsets_of(lens)
    p = grow(make(offsets[-1] + 2, 70, 1, N, len(lens), torch.float32, N, HAVE), offsets)
    out = against_oracle(p, offsets)
    assert out["S"][0, GROWS].abs().min() > 0 and out["dS0"][0, GROWS].abs().min() > 0
    assert out["dS0"][-1, BLOCKED].abs().min() > 0


def test_growth_without_a_gate():
    p = grow(make(400, 70, 2, 16, 1, torch.float32, 1, {"D", "dt_bias", "S0"}), [0, 400])
    against_oracle(p, [0, 400])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_growth_leaves_other_channels_their_bits(dtype):
    offsets = [0, 400, 431]
    plain, p = (make(431, 70, 1, 16, 2, dtype, 2, HAVE) for _ in range(2))
    grow(p, offsets)
    cu = on_device(offsets)
    a, b = outputs(plain, 2), outputs(p, 2)
    for q, out in ((plain, a), (p, b)):
        forward(q, out, False, cu)
        backward(q, out, False, cu)
    rest = torch.ones(70, dtype=torch.bool, device="cuda")
    for channels in (GROWS, GONE, BLOCKED):
        rest[channels] = False
    for k in ("y", "dx", "ddt", "dz", "S", "dS0"):
        assert torch.equal(a[k][:, rest], b[k][:, rest]), k
    for k in ("dA", "dD", "ddt_bias"):
        assert torch.equal(a[k][rest], b[k][rest]), k
    assert all(torch.isfinite(t.float()).all() for t in b.values())
