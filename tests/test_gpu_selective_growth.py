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
from test_gpu_short_conv import TINY, check

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


def against_oracle(p, offsets, softplus=False, gone=slice(0), wider=1.0):
    n, T, W = len(offsets) - 1, *p["x"].shape
    out = outputs(p, n)
    forward(p, out, softplus, on_device(offsets))
    backward(p, out, softplus, on_device(offsets))
    h = in_64_bits(p)
    sums = max(depth(offsets, W, p["B"].shape[1], T))

    def oracle(S0):
        args = [h[k] for k in NAMES]
        y, S = och.select(*args, softplus, S0, offsets)
        return {"y": y, "S": S, **{"d" + k: v for k, v in och.select_backward(
            *args, softplus, S0, offsets, h["dy"], h["dS"], sums).items()}}

    want = oracle(h["S0"])
    missing = {k: np.zeros_like(v) for k, (v, _) in want.items()}
    # A given state below the smallest normal number may be flushed to 0 and
    # what has grown of it be missing: by how much each output is changed by it
    # (they are linear in the states).
    for i in zip(*np.nonzero((h["S0"] != 0) & (np.abs(h["S0"]) < TINY))):
        less = h["S0"].copy()
        less[i] = 0
        for k, (v, _) in oracle(less).items():
            missing[k] += np.abs(v - want[k][0])
    # Decays below 2^-126 are zero: e^-100 = 2^-144 is, so what the tokens before
    # the two of the channels `gone` would get through them may be missing.
    missing["dS0"][:, gone] += np.abs(want["dS0"][0][:, gone])
    for lo, hi in zip(offsets, offsets[1:]):
        before = slice(lo, min(lo + 61, hi))
        for k in ("dx", "ddt"):
            missing[k][before, gone] += np.abs(want[k][0][before, gone])
    for k, (v, off) in want.items():
        if k in out:
            check(out[k], v, wider * off + np.nan_to_num(missing[k]), k)
    return out


@pytest.mark.parametrize("N", [5, 16, 20, 40])
@pytest.mark.parametrize("lens", [(400,), (30, 0, 300, 131)])
def test_growth_of_zeros(lens, N):
    offsets = offsets_of(lens)
    p = grow(make(offsets[-1] + 2, 70, 1, N, len(lens), torch.float32, N, HAVE), offsets)
    out = against_oracle(p, offsets, gone=GONE)
    assert out["S"][0, GROWS].abs().min() > 0 and out["dS0"][0, GROWS].abs().min() > 0
    assert out["dS0"][-1, BLOCKED].abs().min() > 0


def test_growth_without_a_gate():
    p = grow(make(400, 70, 2, 16, 1, torch.float32, 1, {"D", "dt_bias", "S0"}), [0, 400])
    against_oracle(p, [0, 400], gone=GONE)


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


@pytest.mark.parametrize("N", [5, 16, 40])
def test_growth_through_softplus(N):
    """Rates of both signs in one call: only waves with a positive one look for
    growth."""
    offsets = [0, 400, 401, 531]
    p = make(531, 140, 2, N, 3, torch.float32, N, HAVE | {"softplus"})
    p["A"][GROWS, ::2] = 2.0
    p["S0"][:, GROWS] = p["dS"][:, GROWS] = 0.0
    p["dt_bias"][GROWS], p["dt"][:, GROWS] = 0.0, 1.0
    for lo, hi in zip(offsets, offsets[1:]):
        p["x"][lo:hi - 15, GROWS] = 0.0
        p["dy"][lo + 15:hi, GROWS] = 0.0
    against_oracle(p, offsets, softplus=True)


@pytest.mark.parametrize("N", [5, 16])
def test_growth_of_small_states(N):
    """Given states of 1e-36 grow by e^140 over 70 tokens, more than fp32 holds,
    to what it does hold; gradients of 1e-30 likewise on the way back."""
    offsets = [0, 300, 500]
    p = make(500, 70, 1, N, 2, torch.float32, N, HAVE)
    p["A"][GROWS] = 2.0
    p["dt_bias"][GROWS] = 0.0
    p["S0"][:, GROWS] *= 1e-36
    p["dS"][:, GROWS] *= 1e-30
    p["dy"][:, GROWS] *= 1e-30
    p["dt"][:, GROWS] = -0.1
    for lo in offsets[:-1]:
        p["dt"][lo:lo + 70, GROWS], p["x"][lo:lo + 70, GROWS] = 1.0, 0.0
    # A segment's multiplier is 2^(A s), s the running sum of its steps: up to
    # 128 additions, each off by u s.  The oracle's bound follows tokens alone,
    # at least 10 u of a state's magnitude for each of the 70 that grow: 700 u.
    # The sums add A u (70^2 / 2 + 58 x 70) = 13 000 u in the segment with the
    # growth and A u 128 x 13 / 2 = 1700 u in each behind it, less than 17 000 u
    # in all; on the way, t tokens into the growth, 10 t u against at most 128 A t u.
    # So 26 times the bound holds, for products of states and gradients as well.
    out = against_oracle(p, offsets, wider=26)
    assert out["S"][:, GROWS].abs().max() > 1 and out["dS0"][:, GROWS].abs().min() > 0
