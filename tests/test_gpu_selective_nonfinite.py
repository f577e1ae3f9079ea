"""A NaN or infinity in the inputs of the selective scan stays where the
formulas take it: of x and dt in the rest of its sequence in its channel, of z
in its value, of B in its state in the rest of its sequence in its group, of C
in its token and group.  Everything else keeps its bits, in segments and whole
sequences, for every width of states and type, in the step and backwards."""
import pytest
import torch

from gpu_util import requires_gpu
from sink_rank_recurrent_amd import channels
from test_gpu_selective_scan import FULL, NAMES, backward, forward, make, outputs

pytestmark = [pytest.mark.gpu, requires_gpu]

INF, NAN = float("inf"), float("nan")
W, G = 140, 2           # blocks of 64 and 6 channels a group
GROUP = [slice(0, 70), slice(70, 140)]
# lengths on and off the tiles of 8; the first in segments, the second whole
BATCHES = [[0, 93, 400, 600], [0, 13, 37, 60]]


def poison(p, offsets, N):
    """What is changed, and which of y and S that reaches."""
    T, n = offsets[-1], len(offsets) - 1
    y = torch.zeros(T, W, dtype=torch.bool, device="cuda")
    S = torch.zeros(n, W, N, dtype=torch.bool, device="cuda")
    lo, mid, end = offsets[:3]
    last = mid - 1
    # channels
    p["x"][lo + 5, 3] = NAN
    y[lo + 5:mid, 3], S[0, 3] = True, True
    p["dt"][last, 69] = INF                       # the last token, the last channel of a group
    y[last, 69], S[0, 69] = True, True
    p["z"][lo + 2, 80] = NAN
    y[lo + 2, 80] = True
    # the first token of the next sequence, the first group: behind a tile's end
    p["B"][mid, 0, N - 1] = INF
    y[mid:end, GROUP[0]], S[1, GROUP[0], N - 1] = True, True
    p["C"][mid, 1, 0] = INF
    y[mid, GROUP[1]] = True
    p["x"][mid, 100] = INF
    y[mid:end, 100], S[1, 100] = True, True
    # the last sequence: one token's read-outs only
    p["C"][offsets[2] + 9, 0, N // 2] = NAN
    y[offsets[2] + 9, GROUP[0]] = True
    return y, S


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [3, 5, 16, 20, 40, 64])
@pytest.mark.parametrize("offsets", BATCHES, ids=["segments", "whole"])
def test_forward(offsets, N, dtype):
    T, n = offsets[-1], len(offsets) - 1
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    p = make(T, W, G, N, n, dtype, N)
    clean, out = outputs(p, n, back=False), outputs(p, n, back=False)
    forward(p, clean, True, cu)
    y, S = poison(p, offsets, N)
    forward(p, out, True, cu)
    assert torch.isfinite(clean["y"]).all() and torch.isfinite(clean["S"]).all()
    assert torch.equal(out["y"][~y], clean["y"][~y]) and not torch.isfinite(out["y"][y]).any()
    assert torch.equal(out["S"][~S], clean["S"][~S]) and not torch.isfinite(out["S"][S]).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [3, 16, 20, 64])
def test_step(N, dtype):
    """Requests of a step: each is a sequence of its own."""
    p = make(9, W, G, N, 9, dtype, N, FULL)
    args = dict(D=p["D"], dt_bias=p["dt_bias"], S0=p["S0"])
    clean, out = outputs(p, 9, back=False), outputs(p, 9, back=False)
    channels.seed_selective_step(*(p[k] for k in NAMES[:5]), clean["y"], clean["S"], z=p["z"], **args)
    y = torch.zeros(9, W, dtype=torch.bool, device="cuda")
    S = torch.zeros(9, W, N, dtype=torch.bool, device="cuda")
    p["x"][0, 3], p["dt"][3, 69], p["z"][4, 80] = NAN, INF, NAN
    y[0, 3] = y[3, 69] = y[4, 80] = True
    S[0, 3] = S[3, 69] = True
    p["B"][5, 0, N - 1], p["C"][8, 1, 0] = INF, NAN
    y[5, GROUP[0]] = y[8, GROUP[1]] = True
    S[5, GROUP[0], N - 1] = True
    channels.seed_selective_step(*(p[k] for k in NAMES[:5]), out["y"], out["S"], z=p["z"], **args)
    assert torch.equal(out["y"][~y], clean["y"][~y]) and not torch.isfinite(out["y"][y]).any()
    assert torch.equal(out["S"][~S], clean["S"][~S]) and not torch.isfinite(out["S"][S]).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [5, 16, 40])
def test_backward(N, dtype):
    """Values of single channels and of the next sequence's first rows: the
    other channels' and the other sequences' gradients keep their bits."""
    offsets = [0, 93, 400, 600]
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    p = make(600, W, G, N, 3, dtype, N + 1)
    clean, out = outputs(p, 3), outputs(p, 3)
    backward(p, clean, True, cu)
    p["x"][5, 3], p["dt"][92, 69], p["dy"][93, 100], p["z"][94, 101] = NAN, INF, NAN, INF
    p["B"][93, 0, N - 1], p["C"][93, 1, 0], p["C"][94, 0, 1] = INF, INF, NAN
    backward(p, out, True, cu)
    ok = torch.ones(W, dtype=torch.bool, device="cuda")
    ok[3] = ok[69] = False
    for k in ("dx", "ddt", "dz"):
        assert torch.equal(out[k][:93, ok], clean[k][:93, ok]), k
        assert torch.equal(out[k][400:], clean[k][400:]), k
    assert torch.equal(out["dS0"][0, ok], clean["dS0"][0, ok]) and torch.equal(out["dS0"][2], clean["dS0"][2])
    # the first sequence's other group, and the last sequence
    for k in ("dB", "dC"):
        assert torch.equal(out[k][:93, 1], clean[k][:93, 1]) and torch.equal(out[k][400:], clean[k][400:]), k
    # what the values reach is not hidden
    assert not torch.isfinite(out["dx"][93, 100]) and not torch.isfinite(out["dA"][3]).all()
