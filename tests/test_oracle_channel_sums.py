"""The oracle's bounds of the weights' sums, counted by the kernels' order of
additions (channel_sums.py), reject results that have lost a sequence of one
token or a block of channels, at the sizes of test_gpu_channel_sums.py."""
import numpy as np
import pytest

import channel_sums
from oracle import seed_channels as och

SCANS = [(2100, 330, 1, 6), (4200, 150, 1, 16), (2100, 300, 2, 20), (4200, 130, 1, 50)]
CONVS = [(65, 16), (1000, 101), (5000, 16)]


def scan_lengths(n_seq, seed):
    """Sequences of no token or one, a few longer ones."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, 2, n_seq)
    lens[:2], lens[rng.integers(2, n_seq, 3)] = (9, 140), 17
    return lens


def conv_lengths(n_seq):
    rng = np.random.default_rng(n_seq)
    lens = rng.integers(0, 4, n_seq)
    lens[rng.integers(0, n_seq, 3)] = 70
    return lens


def offsets_of(lens):
    return [0, *np.cumsum(lens).tolist()]


def test_runs():
    assert channel_sums._runs([0, 1, 1, 300], 7) == {0: 1, 2: 128, 3: 128, 4: 43}
    assert channel_sums._most({0: 5, 2: 7, 3: 1}, 2, sum) == 12


@pytest.mark.parametrize("n_seq,W,G,N", SCANS)
def test_lost_parts_of_the_scan(n_seq, W, G, N):
    lens = scan_lengths(n_seq, N)
    offsets = offsets_of(lens)
    T = offsets[-1]
    r = np.random.default_rng(1).standard_normal
    args = [r((T, W)), r((T, W)) - 1, -np.exp(0.7 * r((W, N))), r((T, G, N)), r((T, G, N)), r(W), r((T, W)), 0.5 * r(W)]
    S0, dy, dS = r((n_seq, W, N)), r((T, W)), r((n_seq, W, N))
    depth = channel_sums.scan_tokens(offsets, T), channel_sums.scan_channels(W, G)

    def gradients(dy, dS):
        return och.select_backward(*args, True, S0, offsets, dy, dS, depth)

    want = gradients(dy, dS)

    def outside(got, name):
        return (np.abs(got[name][0] - want[name][0]) > want[name][1]).mean()

    lost = int(np.flatnonzero(lens == 1)[40])
    less_dy, less_dS = dy.copy(), dS.copy()
    less_dy[offsets[lost]] = less_dS[lost] = 0
    got = gradients(less_dy, less_dS)
    assert all(outside(got, k) > 0.5 for k in ("A", "D", "dt_bias"))
    each = W // G
    block = [g * each + c for g in range(G) for c in range((each - 1) // 64 * 64, each)]
    less_dy, less_dS = dy.copy(), dS.copy()
    less_dy[:, block] = less_dS[:, block] = 0
    got = gradients(less_dy, less_dS)
    assert all(outside(got, k) > 0.99 for k in ("B", "C"))


@pytest.mark.parametrize("n_seq,C", CONVS)
def test_lost_parts_of_the_convolution(n_seq, C):
    lens = conv_lengths(n_seq)
    offsets = offsets_of(lens)
    T = offsets[-1]
    r = np.random.default_rng(2).standard_normal
    x, w, b, S0, dy = r((T, C)), r((C, 4)) / 2, 0.3 * r(C), r((n_seq, 3, C)), r((T, C))
    depth = channel_sums.conv(offsets, T, C, C % 8 == 0)
    want = och.conv_backward(x, w, b, S0, True, offsets, dy, None, depth)
    less = dy.copy()
    less[offsets[int(np.flatnonzero(lens == 1)[5])]] = 0
    got = och.conv_backward(x, w, b, S0, True, offsets, less, None, depth)
    for k in ("weight", "bias"):
        assert (np.abs(got[k][0] - want[k][0]) > want[k][1]).mean() > 0.5, k
