"""The weights' gradients of the operators on channels, and the scan's sums
over channels, within bounds that count the kernels' own order of additions:
test_oracle_channel_sums.py shows that those reject a result that has lost a
sequence of one token or a block of channels."""
import pytest
import torch

import channel_sums
from gpu_util import f64, requires_gpu
from oracle import seed_channels as och
from sink_rank_recurrent_amd import channels
from test_gpu_selective_scan import NAMES, backward, make, outputs
from test_gpu_short_conv import MARK, check, half
from test_gpu_short_conv import make as make_conv
from test_oracle_channel_sums import CONVS, SCANS, conv_lengths, offsets_of, scan_lengths

pytestmark = [pytest.mark.gpu, requires_gpu]


def on_device(offsets):
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


def scan(offsets, W, G, N, dtype, seed):
    n, T = len(offsets) - 1, offsets[-1]
    p = make(T, W, G, N, n, dtype, seed)
    out = outputs(p, n)
    backward(p, out, True, on_device(offsets))
    h = {k: f64(v) for k, v in p.items()}
    want = och.select_backward(*(h[k] for k in NAMES), True, h["S0"], offsets, h["dy"], h["dS"],
                               (channel_sums.scan_tokens(offsets, T), channel_sums.scan_channels(W, G)),
                               0.0 if dtype == torch.float32 else half(dtype))
    for k in (*NAMES, "S0"):
        check(out["d" + k], *want[k], "d" + k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n_seq,W,G,N", SCANS)
def test_scan_of_many_sequences(n_seq, W, G, N, dtype):
    """Several blocks of channels and further segments a workgroup."""
    scan(offsets_of(scan_lengths(n_seq, N)), W, G, N, dtype, N)


@pytest.mark.parametrize("offsets,W,G,N", [([0, 1200], 200, 1, 16), ([0, 5, 700, 1500], 130, 2, 7), ([0, 90, 1001], 70, 1, 33)])
def test_scan_of_long_sequences(offsets, W, G, N):
    scan(offsets, W, G, N, torch.float32, 3)


@pytest.mark.parametrize("offsets,C", [(offsets_of(conv_lengths(n)), C) for n, C in CONVS]
                         + [([0, 3000, 3001, 7000], 520), ([0, 5000], 101), ([0, 40, 70], 2048)],
                         ids=lambda a: str(a) if isinstance(a, int) else str(len(a) - 1))
def test_convolution(offsets, C):
    T, n = offsets[-1], len(offsets) - 1
    p = make_conv(T, C, 4, n, torch.float32, 5)
    dx, dw, db = torch.empty_like(p["x"]), torch.full((C, 4), MARK, device="cuda"), torch.full((C,), MARK, device="cuda")
    channels.seed_short_conv_backward(p["dy"], p["x"], p["w"], dx, dweight=dw, dbias=db, bias=p["b"], S0=p["S0"],
                                      cu_seqlens=on_device(offsets))
    h = {k: f64(v) for k, v in p.items()}
    want = och.conv_backward(h["x"], h["w"], h["b"], h["S0"], True, offsets, h["dy"], None,
                             channel_sums.conv(offsets, T, C, C % 8 == 0))
    for name, got in (("x", dx), ("weight", dw), ("bias", db)):
        check(got, *want[name], name)
