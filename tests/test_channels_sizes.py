"""Sizes beyond a C int in the calls of the operators on channels: refused by
the binding, which would otherwise pass on what is left of them modulo 2^32.
On the CPU: tensors without memory, and the calls themselves replaced."""
import ctypes

import pytest
import torch

from sink_rank_recurrent_amd import channels
import test_channels_abi as abi

FAR = (1 << 32) + 5


@pytest.fixture
def calls(monkeypatch):
    """The calls that get past the binding's checks."""
    made = []
    monkeypatch.setattr(channels, "_device", lambda *a: 0)
    monkeypatch.setattr(channels, "_need", lambda *a: None)
    monkeypatch.setattr(channels, "_space", lambda *a: None)
    monkeypatch.setattr(channels, "_call", lambda name, *a: made.append(name))
    return made


def t(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def conv(n, C, K, **more):
    channels.seed_short_conv(t(n, 1, C), t(C, K), t(n, 1, C), **more)


def conv_packed(n_seq):
    channels.seed_short_conv(t(3, 4), t(4, 4), t(3, 4), cu_seqlens=t(n_seq + 1, dtype=torch.int32))


def conv_backward(n, C, K):
    channels.seed_short_conv_backward(t(n, 1, C), t(n, 1, C), t(C, K), t(n, 1, C))


def conv_step(n, C, K):
    channels.seed_short_conv_step(t(n, C), t(C, K), t(n, C), t(n, K - 1, C))


def scan(n, C, G, N):
    x, bc = t(n, 1, C), t(n, 1, G, N)
    try:
        channels.seed_selective_scan(x, x, t(C, N), bc, bc, x, None)
    except AttributeError:      # (no workspace here: all checks are passed)
        channels._call("seed_selective_scan")


def scan_backward(n, C, G, N):
    x, bc = t(n, 1, C), t(n, 1, G, N)
    try:
        channels.seed_selective_scan_backward(x, x, x, t(C, N), bc, bc, x, x, None, bc, bc)
    except AttributeError:
        channels._call("seed_selective_scan_backward")


def step(n, C, G, N):
    x, bc = t(n, C), t(n, G, N)
    channels.seed_selective_step(x, x, t(C, N), bc, bc, x, None)


@pytest.mark.parametrize("call,fits,beyond", [
    (conv, (3, 4, 4), [(FAR, 4, 4), (3, FAR, 4), (3, 4, FAR)]),
    (conv_packed, (3,), [(FAR,)]),
    (conv_backward, (3, 4, 4), [(FAR, 4, 4), (3, FAR, 4), (3, 4, FAR)]),
    (conv_step, (3, 4, 4), [(FAR, 4, 4), (1 << 31, 4, 4), (3, FAR, 4), (3, 4, FAR)]),
    (scan, (3, 4, 2, 4), [(FAR, 4, 2, 4), (3, FAR, 2, 4), (3, 4, FAR, 4), (3, 4, 2, FAR)]),
    (scan_backward, (3, 4, 2, 4), [(FAR, 4, 2, 4), (3, FAR, 2, 4), (3, 4, FAR, 4), (3, 4, 2, FAR)]),
    (step, (3, 4, 2, 4), [(FAR, 4, 2, 4), (1 << 31, 4, 2, 4), (3, FAR, 2, 4), (3, 4, FAR, 4), (3, 4, 2, FAR)])],
    ids=lambda a: getattr(a, "__name__", ""))
def test_sizes_beyond_an_int(calls, call, fits, beyond):
    call(*fits)
    assert len(calls) == 1
    for sizes in beyond:
        with pytest.raises(ValueError, match="2\\^31"):
            call(*sizes)
    assert len(calls) == 1


@pytest.mark.parametrize("query", [
    lambda n: channels.short_conv_workspace(t(n, 8), t(8, 4), 1),
    lambda n: channels.short_conv_workspace(t(3, 8), t(8, 4), n),
    lambda n: channels.short_conv_workspace(t(3, 8), t(n, 4), 1),
    lambda n: channels.selective_scan_workspace(t(n, 8), t(n, 1, 16), 1),
    lambda n: channels.selective_scan_workspace(t(3, 8), t(3, 1, 16), n),
    lambda n: channels.selective_scan_workspace(t(3, 8), t(3, n, 16), 1),
    lambda n: channels.selective_scan_workspace(t(3, n), t(3, 1, 16), 1),
    lambda n: channels.selective_scan_workspace(t(3, 8), t(3, 1, n), 1)])
def test_workspaces_of_sizes_beyond_an_int(query):
    """5 in place of 2^32 + 5 would be a size that is taken."""
    assert query(4).device.type == "meta"
    with pytest.raises(ValueError, match="2\\^31"):
        query(FAR)


def test_largest_batch_of_a_selective_step():
    """Its kernel counts requests in an int, 2 x 65535 at a time: the largest
    batch that is accepted leaves that much below 2^31."""
    def call(batch):
        return abi._call("seed_selective_step", abi.STEP, dict(batch=batch, channels=1, groups=1, d_state=1,
                                                               B_stride=1, C_stride=1, x=ctypes.c_void_p(None)))
    most = (1 << 30) - 65
    assert call(most)[1].endswith("x is NULL")                  # (the sizes are taken)
    got, why = call(most + 1)
    assert got == 3 and "grid" in why
    assert most + 2 * 65535 < 1 << 31
