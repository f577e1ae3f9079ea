"""Sizes beyond a C int in the calls over sequences: refused by the binding,
which would otherwise pass on what is left of them modulo 2^32.  On the CPU:
tensors without memory, the library replaced."""
import pytest
import torch

from sink_rank_recurrent_amd import sequence

FAR = (1 << 32) + 64


class Library:
    """Takes every call and answers 0."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def calls(monkeypatch):
    library = Library()
    monkeypatch.setattr(sequence, "lib", lambda: library)
    monkeypatch.setattr(sequence, "_same_device", lambda **t: torch.device("cuda", 0))
    monkeypatch.setattr(sequence, "_need", lambda *a: None)
    monkeypatch.setattr(sequence, "_stream", lambda *a: None)
    monkeypatch.setattr(sequence, "_On", lambda device: __import__("contextlib").nullcontext())
    return library.calls


def t(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def norm(G, d):
    x = t(1, G, d)
    sequence.seed_group_norm(x, x)


def norm_backward(G, d):
    x = t(1, G, d)
    sequence.seed_group_norm_backward(x, x, x)


def norm_workspace(G, d):
    sequence.group_norm_workspace(t(1, G, d))


def scan(n, H, HK, d_k, d_v):
    ws = t(0, dtype=torch.uint8)
    q, v, g = t(n, 1, HK, d_k), t(n, 1, H, d_v), t(n, 1, H)
    sequence.seed_scan("gdn", q, q, v, g, g, v, g, workspace=ws)


def scan_backward(n, H, HK, d_k, d_v):
    ws = t(0, dtype=torch.uint8)
    q, v, g = t(n, 1, HK, d_k), t(n, 1, H, d_v), t(n, 1, H)
    sequence.seed_scan_backward("gdn", q, q, v, g, g, v, q, q, v, g, g, workspace=ws)


def scan_workspace(n, H, HK, d_k, d_v):
    sequence.scan_workspace("gdn", t(1, HK, d_k), t(1, H, d_v), n)


@pytest.mark.parametrize("call,fits,count", [(norm, (4, 64), 1), (norm_backward, (4, 64), 1), (norm_workspace, (4, 64), 1),
                                             (scan, (2, 4, 2, 64, 64), 2), (scan_backward, (2, 4, 2, 64, 64), 2),
                                             (scan_workspace, (2, 4, 2, 64, 64), 1)],
                         ids=lambda a: getattr(a, "__name__", ""))
def test_sizes_beyond_an_int(calls, call, fits, count):
    call(*fits)
    assert len(calls) == count
    for i in range(len(fits)):
        with pytest.raises(ValueError, match="2\\^31"):
            call(*fits[:i], FAR, *fits[i + 1:])
    assert len(calls) == count
