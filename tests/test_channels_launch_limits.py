"""Grids of the operators on channels at the largest sizes they accept, on the
CPU: the built library with the runtime's launch call replaced by one that
writes the grid down (see test_launch_limits.py).  An accepted call has to fit:
fewer than 2^32 threads along x, at most 65535 blocks along y and z."""
import ctypes
import os
import subprocess
import sys

import pytest

from sink_rank_recurrent_amd import binding
from test_launch_limits import FAR, ROOT, recorder  # noqa: F401



def _call(name, *args):
    """`name` with "p" for an address of its own, "r" for that of an array
    over tokens and its stride, None for NULL."""
    from sink_rank_recurrent_amd import channels
    at, out = iter(range(1, 64)), []
    for a in args:
        out += [ctypes.c_void_p(next(at) * FAR)] if a in ("p", "r") and isinstance(a, str) else [a]
        if isinstance(a, str) and a == "r":
            out.append(STRIDE)
    got = getattr(channels.lib(), name)(*out)
    assert got == 0, (name, args, binding.lib().seed_last_error())


STRIDE = 1 << 12


def conv(n_seq, channels, tokens, width=4):
    global STRIDE
    STRIDE = channels
    _call("seed_short_conv", n_seq, channels, width, tokens, "p", "r", 1, "p", "p", "p", 1, "r", "p", None)


def conv_backward(n_seq, channels, tokens, width=4):
    global STRIDE
    STRIDE = channels
    _call("seed_short_conv_backward", n_seq, channels, width, tokens, "p", "r", 1, "p", "p", "p", 1, "r", "p", "r",
          "p", "p", "p", "p", FAR, None)


def conv_step(batch, channels, width=4):
    global STRIDE
    STRIDE = channels
    _call("seed_short_conv_step", batch, channels, width, "r", 1, "p", "p", "p", 1, "r", "p", None)


def scan(n_seq, channels, groups, d_state, tokens):
    global STRIDE
    STRIDE = max(channels, groups * d_state)
    _call("seed_selective_scan", n_seq, channels, groups, d_state, tokens, "p", "r", "r", "p", "r", "r", 1, "p", "r",
          "p", 1, "p", "r", "p", "p", FAR, None)


def scan_backward(n_seq, channels, groups, d_state, tokens):
    global STRIDE
    STRIDE = max(channels, groups * d_state)
    _call("seed_selective_scan_backward", n_seq, channels, groups, d_state, tokens, "p", "r", "r", "p", "r", "r", 1,
          "p", "r", "p", 1, "p", "r", "p", "r", "r", "p", "r", "r", "p", "r", "p", "p", "p", FAR, None)


def step(batch, channels, groups, d_state):
    global STRIDE
    STRIDE = max(channels, groups * d_state)
    _call("seed_selective_step", batch, channels, groups, d_state, "r", "r", "p", "r", "r", 1, "p", "r", "p", 1, "p",
          "r", "p", None)


MOST = (1 << 24) - 2
CONVS = [(1, 1 << 20, 1), (1, (1 << 20) - 1, 7), (MOST - 2, 1, 32), (1, 1, (MOST - 2) * 32), (1, 256, (MOST - 2) * 32),
         (4000, 7, 100), (1, 1 << 20, 4096)]
SCANS = [(1, 1 << 20, 1, 64, 300), (1, 65535, 65535, 1, 5), (MOST - 2, 1, 1, 16, 64), (1, 1, 1, 16, (MOST - 2) * 64),
         (65536, 64, 1, 5, 100), (1, 64 * 65535 // 64, 1, 16, 129), (3, 1 << 20, 1 << 14, 16, 100),
         (200000, 256, 4, 16, 1 << 20)]
CASES = ([("conv", a) for a in CONVS] + [("conv_backward", a) for a in CONVS] + [("scan", a) for a in SCANS]
         + [("scan_backward", a) for a in SCANS]
         + [("conv_step", a) for a in ((15 << 20, 1), (15 << 20, 256), (1, 1 << 20), (70000, 2048))]
         + [("step", a) for a in ((1 << 28, 1, 1, 1), (1, 1 << 20, 1, 64), (1 << 20, 1 << 10, 2, 16))])


@pytest.mark.parametrize("call", ["conv", "conv_backward", "conv_step", "scan", "scan_backward", "step"])
def test_largest_accepted_sizes_fit_a_grid(recorder, tmp_path, call):  # noqa: F811
    out = tmp_path / "launches"
    code = ("import sys; sys.path[:0] = ['tests']; import test_channels_launch_limits as t\n"
            f"for f, a in t.CASES:\n    if f == {call!r}:\n"
            "        print('call', f, a, file=open(sys.argv[1], 'a'))\n        getattr(t, f)(*a)\n")
    r = subprocess.run([sys.executable, "-c", code, str(out)], capture_output=True, text=True, cwd=ROOT,
                       timeout=300, env=dict(os.environ, LD_PRELOAD=recorder, SEED_LAUNCHES=str(out)))
    assert r.returncode == 0, r.stderr[-3000:]
    launches, which = 0, ""
    for line in out.read_text().splitlines():
        if line.startswith("call"):
            which = line
            continue
        gx, gy, gz, bx, by, bz = map(int, line.split())
        launches += 1
        assert 0 < gx and gx * bx < 1 << 32, (which, line)
        assert 0 < gy <= 65535 and 0 < gz <= 65535 and 0 < bx * by * bz <= 1024, (which, line)
    assert launches >= sum(f == call for f, _ in CASES)
