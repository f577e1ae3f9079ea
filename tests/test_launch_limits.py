"""Grids of the sequence operators at the largest sizes they accept, on the
CPU: the built library with the runtime's launch call replaced by one that
writes the grid down (tests/sanitize/record_launches.c).  An accepted call has
to fit: fewer than 2^32 threads along x, at most 65535 blocks along y and z."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest

from sink_rank_recurrent_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAR = 1 << 46     # between two made-up addresses


def _call(name, *args):
    """`name` with "p" for an address of its own and None for NULL."""
    from sink_rank_recurrent_amd import sequence
    at = iter(range(1, 64))
    got = getattr(sequence.lib(), name)(*(ctypes.c_void_p(next(at) * FAR) if a == "p" else a for a in args))
    assert got == 0, (name, args, binding.lib().seed_last_error())


def norm(rows, groups, d, weight_groups):
    _call("seed_group_norm", rows, groups, d, "p", 1, "p", 1, "p", "p", weight_groups, 1e-5, 0, 1, 0, "p", None)


def norm_backward(rows, groups, d, weight_groups):
    _call("seed_group_norm_backward", rows, groups, d, "p", "p", 1, "p", 1, "p", "p", weight_groups, 1e-5, 0, 1,
          0, "p", "p", "p", "p", "p", FAR, None)


def scan(rule, n_seq, heads, key_heads, tokens):
    beta = None if rule == 2 else "p"
    _call("seed_scan", rule, n_seq, heads, key_heads, 128, 128, tokens, "p", "p", "p", "p", 1, "p", beta, "p",
          "p", "p", "p", FAR, None)


def scan_backward(rule, n_seq, heads, key_heads, tokens):
    beta = None if rule == 2 else "p"
    _call("seed_scan_backward", rule, n_seq, heads, key_heads, 128, 128, tokens, "p", "p", "p", "p", 1, "p", beta,
          "p", "p", "p", "p", "p", "p", "p", beta, "p", "p", FAR, None)


NORMS = [(1, 65535, 8192, 65535), (1, 65535, 8191, 65535), (0, 65535, 8192, 65535), (1, 4096, 8192, 4096),
         (32767, 65535, 8, 65535), (0x7fffffff, 1, 8192, 1), (0x7fffffff // 65535, 65535, 1, 1)]
SCANS = [(1, 65535, 65535, 64 * 62), (63, 65535, 1, 63), ((1 << 22) - 65, 1, 1, 64 * 64), (1, 1, 1, 0x7fffffff // 64 * 2),
         (1, 4, 2, 1 << 24)]
CASES = [(f, a) for f in ("norm", "norm_backward") for a in NORMS] + [
    (f, (rule, *a)) for f in ("scan", "scan_backward") for rule in range(3) for a in SCANS]


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    if shutil.which("gcc") is None or not os.path.exists(binding.LIB_PATH):
        pytest.skip("needs gcc and the built library")
    so = str(tmp_path_factory.mktemp("record") / "record.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", so,
                    os.path.join(ROOT, "tests", "sanitize", "record_launches.c")], check=True)
    return so


@pytest.mark.parametrize("call", ["norm", "norm_backward", "scan", "scan_backward"])
def test_largest_accepted_sizes_fit_a_grid(recorder, tmp_path, call):
    out = tmp_path / "launches"
    code = ("import sys; sys.path[:0] = ['tests']; import test_launch_limits as t\n"
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
    assert launches >= sum(f == call for f, _ in CASES) - (call == "norm")   # no rows: none
