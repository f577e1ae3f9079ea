"""The C ABI of the sequence operators without a GPU: exports, and refusals
on the host before any HIP call; the same under AddressSanitizer and
UndefinedBehaviorSanitizer."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import pytest
import torch

from sink_rank_recurrent_amd import binding, sequence
from test_abi_sanitized import ROCM, ROOT, _gcc_lib

L = sequence.lib()
HOST_ONLY = "SEED_LIBRARY" in os.environ     # the sanitizer build: no call reaches a device
BIG = 1 << 44


class Space:
    """Disjoint made-up device addresses (never dereferenced: every call
    below is refused, or runs on the host-only build)."""

    def __init__(self):
        self.at = 1 << 20

    def __call__(self):
        self.at += 1 << 40
        return ctypes.c_void_p(self.at)


def test_exports_every_declared_function():
    text = re.sub(r"/\*.*?\*/", "", open(sequence.HEADER_PATH).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:seed_status|size_t)\s+([a-z_0-9]+)\s*\(", text, flags=re.M))
    assert names == {"seed_scan", "seed_scan_backward", "seed_scan_workspace_bytes",
                     "seed_group_norm", "seed_group_norm_backward",
                     "seed_group_norm_workspace_bytes"}
    for n in names:
        assert hasattr(L, n), n


SCAN = ("rule", "n_seq", "heads", "key_heads", "d_k", "d_v", "tokens", "cu", "q", "k", "v", "dtype",
        "g", "beta", "S0", "o", "S", "ws", "ws_bytes", "stream")
BACK = ("rule", "n_seq", "heads", "key_heads", "d_k", "d_v", "tokens", "cu", "q", "k", "v", "dtype",
        "g", "beta", "S0", "dO", "dS", "dq", "dk", "dv", "dg", "dbeta", "dS0", "ws", "ws_bytes",
        "stream")
SIZES = {"rule": 0, "n_seq": 2, "heads": 4, "key_heads": 2, "d_k": 128, "d_v": 64, "tokens": 100,
         "dtype": 1, "ws_bytes": BIG >> 5, "stream": None}


def _call(fn, names, sizes, over):
    space = Space()
    a = {n: sizes[n] if n in sizes else space() for n in names}
    for k, v in over.items():
        a[k] = v(a) if callable(v) else v
    status = getattr(L, fn)(*(a[n] for n in names))
    return status, L.seed_last_error().decode()


MISALIGNED = ctypes.c_void_p(0x10008)
SCAN_BAD = [
    (dict(rule=3), 1, "unknown rule"),
    (dict(n_seq=0), 2, "positive"),
    (dict(tokens=-1), 2, "at least 0"),
    (dict(key_heads=3), 2, "multiple"),
    (dict(key_heads=8), 2, "multiple"),
    (dict(d_k=64, d_v=128), 3, "not supported"),
    (dict(heads=65536, key_heads=1), 3, "grid"),
    (dict(n_seq=1 << 30), 3, "grid"),
    (dict(tokens=0x7fffffff), 3, "grid"),
    (dict(dtype=2), 1, "dtype"),
    (dict(tokens=101, cu=None), 2, "equal"),
    (dict(q=None), 1, "q is NULL"),
    (dict(k=MISALIGNED), 1, "k is not 16-byte"),
    (dict(v=None), 1, "v is NULL"),
    (dict(g=None), 1, "g is NULL"),
    (dict(beta=None), 1, "beta is NULL"),
    (dict(rule=2), 1, "beta must be NULL"),
    (dict(S0=MISALIGNED), 1, "S0 is not"),
    (dict(cu=ctypes.c_void_p(0x10002)), 1, "cu_seqlens"),
    (dict(ws=None), 1, "workspace is NULL"),
    (dict(ws_bytes=16), 1, "needed"),
]


@pytest.mark.parametrize("over,status,text", SCAN_BAD + [
    (dict(o=None), 1, "o is NULL"), (dict(S=None), 1, "S is NULL"),
    (dict(o=lambda a: a["v"]), 1, "o overlaps v"), (dict(S=lambda a: a["o"]), 1, "S overlaps o"),
    (dict(ws=lambda a: a["q"]), 1, "workspace overlaps q"),
    (dict(S=lambda a: ctypes.c_void_p(a["S0"].value + 64)), 1, "S overlaps S0")])
def test_scan_refuses(over, status, text):
    got, why = _call("seed_scan", SCAN, SIZES, over)
    assert got == status and text in why, (got, why)


@pytest.mark.parametrize("over,status,text", SCAN_BAD + [
    (dict(dO=None), 1, "dO is NULL"), (dict(dq=None), 1, "dq is NULL"),
    (dict(dk=MISALIGNED), 1, "dk is not"), (dict(dv=None), 1, "dv is NULL"),
    (dict(dg=None), 1, "dg is NULL"), (dict(dbeta=None), 1, "dbeta is NULL"),
    (dict(rule=2, beta=None), 1, "dbeta must be NULL"), (dict(dS=MISALIGNED), 1, "dS is not"),
    (dict(dS0=MISALIGNED), 1, "dS0 is not"), (dict(dq=lambda a: a["q"]), 1, "dq overlaps q"),
    (dict(dk=lambda a: a["dq"]), 1, "dk overlaps dq"),
    (dict(dv=lambda a: a["dO"]), 1, "dv overlaps dO"),
    (dict(dS0=lambda a: a["S0"]), 1, "dS0 overlaps S0")])
def test_scan_backward_refuses(over, status, text):
    got, why = _call("seed_scan_backward", BACK, SIZES, over)
    assert got == status and text in why, (got, why)


NORM = ("rows", "groups", "d", "x", "x_dtype", "gate", "io_dtype", "weight", "bias",
        "weight_groups", "eps", "centered", "activation", "gate_first", "y", "stream")
NORMB = ("rows", "groups", "d", "dy", "x", "x_dtype", "gate", "io_dtype", "weight", "bias",
         "weight_groups", "eps", "centered", "activation", "gate_first", "dx", "dgate", "dweight",
         "dbias", "ws", "ws_bytes", "stream")
NSIZES = {"rows": 7, "groups": 4, "d": 128, "x_dtype": 0, "io_dtype": 1, "weight_groups": 1,
          "eps": 1e-5, "centered": 0, "activation": 1, "gate_first": 0, "ws_bytes": BIG >> 5,
          "stream": None}
NORM_BAD = [
    (dict(rows=-1), 2, "at least 0"),
    (dict(groups=0), 2, "positive"),
    (dict(d=0), 2, "positive"),
    (dict(weight_groups=2), 2, "weight_groups"),
    (dict(d=8193), 3, "8192"),
    (dict(groups=65536), 3, "grid"),
    (dict(rows=1 << 30), 3, "grid"),
    (dict(x_dtype=2), 1, "dtype"),
    (dict(io_dtype=-1), 1, "dtype"),
    (dict(activation=3), 1, "activation"),
    (dict(eps=-1.0), 1, "eps"),
    (dict(eps=float("nan")), 1, "eps"),
    (dict(gate=MISALIGNED), 1, "gate is not"),
    (dict(weight=MISALIGNED), 1, "weight is not"),
    (dict(x=None), 1, "x is NULL"),
]


@pytest.mark.parametrize("over,status,text", NORM_BAD + [
    (dict(gate_first=1, gate=None), 1, "without a gate"),
    (dict(y=None), 1, "y is NULL"), (dict(y=lambda a: a["x"]), 1, "y overlaps x"),
    (dict(y=lambda a: a["weight"]), 1, "y overlaps weight"),
    (dict(y=lambda a: ctypes.c_void_p(a["gate"].value + 32)), 1, "y overlaps gate")])
def test_norm_refuses(over, status, text):
    got, why = _call("seed_group_norm", NORM, NSIZES, over)
    assert got == status and text in why, (got, why)


@pytest.mark.parametrize("over,status,text", NORM_BAD + [
    (dict(dgate=None), 1, "exactly if"), (dict(gate=None), 1, "exactly if"),
    (dict(dy=None), 1, "dy is NULL"), (dict(dx=None), 1, "dx is NULL"),
    (dict(ws=None), 1, "workspace is NULL"), (dict(ws_bytes=8), 1, "needed"),
    (dict(dx=lambda a: a["dy"]), 1, "dx overlaps dy"),       # float32 over bf16
    (dict(dgate=lambda a: a["x"]), 1, "dgate overlaps x"),
    (dict(dweight=lambda a: a["weight"]), 1, "dweight overlaps weight"),
    (dict(dbias=lambda a: a["dweight"]), 1, "dbias overlaps dweight")])
def test_norm_backward_refuses(over, status, text):
    got, why = _call("seed_group_norm_backward", NORMB, NSIZES, over)
    assert got == status and text in why, (got, why)


def test_workspace_queries():
    reject = ctypes.c_size_t(-1).value
    one = L.seed_scan_workspace_bytes(0, 2, 4, 2, 128, 64, 100, 0)
    assert 0 < one < L.seed_scan_workspace_bytes(0, 2, 4, 2, 128, 64, 1000, 0)
    assert one <= L.seed_scan_workspace_bytes(0, 2, 4, 2, 128, 64, 100, 1)
    assert L.seed_scan_workspace_bytes(0, 2, 4, 2, 128, 64, 0, 1) == 0
    assert L.seed_scan_workspace_bytes(0, 2, 4, 3, 128, 64, 100, 0) == reject
    assert 0 < L.seed_group_norm_workspace_bytes(7, 4, 128, 1) < 1 << 20
    assert L.seed_group_norm_workspace_bytes(7, 4, 9000, 1) == reject


def test_nothing_to_do():
    """No rows: nothing is launched and no pointer is needed."""
    none = {n: None for n in ("x", "gate", "y", "weight", "bias")}
    assert _call("seed_group_norm", NORM, NSIZES, dict(none, rows=0)) == (0, "")
    none = {n: None for n in ("dy", "x", "gate", "weight", "bias", "dx", "dgate", "dweight",
                              "dbias", "ws")}
    assert _call("seed_group_norm_backward", NORMB, NSIZES, dict(none, rows=0)) == (0, "")


@pytest.mark.skipif(not HOST_ONLY, reason="these calls would launch: the host-only build runs them")
def test_valid_calls_pass_validation():
    assert _call("seed_scan", SCAN, SIZES, {})[0] == 0
    assert _call("seed_scan", SCAN, SIZES, dict(S=lambda a: a["S0"]))[0] == 0
    assert _call("seed_scan_backward", BACK, SIZES, dict(dS0=lambda a: a["dS"]))[0] == 0
    assert _call("seed_scan_backward", BACK, SIZES, dict(rule=2, beta=None, dbeta=None))[0] == 0
    assert _call("seed_group_norm", NORM, NSIZES, dict(y=lambda a: a["gate"]))[0] == 0
    assert _call("seed_group_norm_backward", NORMB, NSIZES,
                 dict(dx=lambda a: a["x"], dgate=lambda a: a["dy"]))[0] == 0


def test_binding_refuses():
    q = torch.zeros(10, 2, 128)
    with pytest.raises(ValueError, match="device memory"):
        sequence.seed_scan("gdn", q, q, q, q[..., 0], q[..., 0], q, q)
    with pytest.raises(ValueError, match="device memory"):
        sequence.seed_group_norm(q, q)
    with pytest.raises(TypeError):
        sequence.seed_group_norm(q.numpy(), q)
    st = binding.ShallowState("gdn", 5, 2, 128, 128, 16, 16, torch.ones(2, 128), device="cpu")
    x = q.view(5, 2, 2, 128)
    with pytest.raises(ValueError):
        st.prefill(x, x, x, x[..., 0], x[..., 0], x)
    assert st.r == 0


@pytest.mark.skipif(HOST_ONLY or shutil.which("g++") is None or _gcc_lib("libasan.so") is None
                    or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")),
                    reason="needs g++ with AddressSanitizer and the HIP headers")
def test_validation_under_asan_and_ubsan(tmp_path):
    lib = str(tmp_path / "libseed_sequence_sanitized.so")
    csrc = os.path.join(ROOT, "sink_rank_recurrent_amd", "csrc")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-shared",
           "-fsanitize=address,undefined", "-fno-omit-frame-pointer", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
           "-I", os.path.join(ROOT, "include"), "-I", csrc,
           os.path.join(csrc, "seed_api.cpp"), os.path.join(csrc, "seed_sequence_api.cpp"),
           os.path.join(ROOT, "tests", "sanitize", "stub_launch.cpp"),
           os.path.join(ROOT, "tests", "sanitize", "stub_launch_sequence.cpp"),
           "-L", os.path.join(ROCM, "lib"), "-lamdhip64", "-o", lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ, SEED_LIBRARY=lib, LD_PRELOAD=_gcc_lib("libasan.so"),
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_sequence_abi.py")],
                       capture_output=True, text=True, env=env, cwd=ROOT, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
