"""The C ABI of the operators on channels without a GPU: exports, and refusals
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

from sink_rank_recurrent_amd import channels
from test_abi_sanitized import ROCM, ROOT, _gcc_lib

L = channels.lib()
HOST_ONLY = "SEED_LIBRARY" in os.environ     # the sanitizer build: no call reaches a device
BIG = 1 << 44
MISALIGNED = ctypes.c_void_p(0x10008)
ODD = ctypes.c_void_p(0x10001)


class Space:
    """Disjoint made-up device addresses (never dereferenced: every call
    below is refused, or runs on the host-only build)."""

    def __init__(self):
        self.at = 1 << 20

    def __call__(self):
        self.at += 1 << 40
        return ctypes.c_void_p(self.at)


def test_exports_every_declared_function():
    text = re.sub(r"/\*.*?\*/", "", open(channels.HEADER_PATH).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:seed_status|size_t)\s+([a-z_0-9]+)\s*\(", text, flags=re.M))
    assert names == {"seed_short_conv", "seed_short_conv_backward", "seed_short_conv_workspace_bytes",
                     "seed_short_conv_step", "seed_selective_scan", "seed_selective_scan_backward",
                     "seed_selective_scan_workspace_bytes", "seed_selective_step"}
    for n in names:
        assert hasattr(L, n), n


CONV_IN = ("x", "x_stride", "dtype", "weight", "bias", "S0", "activation")
CONV = ("n_seq", "channels", "width", "tokens", "cu", *CONV_IN, "y", "y_stride", "S", "stream")
CONVB = ("n_seq", "channels", "width", "tokens", "cu", *CONV_IN, "dy", "dy_stride", "dS", "dx", "dx_stride",
         "dweight", "dbias", "dS0", "ws", "ws_bytes", "stream")
CONVS = ("batch", "channels", "width", *CONV_IN, "y", "y_stride", "S", "stream")
SCAN_IN = ("x", "x_stride", "dt", "dt_stride", "A", "B", "B_stride", "C", "C_stride", "dtype", "D", "z", "z_stride",
           "dt_bias", "softplus", "S0")
SCAN = ("n_seq", "channels", "groups", "d_state", "tokens", "cu", *SCAN_IN, "y", "y_stride", "S", "ws", "ws_bytes",
        "stream")
SCANB = ("n_seq", "channels", "groups", "d_state", "tokens", "cu", *SCAN_IN, "dy", "dy_stride", "dS", "dx",
         "dx_stride", "ddt", "ddt_stride", "dA", "dB", "dB_stride", "dC", "dC_stride", "dD", "dz", "dz_stride",
         "ddt_bias", "dS0", "ws", "ws_bytes", "stream")
STEP = ("batch", "channels", "groups", "d_state", *SCAN_IN, "y", "y_stride", "S", "stream")
SIZES = {"n_seq": 2, "batch": 5, "channels": 96, "width": 4, "tokens": 1000, "dtype": 1, "activation": 1,
         "groups": 2, "d_state": 16, "softplus": 1, "ws_bytes": BIG >> 5, "stream": None}
STRIDES = {"B_stride": 32, "C_stride": 32, "dB_stride": 40, "dC_stride": 32}


def _call(fn, names, over):
    space = Space()
    a = {}
    for n in names:
        a[n] = SIZES[n] if n in SIZES else STRIDES.get(n, 96) if n.endswith("_stride") else space()
    for k, v in over.items():
        a[k] = v(a) if callable(v) else v
    status = getattr(L, fn)(*(a[n] for n in names))
    return status, L.seed_last_error().decode()


def at(name, offset=0):
    return lambda a: ctypes.c_void_p(a[name].value + offset)


SEQ_BAD = [
    (dict(n_seq=0), 2, "positive"), (dict(tokens=-1), 2, "at least 0"), (dict(channels=0), 2, "positive"),
    (dict(channels=(1 << 20) + 2), 3, "2^20"), (dict(tokens=1001, cu=None), 2, "equal"),
    (dict(n_seq=1 << 25), 3, "grid"), (dict(cu=ctypes.c_void_p(0x10002)), 1, "cu_seqlens is not"),
    (dict(tokens=0x7fffffff), 3, "grid"),
]
CONV_BAD = [
    (dict(width=1), 3, "width"), (dict(width=5), 3, "width"), (dict(dtype=2), 1, "dtype"),
    (dict(activation=2), 1, "activation"), (dict(x=None), 1, "x is NULL"), (dict(x=ODD), 1, "x is not 2-byte"),
    (dict(x_stride=95), 2, "rows of 96"), (dict(x_stride=-96), 2, "rows of 96"),
    (dict(x_stride=(1 << 40) + 1), 3, "2^40"),
    (dict(weight=None), 1, "weight is NULL"), (dict(weight=MISALIGNED), 1, "weight is not"),
    (dict(bias=MISALIGNED), 1, "bias is not"), (dict(S0=MISALIGNED), 1, "S0 is not"),
]


@pytest.mark.parametrize("over,status,text", SEQ_BAD + CONV_BAD + [
    (dict(y=None), 1, "y is NULL"), (dict(y_stride=8), 2, "rows of 96"), (dict(S=MISALIGNED), 1, "S is not"),
    (dict(y=at("x")), 1, "y overlaps x"), (dict(y=at("weight")), 1, "y overlaps weight"),
    (dict(S=at("y")), 1, "S overlaps y"), (dict(S=at("S0", 16)), 1, "S overlaps S0"),
    (dict(y=at("cu")), 1, "y overlaps cu_seqlens"), (dict(S=at("x")), 1, "S overlaps x"),
    # two slices of one buffer's rows that share a column
    (dict(x_stride=200, y_stride=200, y=at("x", 2 * 95)), 1, "y overlaps x"),
    (dict(x_stride=200, y_stride=200, x=at("y", 2 * 110)), 1, "y overlaps x")])
def test_conv_refuses(over, status, text):
    got, why = _call("seed_short_conv", CONV, over)
    assert got == status and text in why, (got, why)


@pytest.mark.parametrize("over,status,text", SEQ_BAD + CONV_BAD + [
    (dict(dy=None), 1, "dy is NULL"), (dict(dx=None), 1, "dx is NULL"), (dict(dy_stride=3), 2, "rows of 96"),
    (dict(dx_stride=3), 2, "rows of 96"), (dict(dS=MISALIGNED), 1, "dS is not"),
    (dict(dS0=MISALIGNED), 1, "dS0 is not"), (dict(dweight=MISALIGNED), 1, "dweight is not"),
    (dict(ws=None), 1, "workspace is NULL"), (dict(ws_bytes=16), 1, "needed"),
    (dict(dx=at("dy")), 1, "dx overlaps dy"), (dict(dx=at("x")), 1, "dx overlaps x"),
    (dict(dS0=at("dS")), 1, "dS0 overlaps dS"), (dict(dbias=at("bias")), 1, "dbias overlaps bias"),
    (dict(dbias=at("dweight")), 1, "dbias overlaps dweight"), (dict(ws=at("x")), 1, "workspace overlaps x")])
def test_conv_backward_refuses(over, status, text):
    got, why = _call("seed_short_conv_backward", CONVB, over)
    assert got == status and text in why, (got, why)


@pytest.mark.parametrize("over,status,text", CONV_BAD + [
    (dict(batch=-1), 2, "at least 0"), (dict(S0=None), 1, "S0 is NULL"), (dict(S=None), 1, "S is NULL"),
    (dict(y=at("x", 2)), 1, "y overlaps x"), (dict(y=at("x"), y_stride=97), 1, "y overlaps x"),
    (dict(S=at("S0", 16)), 1, "S overlaps S0"), (dict(y=at("S0")), 1, "y overlaps S0"),
    (dict(S=at("x")), 1, "S overlaps x"), (dict(S=at("weight")), 1, "S overlaps weight"),
    (dict(S=at("y")), 1, "S overlaps y")])
def test_conv_step_refuses(over, status, text):
    got, why = _call("seed_short_conv_step", CONVS, over)
    assert got == status and text in why, (got, why)


SCAN_BAD = [
    (dict(groups=0), 2, "multiple"), (dict(groups=5), 2, "multiple"), (dict(d_state=0), 3, "d_state"),
    (dict(d_state=65), 3, "d_state"), (dict(dtype=-1), 1, "dtype"), (dict(x=None), 1, "x is NULL"),
    (dict(dt=None), 1, "dt is NULL"), (dict(A=None), 1, "A is NULL"), (dict(B=None), 1, "B is NULL"),
    (dict(C=ODD), 1, "C is not 2-byte"), (dict(B_stride=31), 2, "rows of 32"), (dict(z=ODD), 1, "z is not"),
    (dict(z_stride=0), 2, "rows of 96"), (dict(D=MISALIGNED), 1, "D is not"),
    (dict(dt_bias=MISALIGNED), 1, "dt_bias is not"), (dict(S0=MISALIGNED), 1, "S0 is not"),
]


@pytest.mark.parametrize("over,status,text", SEQ_BAD + SCAN_BAD + [
    (dict(channels=1 << 20, groups=1 << 17, B_stride=1 << 21, C_stride=1 << 21), 3, "grid"),
    (dict(y=None), 1, "y is NULL"), (dict(S=None), 1, "S is NULL"), (dict(ws=None), 1, "workspace is NULL"),
    (dict(ws_bytes=16), 1, "needed"), (dict(y=at("z")), 1, "y overlaps z"), (dict(S=at("A")), 1, "S overlaps A"),
    (dict(S=at("S0", 64)), 1, "S overlaps S0"), (dict(ws=at("B")), 1, "workspace overlaps B"),
    (dict(ws=at("cu")), 1, "workspace overlaps cu_seqlens"), (dict(S=at("y")), 1, "S overlaps y")])
def test_scan_refuses(over, status, text):
    got, why = _call("seed_selective_scan", SCAN, over)
    assert got == status and text in why, (got, why)


@pytest.mark.parametrize("over,status,text", SEQ_BAD + SCAN_BAD + [
    (dict(dz=None), 1, "exactly if"), (dict(z=None), 1, "exactly if"), (dict(dy=None), 1, "dy is NULL"),
    (dict(dx=None), 1, "dx is NULL"), (dict(ddt=None), 1, "ddt is NULL"), (dict(dA=None), 1, "dA is NULL"),
    (dict(dB=None), 1, "dB is NULL"), (dict(dC=None), 1, "dC is NULL"), (dict(dC_stride=5), 2, "rows of 32"),
    (dict(ws_bytes=8), 1, "needed"), (dict(dx=at("dy")), 1, "dx overlaps dy"),
    (dict(ddt=at("dx")), 1, "ddt overlaps dx"), (dict(dS0=at("S0")), 1, "dS0 overlaps S0"),
    (dict(dD=at("dA")), 1, "dD overlaps dA"), (dict(ddt_bias=at("dt_bias")), 1, "ddt_bias overlaps dt_bias"),
    (dict(ws=at("dB")), 1, "workspace overlaps dB"), (dict(dS0=at("dS", 16)), 1, "dS0 overlaps dS")])
def test_scan_backward_refuses(over, status, text):
    got, why = _call("seed_selective_scan_backward", SCANB, over)
    assert got == status and text in why, (got, why)


@pytest.mark.parametrize("over,status,text", SCAN_BAD + [
    (dict(batch=-1), 2, "at least 0"), (dict(S0=None), 1, "S0 is NULL"), (dict(S=None), 1, "S is NULL"),
    (dict(y=at("x", 2)), 1, "y overlaps x"), (dict(y=at("z"), y_stride=98), 1, "y overlaps z"),
    (dict(S=at("S0", 16)), 1, "S overlaps S0"), (dict(y=at("S0")), 1, "y overlaps S0"),
    (dict(S=at("A")), 1, "S overlaps A"), (dict(y=at("B")), 1, "y overlaps B")])
def test_step_refuses(over, status, text):
    got, why = _call("seed_selective_step", STEP, over)
    assert got == status and text in why, (got, why)


def test_workspace_queries():
    reject = ctypes.c_size_t(-1).value
    one = L.seed_selective_scan_workspace_bytes(2, 96, 2, 16, 1000, 0)
    assert 0 < one < L.seed_selective_scan_workspace_bytes(2, 96, 2, 16, 10000, 0)
    assert one <= L.seed_selective_scan_workspace_bytes(2, 96, 2, 16, 1000, 1)
    assert L.seed_selective_scan_workspace_bytes(2, 96, 2, 16, 0, 1) == 0
    assert L.seed_selective_scan_workspace_bytes(2, 96, 5, 16, 100, 0) == reject
    assert 0 < L.seed_short_conv_workspace_bytes(2, 96, 4, 1000) < 1 << 20
    assert L.seed_short_conv_workspace_bytes(2, 96, 5, 100) == reject


def test_nothing_to_do():
    """No rows: nothing is launched, and only the weights' pointers are needed."""
    none = {n: None for n in ("x", "y", "S0", "S", "cu")}
    assert _call("seed_short_conv", CONV, dict(none, tokens=0)) == (0, "")
    none = {n: None for n in ("x", "dy", "dx", "S0", "dS", "dS0", "dweight", "dbias", "ws", "cu")}
    assert _call("seed_short_conv_backward", CONVB, dict(none, tokens=0)) == (0, "")
    none = {n: None for n in ("x", "y", "S0", "S", "dt", "B", "C", "z")}
    assert _call("seed_short_conv_step", CONVS, dict({k: none[k] for k in ("x", "y", "S0", "S")}, batch=0)) == (0, "")
    assert _call("seed_selective_step", STEP, dict(none, batch=0)) == (0, "")


@pytest.mark.skipif(not HOST_ONLY, reason="these calls would launch: the host-only build runs them")
def test_valid_calls_pass_validation():
    for over in ({}, dict(S=at("S0")), dict(S=None), dict(S0=None), dict(cu=None), dict(bias=None),
                 dict(x_stride=200, y_stride=200, y=at("x", 2 * 96)),
                 dict(x_stride=200, y_stride=200, x=at("y", 2 * 104))):
        assert _call("seed_short_conv", CONV, over)[0] == 0, over
    for over in ({}, dict(dweight=None, dbias=None, ws=None), dict(dS=None, dS0=None)):
        assert _call("seed_short_conv_backward", CONVB, over)[0] == 0, over
    for over in ({}, dict(S=at("S0")), dict(y=at("x"))):
        assert _call("seed_short_conv_step", CONVS, over)[0] == 0, over
    for over in ({}, dict(S=at("S0")), dict(z=None), dict(D=None, dt_bias=None, S0=None),
                 dict(x_stride=192, z_stride=192, z=at("x", 192)), dict(tokens=0, ws=None, ws_bytes=0)):
        assert _call("seed_selective_scan", SCAN, over)[0] == 0, over
    for over in ({}, dict(dS0=at("dS")), dict(z=None, dz=None), dict(dD=None, ddt_bias=None, dS0=None),
                 dict(dx_stride=192, dz_stride=192, dz=at("dx", 192))):
        assert _call("seed_selective_scan_backward", SCANB, over)[0] == 0, over
    for over in ({}, dict(S=at("S0")), dict(y=at("x")), dict(y=at("z")), dict(y=at("dt"))):
        assert _call("seed_selective_step", STEP, over)[0] == 0, over


def test_rows_of_tensors():
    """What the binding takes as rows one distance apart."""
    rows = channels._rows
    t = torch.zeros(4, 6, 10, dtype=torch.bfloat16)
    io = (torch.bfloat16,)
    assert rows(t, "t", (4, 6), (10,), io)[1] == 10
    assert rows(t[..., 2:7], "t", (4, 6), (5,), io) == (t.data_ptr() + 4, 10)
    assert rows(t[:1, :, :3], "t", (1, 6), (3,), io)[1] == 10
    assert rows(t[:, :1], "t", (4, 1), (10,), io)[1] == 60
    assert rows(t[:0], "t", (0, 6), (10,), io)[1] >= 10
    assert rows(t.view(24, 2, 5), "t", (24,), (2, 5), io)[1] == 10
    for bad, lead in ((t[:, :3], (4, 3)), (t[..., ::2], (4, 6)), (t.transpose(0, 1), (6, 4))):
        with pytest.raises(ValueError):
            rows(bad, "t", lead, (bad.shape[-1],), io)
    with pytest.raises(ValueError, match="apart"):
        rows(t[0, :1].expand(5, 10), "t", (5,), (10,), io)
    with pytest.raises(ValueError, match="behind each other"):
        rows(t.view(24, 2, 5)[:, :, :4], "t", (24,), (2, 4), io)
    with pytest.raises(ValueError, match="dtype"):
        rows(t, "t", (4, 6), (10,), (torch.float32,))


def test_rows_on_the_shorter_way():
    """The calls' shorter way takes and refuses the same rows."""
    io = (torch.bfloat16,)
    t = torch.zeros(24, 10, dtype=torch.bfloat16)
    wide = torch.zeros(24, 3, 10, dtype=torch.bfloat16)
    for a, dims in ((t, 1), (t[:, 2:7], 1), (t[:1, :3], 1), (t[:0], 1), (t[::2], 1), (t[:, :1], 1),
                    (t.view(4, 6, 10), 1), (t.view(4, 6, 10)[:1, :, :3], 1), (t.view(24, 2, 5), 2),
                    (t[:, 2:6].view(24, 2, 2), 2), (t[:, :5].unsqueeze(1), 2), (wide[:, :2], 2),
                    (wide[:, 1:2], 2), (wide[:, :, :1], 1), (t.view(4, 6, 2, 5), 2), (None, 1)):
        shape = (24, 10) if a is None else tuple(a.shape)
        assert channels._row(a, "t", shape, dims, io) == channels._rows(a, "t", shape[:-dims], shape[-dims:], io), shape
    for a, dims in ((t.view(4, 6, 10)[:, :3], 1), (t[:, ::2], 1), (wide[:, :, :4], 2), (t.t(), 1),
                    (t[:1].expand(5, 10), 1), (wide.transpose(0, 1), 2)):
        shape = tuple(a.shape)
        for f in (lambda: channels._row(a, "t", shape, dims, io),
                  lambda: channels._rows(a, "t", shape[:-dims], shape[-dims:], io)):
            with pytest.raises(ValueError):
                f()
    with pytest.raises(ValueError, match="dtype"):
        channels._row(t, "t", (24, 10), 1, (torch.float32,))
    with pytest.raises(ValueError, match="shape"):
        channels._row(t, "t", (24, 11), 1, io)
    with pytest.raises(TypeError):
        channels._row(3, "t", (24, 10), 1, io)


def test_binding_refuses():
    x = torch.zeros(10, 32)
    with pytest.raises(ValueError, match="device memory"):
        channels.seed_short_conv(x, x, x)
    with pytest.raises(ValueError, match="device memory"):
        channels.seed_selective_scan(x, x, x, x, x, x, x)
    with pytest.raises(TypeError):
        channels.seed_short_conv_step(x.numel(), x, x, x)


@pytest.mark.skipif(HOST_ONLY or shutil.which("g++") is None or _gcc_lib("libasan.so") is None
                    or not os.path.exists(os.path.join(ROCM, "include", "hip", "hip_runtime.h")),
                    reason="needs g++ with AddressSanitizer and the HIP headers")
def test_validation_under_asan_and_ubsan(tmp_path):
    lib = str(tmp_path / "libseed_channels_sanitized.so")
    csrc = os.path.join(ROOT, "sink_rank_recurrent_amd", "csrc")
    stubs = os.path.join(ROOT, "tests", "sanitize")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fPIC", "-shared",
           "-fsanitize=address,undefined", "-fno-omit-frame-pointer", "-fno-sanitize-recover=all",
           "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
           "-I", os.path.join(ROOT, "include"), "-I", csrc,
           os.path.join(csrc, "seed_api.cpp"), os.path.join(csrc, "seed_channels_api.cpp"),
           os.path.join(stubs, "stub_launch.cpp"), os.path.join(stubs, "stub_launch_channels.cpp"),
           "-L", os.path.join(ROCM, "lib"), "-lamdhip64", "-o", lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ, SEED_LIBRARY=lib, LD_PRELOAD=_gcc_lib("libasan.so"),
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_channels_abi.py")],
                       capture_output=True, text=True, env=env, cwd=ROOT, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
