"""Operators on channels: argument marshalling only.

The short causal convolution in front of a recurrence and the selective state
space scan, each over (packed) sequences, backward, and for single tokens.  As
in ``sequence``, every function takes torch tensors in device memory, checks
their shapes, and passes raw pointers to the C ABI (declared in
include/seed_channels.h) on torch's current stream of the tensors' device; all
arithmetic happens in the HIP kernels.  A workspace that is not given is
allocated for the call.  Nothing is recorded for autograd: the backward passes
are calls of their own.

Arrays over tokens are [tokens, ...] with cu_seqlens (int32, n_seq + 1
offsets), [sequences, length, ...] without.  They may be slices of wider
tensors (a part of a projection's last dimension) as long as all rows are one
distance apart; everything else is contiguous.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import binding
from .binding import _F32, _IN, _check, _need, _ptr, _stream
from .sequence import ACTIVATIONS, _code, _ints, _same_device, _workspace

HEADER_PATH = os.path.join(os.path.dirname(binding.HEADER_PATH), "seed_channels.h")

_lib = None


def lib() -> ctypes.CDLL:
    """libseed.so with the argument types of the operators on channels set."""
    global _lib
    if _lib is None:
        L = binding.lib()
        i, p, n, s = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_longlong
        row = [p, s]                        # an array over tokens: pointer, row stride
        conv = [*row, i, p, p, p, i]        # x, io_dtype, weight, bias, S0, activation
        L.seed_short_conv.argtypes = [i, i, i, i, p, *conv, *row, p, p]
        L.seed_short_conv_backward.argtypes = [i, i, i, i, p, *conv, *row, p, *row, p, p, p, p, n, p]
        L.seed_short_conv_workspace_bytes.argtypes = [i, i, i, i]
        L.seed_short_conv_step.argtypes = [i, i, i, *conv, *row, p, p]
        # x, dt, A, B, C, io_dtype, D, z, dt_bias, softplus, S0
        scan = [*row, *row, p, *row, *row, i, p, *row, p, i, p]
        L.seed_selective_scan.argtypes = [i, i, i, i, i, p, *scan, *row, p, p, n, p]
        L.seed_selective_scan_backward.argtypes = [i, i, i, i, i, p, *scan, *row, p, *row, *row, p, *row,
                                                   *row, p, *row, p, p, p, n, p]
        L.seed_selective_scan_workspace_bytes.argtypes = [i, i, i, i, i, i]
        L.seed_selective_step.argtypes = [i, i, i, i, *scan, *row, p, p]
        for fn in ("seed_short_conv", "seed_short_conv_backward", "seed_short_conv_step",
                   "seed_selective_scan", "seed_selective_scan_backward", "seed_selective_step"):
            getattr(L, fn).restype = i
        for fn in ("seed_short_conv_workspace_bytes", "seed_selective_scan_workspace_bytes"):
            getattr(L, fn).restype = n
        _lib = L
    return _lib


def _bytes(n: int) -> int:
    if n == ctypes.c_size_t(-1).value:
        raise ValueError(binding.lib().seed_last_error().decode())
    return int(n)


def _rows(t, name: str, lead: tuple, tail: tuple, dtypes) -> tuple:
    """(pointer, row stride in values) of an array over tokens with `tail`
    behind each other in every row; (None, 0) for None."""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.shape != (*lead, *tail):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(*lead, *tail)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    width = tail[0] if len(tail) == 1 else tail[0] * tail[1]
    if t.is_contiguous():
        return t.data_ptr(), width
    strides = t.stride()
    inner = 1
    for size, stride in zip(reversed(tail), reversed(strides[len(lead):])):
        if size > 1 and stride != inner:
            raise ValueError(f"{name}: the values of a row must lie behind each other")
        inner *= size
    if len(lead) == 1:
        step = strides[0] if lead[0] > 1 else width
    elif lead[1] > 1:
        step = strides[1]
        if lead[0] > 1 and strides[0] != lead[1] * step:
            raise ValueError(f"{name}: all rows must be one distance apart")
    else:
        step = strides[0] if lead[0] > 1 else width
    if step < width and t.numel() > 0:
        raise ValueError(f"{name}: rows of {width} values lie {step} apart")
    return t.data_ptr(), max(step, width)


def _row(t, name: str, shape: tuple, dims: int, dtypes) -> tuple:
    """_rows of a shape whose last `dims` dimensions make a row: packed arrays
    of two rows or more, the common case, on a shorter way."""
    if t is None:
        return None, 0
    if isinstance(t, torch.Tensor) and len(shape) == dims + 1 and t.shape == shape and t.dtype in dtypes:
        strides = t.stride()
        width = shape[1] if dims == 1 else shape[1] * shape[2]
        if (strides[-1] == 1 and strides[0] >= width and shape[0] > 1
                and (dims == 1 or strides[1] == shape[2])):
            return t.data_ptr(), strides[0]
    return _rows(t, name, shape[:-dims], shape[-dims:], dtypes)


def _device(first, names: str, *others) -> int:
    """The index of the one device that all tensors are on."""
    try:
        index = first.get_device()
        if index >= 0:
            for t in others:
                if t is not None and t.get_device() != index:
                    break
            else:
                return index
    except AttributeError:
        pass
    _same_device(**dict(zip(names.split(), (first, *others))))     # says which is not
    raise ValueError("the tensors are not on one device")


def _call(name: str, index: int, stream, *args) -> None:
    """Call the library on torch's current stream of device `index`, or on
    `stream`, with that device made current."""
    fn = getattr(_lib or lib(), name)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, _stream(stream, index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _stream(stream, index))
    if st != 0:
        _check(name, st)


def _space(workspace, nbytes, index: int, stream) -> torch.Tensor:
    """The caller's workspace, or one of nbytes() bytes made for the call."""
    if workspace is not None:
        return _workspace(workspace, 0, None, stream)
    with torch.cuda.device(index):
        return _workspace(None, nbytes(), torch.device("cuda", index), stream)


def _lead(x, dims: int, cu_seqlens):
    """(n_seq, tokens, leading shape) of a call whose x has `dims` trailing
    dimensions."""
    want = dims + (1 if cu_seqlens is not None else 2)
    if x.dim() != want:
        raise ValueError(f"x must have {want} dimensions (packed [tokens, channels] with cu_seqlens, "
                         f"[sequences, length, channels] without)")
    lead = tuple(x.shape[:-1])
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
            raise ValueError("cu_seqlens must hold n_seq + 1 offsets")
        n_seq = cu_seqlens.shape[0] - 1
        _need(cu_seqlens, "cu_seqlens", (n_seq + 1,), (torch.int32,))
    else:
        n_seq = lead[0]
    tokens = 1
    for size in lead:
        tokens *= size
    _ints(tokens, n_seq)
    return n_seq, tokens, lead


def _conv_inputs(x, lead, weight, bias, activation):
    if weight.dim() != 2:
        raise ValueError("weight must be [channels, width]")
    channels, width = weight.shape
    _ints(channels, width)
    _need(weight, "weight", (channels, width), _F32)
    if bias is not None:
        _need(bias, "bias", (channels,), _F32)
    if activation not in (None, "silu"):
        raise ValueError(f"unknown activation {activation!r} (use None or 'silu')")
    shape = (*lead, channels)
    return channels, width, shape, _row(x, "x", shape, 1, _IN)


def seed_short_conv(x, weight, y, bias=None, activation="silu", S0=None, S=None, cu_seqlens=None,
                    stream=None) -> None:
    """Convolve each channel of x [..., channels] over its sequence with
    weight [channels, width] into y (see include/seed_channels.h).  S0 and S
    [n_seq, width - 1, channels] of x's type are the inputs before and behind
    each sequence."""
    index = _device(x, "x weight y bias S0 S cu_seqlens", weight, y, bias, S0, S, cu_seqlens)
    n_seq, tokens, lead = _lead(x, 1, cu_seqlens)
    channels, width, shape, xr = _conv_inputs(x, lead, weight, bias, activation)
    yr = _row(y, "y", shape, 1, (x.dtype,))
    for name, t in (("S0", S0), ("S", S)):
        if t is not None:
            _need(t, name, (n_seq, width - 1, channels), (x.dtype,))
    _call("seed_short_conv", index, stream, n_seq, channels, width, tokens, _ptr(cu_seqlens), *xr,
          _code(x.dtype), _ptr(weight), _ptr(bias), _ptr(S0), ACTIVATIONS[activation], *yr, _ptr(S))


def short_conv_workspace(x, weight, n_seq: int) -> torch.Tensor:
    """A workspace for seed_short_conv_backward calls on x [..., channels] in
    n_seq sequences."""
    channels, width = weight.shape
    tokens = x.shape[:-1].numel()
    _ints(n_seq, channels, width, tokens)
    return torch.empty(_bytes(lib().seed_short_conv_workspace_bytes(n_seq, channels, width, tokens)),
                       dtype=torch.uint8, device=x.device)


def seed_short_conv_backward(dy, x, weight, dx, dweight=None, dbias=None, bias=None, activation="silu",
                             S0=None, dS=None, dS0=None, cu_seqlens=None, workspace=None,
                             stream=None) -> None:
    """Gradients of seed_short_conv from dy (and dS, that of S) into dx and,
    where given, dweight, dbias and dS0 (see include/seed_channels.h)."""
    index = _device(x, "x dy weight dx dweight dbias bias S0 dS dS0 cu_seqlens workspace", dy, weight, dx,
                    dweight, dbias, bias, S0, dS, dS0, cu_seqlens, workspace)
    n_seq, tokens, lead = _lead(x, 1, cu_seqlens)
    channels, width, shape, xr = _conv_inputs(x, lead, weight, bias, activation)
    dyr = _row(dy, "dy", shape, 1, (x.dtype,))
    dxr = _row(dx, "dx", shape, 1, (x.dtype,))
    for name, t in (("S0", S0), ("dS", dS), ("dS0", dS0)):
        if t is not None:
            _need(t, name, (n_seq, width - 1, channels), (x.dtype,))
    if dweight is not None:
        _need(dweight, "dweight", (channels, width), _F32)
    if dbias is not None:
        _need(dbias, "dbias", (channels,), _F32)
    ws = None
    if dweight is not None or dbias is not None:
        ws = _space(workspace, lambda: _bytes(lib().seed_short_conv_workspace_bytes(n_seq, channels, width,
                                                                                    tokens)), index, stream)
    _call("seed_short_conv_backward", index, stream, n_seq, channels, width, tokens, _ptr(cu_seqlens), *xr,
          _code(x.dtype), _ptr(weight), _ptr(bias), _ptr(S0), ACTIVATIONS[activation], *dyr, _ptr(dS), *dxr,
          _ptr(dweight), _ptr(dbias), _ptr(dS0), _ptr(ws), 0 if ws is None else ws.numel())


def seed_short_conv_step(x, weight, y, S, bias=None, activation="silu", S0=None, stream=None) -> None:
    """One token of every sequence: row b of x [batch, channels] behind the
    inputs in S0[b] (None: S[b], the step in place) into y, the inputs behind
    it into S [batch, width - 1, channels] (see include/seed_channels.h)."""
    index = _device(x, "x weight y S bias S0", weight, y, S, bias, S0)
    if x.dim() != 2:
        raise ValueError("x must be [batch, channels]")
    lead = tuple(x.shape[:1])
    _ints(lead[0], 0)
    channels, width, shape, xr = _conv_inputs(x, lead, weight, bias, activation)
    yr = _row(y, "y", shape, 1, (x.dtype,))
    _need(S, "S", (lead[0], width - 1, channels), (x.dtype,))
    if S0 is not None:
        _need(S0, "S0", (lead[0], width - 1, channels), (x.dtype,))
    _call("seed_short_conv_step", index, stream, lead[0], channels, width, *xr, _code(x.dtype), _ptr(weight),
          _ptr(bias), _ptr(S if S0 is None else S0), ACTIVATIONS[activation], *yr, _ptr(S))


def _select_inputs(x, dt, A, B, C, D, z, dt_bias, softplus, lead):
    """(channels, groups, d_state, shapes of x and B, arguments from x to
    softplus)."""
    if A.dim() != 2 or B.dim() != len(lead) + 2:
        raise ValueError("A must be [channels, d_state], B and C [..., groups, d_state]")
    channels, d_state = A.shape
    groups = B.shape[-2]
    _ints(channels, groups, d_state)
    _need(A, "A", (channels, d_state), _F32)
    if D is not None:
        _need(D, "D", (channels,), _F32)
    if dt_bias is not None:
        _need(dt_bias, "dt_bias", (channels,), _F32)
    shape, rows = (*lead, channels), (*lead, groups, d_state)
    xr = _row(x, "x", shape, 1, _IN)
    io = (x.dtype,)
    return channels, groups, d_state, shape, rows, (
        *xr, *_row(dt, "dt", shape, 1, io), A.data_ptr(), *_row(B, "B", rows, 2, io),
        *_row(C, "C", rows, 2, io), _code(x.dtype), _ptr(D), *_row(z, "z", shape, 1, io), _ptr(dt_bias),
        1 if softplus else 0)


def _select_bytes(n_seq, channels, groups, d_state, tokens, backward: bool) -> int:
    return _bytes(lib().seed_selective_scan_workspace_bytes(n_seq, channels, groups, d_state, tokens,
                                                            1 if backward else 0))


def selective_scan_workspace(x, B, n_seq: int, backward: bool = False) -> torch.Tensor:
    """A workspace for seed_selective_scan (or seed_selective_scan_backward)
    calls on x [..., channels] and B [..., groups, d_state] in n_seq sequences."""
    sizes = (n_seq, x.shape[-1], B.shape[-2], B.shape[-1], x.shape[:-1].numel())
    _ints(*sizes)
    return torch.empty(_select_bytes(*sizes, backward), dtype=torch.uint8, device=x.device)


def seed_selective_scan(x, dt, A, B, C, y, S, D=None, z=None, dt_bias=None, softplus: bool = True,
                        S0=None, cu_seqlens=None, workspace=None, stream=None) -> None:
    """The selective scan of x [..., channels] with steps dt, rates A
    [channels, d_state], inputs and read-outs B, C [..., groups, d_state] into
    y and the last states S [n_seq, channels, d_state] (see
    include/seed_channels.h)."""
    index = _device(x, "x dt A B C y S D z dt_bias S0 cu_seqlens workspace", dt, A, B, C, y, S, D, z, dt_bias,
                    S0, cu_seqlens, workspace)
    n_seq, tokens, lead = _lead(x, 1, cu_seqlens)
    channels, groups, d_state, shape, rows, args = _select_inputs(x, dt, A, B, C, D, z, dt_bias, softplus, lead)
    yr = _row(y, "y", shape, 1, (x.dtype,))
    for name, t in (("S", S), ("S0", S0)):
        if t is not None:
            _need(t, name, (n_seq, channels, d_state), _F32)
    ws = _space(workspace, lambda: _select_bytes(n_seq, channels, groups, d_state, tokens, False), index, stream)
    _call("seed_selective_scan", index, stream, n_seq, channels, groups, d_state, tokens, _ptr(cu_seqlens),
          *args, _ptr(S0), *yr, _ptr(S), _ptr(ws), ws.numel())


def seed_selective_scan_backward(dy, x, dt, A, B, C, dx, ddt, dA, dB, dC, D=None, z=None, dt_bias=None,
                                 dD=None, dz=None, ddt_bias=None, softplus: bool = True, S0=None,
                                 dS=None, dS0=None, cu_seqlens=None, workspace=None,
                                 stream=None) -> None:
    """Gradients of seed_selective_scan's inputs from dy (and dS, that of S)
    into dx, ddt, dA, dB, dC, dz (with z) and, where given, dD, ddt_bias and
    dS0 (see include/seed_channels.h).  Shapes and types are the inputs'."""
    index = _device(x, "x dy dt A B C dx ddt dA dB dC D z dt_bias dD dz ddt_bias S0 dS dS0 cu_seqlens workspace",
                    dy, dt, A, B, C, dx, ddt, dA, dB, dC, D, z, dt_bias, dD, dz, ddt_bias, S0, dS, dS0,
                    cu_seqlens, workspace)
    n_seq, tokens, lead = _lead(x, 1, cu_seqlens)
    channels, groups, d_state, shape, rows, args = _select_inputs(x, dt, A, B, C, D, z, dt_bias, softplus, lead)
    io = (x.dtype,)
    dyr, dxr, ddtr, dzr = (_row(t, name, shape, 1, io) for name, t in
                           (("dy", dy), ("dx", dx), ("ddt", ddt), ("dz", dz)))
    dBr, dCr = (_row(t, name, rows, 2, io) for name, t in (("dB", dB), ("dC", dC)))
    _need(dA, "dA", (channels, d_state), _F32)
    for name, t in (("dD", dD), ("ddt_bias", ddt_bias)):
        if t is not None:
            _need(t, name, (channels,), _F32)
    for name, t in (("S0", S0), ("dS", dS), ("dS0", dS0)):
        if t is not None:
            _need(t, name, (n_seq, channels, d_state), _F32)
    ws = _space(workspace, lambda: _select_bytes(n_seq, channels, groups, d_state, tokens, True), index, stream)
    _call("seed_selective_scan_backward", index, stream, n_seq, channels, groups, d_state, tokens,
          _ptr(cu_seqlens), *args, _ptr(S0), *dyr, _ptr(dS), *dxr, *ddtr, _ptr(dA), *dBr, *dCr, _ptr(dD), *dzr,
          _ptr(ddt_bias), _ptr(dS0), _ptr(ws), ws.numel())


def seed_selective_step(x, dt, A, B, C, y, S, D=None, z=None, dt_bias=None, softplus: bool = True,
                        S0=None, stream=None) -> None:
    """One token of every sequence: seed_selective_scan of row b of x [batch,
    channels] from S0[b] (None: S[b], the step in place) into y and S [batch,
    channels, d_state] (see include/seed_channels.h)."""
    index = _device(x, "x dt A B C y S D z dt_bias S0", dt, A, B, C, y, S, D, z, dt_bias, S0)
    if x.dim() != 2:
        raise ValueError("x must be [batch, channels]")
    lead = tuple(x.shape[:1])
    _ints(lead[0], 0)
    channels, groups, d_state, shape, rows, args = _select_inputs(x, dt, A, B, C, D, z, dt_bias, softplus, lead)
    yr = _row(y, "y", shape, 1, (x.dtype,))
    _need(S, "S", (lead[0], channels, d_state), _F32)
    if S0 is not None:
        _need(S0, "S0", (lead[0], channels, d_state), _F32)
    _call("seed_selective_step", index, stream, lead[0], channels, groups, d_state, *args,
          _ptr(S if S0 is None else S0), *yr, _ptr(S))
