"""Operators over whole sequences: argument marshalling only.

The gated linear recurrence of the three rules over (packed) sequences, its
backward pass, and the gated group norm of the read-outs with its backward
pass.  As in ``binding``, every function takes torch tensors in device
memory, checks their shapes, and passes raw pointers to the C ABI (declared
in include/seed_sequence.h) on torch's current stream of the tensors'
device; all arithmetic happens in the HIP kernels.  A workspace that is not
given is allocated for the call.  Nothing is recorded for autograd, whether the
tensors require gradients or not: the backward passes are calls of their own.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import binding
from .binding import RULES, _F32, _IN, _check, _need, _ptr, _stream

HEADER_PATH = os.path.join(os.path.dirname(binding.HEADER_PATH), "seed_sequence.h")
ACTIVATIONS = {None: 0, "silu": 1, "sigmoid": 2}

_lib = None


def lib() -> ctypes.CDLL:
    """libseed.so with the argument types of the sequence operators set."""
    global _lib
    if _lib is None:
        L = binding.lib()
        i, p, f, n, ll = (ctypes.c_int, ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t,
                          ctypes.c_longlong)
        shape = [i, i, i, i, i, i, i]       # rule, n_seq, heads, key_heads, d_k, d_v, tokens
        L.seed_scan.argtypes = [*shape, p, p, p, p, i, p, p, p, p, p, p, n, p]
        L.seed_scan_backward.argtypes = [*shape, p, p, p, p, i, p, p, p, p, p, p, p, p, p, p, p,
                                         p, n, p]
        L.seed_scan_workspace_bytes.argtypes = [*shape, i]
        L.seed_group_norm.argtypes = [ll, i, i, p, i, p, i, p, p, i, f, i, i, i, p, p]
        L.seed_group_norm_backward.argtypes = [ll, i, i, p, p, i, p, i, p, p, i, f, i, i, i, p, p,
                                               p, p, p, n, p]
        L.seed_group_norm_workspace_bytes.argtypes = [ll, i, i, i]
        for fn in ("seed_scan", "seed_scan_backward", "seed_group_norm",
                   "seed_group_norm_backward"):
            getattr(L, fn).restype = i
        for fn in ("seed_scan_workspace_bytes", "seed_group_norm_workspace_bytes"):
            getattr(L, fn).restype = n
        _lib = L
    return _lib


def _same_device(**tensors) -> torch.device:
    first = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be in device memory (got {t.device})")
        index = t.get_device()
        if first is None:
            first = index
        elif index != first:
            raise ValueError(f"{name} is on device {index}, the other tensors on {first}")
    return torch.device("cuda", first)


class _On:
    """The tensors' device made current, where it is not."""

    def __init__(self, device):
        self.device = device if device.index != torch.cuda.current_device() else None

    def __enter__(self):
        if self.device is not None:
            self.guard = torch.cuda.device(self.device)
            self.guard.__enter__()

    def __exit__(self, *error):
        if self.device is not None:
            self.guard.__exit__(*error)


def _scan_shape(rule: str, q, v, cu_seqlens):
    """(n_seq, tokens, leading shape, heads, key_heads, d_k, d_v) of a call:
    [tokens, heads, d] arrays with cu_seqlens, [n_seq, length, heads, d]
    arrays without."""
    if rule not in RULES:
        raise ValueError(f"unknown rule {rule!r}")
    want = 3 if cu_seqlens is not None else 4
    if v.dim() != want or q.dim() != want:
        raise ValueError(f"q and v must have {want} dimensions (packed [tokens, heads, d] with "
                         f"cu_seqlens, [sequences, length, heads, d] without)")
    lead = tuple(v.shape[:-2])
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
            raise ValueError("cu_seqlens must hold n_seq + 1 offsets")
        n_seq = cu_seqlens.shape[0] - 1
    else:
        n_seq = lead[0]
    tokens = 1
    for x in lead:
        tokens *= x
    if tokens > 0x7fffffff:
        raise ValueError("more than 2^31 - 1 tokens")
    return n_seq, tokens, lead, v.shape[-2], q.shape[-2], q.shape[-1], v.shape[-1]


def _scan_inputs(rule, q, k, v, g, beta, S0, cu_seqlens):
    n_seq, tokens, lead, H, HK, d_k, d_v = _scan_shape(rule, q, v, cu_seqlens)
    _need(q, "q", (*lead, HK, d_k), _IN)
    _need(k, "k", (*lead, HK, d_k), (q.dtype,))
    _need(v, "v", (*lead, H, d_v), (q.dtype,))
    _need(g, "g", (*lead, H, d_k) if rule == "kda" else (*lead, H), _F32)
    if beta is not None:
        _need(beta, "beta", (*lead, H), _F32)
    if S0 is not None:
        _need(S0, "S0", (n_seq, H, d_k, d_v), _F32)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", (n_seq + 1,), (torch.int32,))
    return n_seq, tokens, lead, H, HK, d_k, d_v


def _workspace_bytes(rule, n_seq, H, HK, d_k, d_v, tokens, backward: bool) -> int:
    n = int(lib().seed_scan_workspace_bytes(RULES[rule], n_seq, H, HK, d_k, d_v, tokens,
                                            1 if backward else 0))
    if n == ctypes.c_size_t(-1).value:
        raise ValueError(binding.lib().seed_last_error().decode())
    return n


def _workspace(workspace, nbytes: int, device, stream) -> torch.Tensor:
    if workspace is None:
        # from the pool of the stream that uses it: that of torch's current
        # stream may hand out memory which that stream is still using
        with torch.cuda.stream(stream):
            return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if workspace.dtype != torch.uint8 or workspace.dim() != 1 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 vector")
    return workspace


def scan_workspace(rule: str, q, v, n_seq: int, backward: bool = False) -> torch.Tensor:
    """A workspace for seed_scan (or seed_scan_backward) calls of these
    shapes: q [..., key_heads, d_k], v [..., heads, d_v] in n_seq sequences."""
    lead = v.shape[:-2].numel()
    return torch.empty(_workspace_bytes(rule, n_seq, v.shape[-2], q.shape[-2], q.shape[-1],
                                        v.shape[-1], lead, backward),
                       dtype=torch.uint8, device=v.device)


def seed_scan(rule: str, q, k, v, g, beta, o, S, S0=None, cu_seqlens=None, workspace=None,
              stream=None) -> None:
    """Run the recurrence over sequences into o and the last states S
    [n_seq, heads, d_k, d_v] (see include/seed_sequence.h).  q, k are
    [tokens, key_heads, d_k], v and o [tokens, heads, d_v], with cu_seqlens
    (int32, n_seq + 1 offsets); without it [n_seq, length, ...]."""
    device = _same_device(q=q, k=k, v=v, g=g, beta=beta, o=o, S=S, S0=S0, cu_seqlens=cu_seqlens,
                          workspace=workspace)
    n_seq, tokens, lead, H, HK, d_k, d_v = _scan_inputs(rule, q, k, v, g, beta, S0, cu_seqlens)
    _need(o, "o", (*lead, H, d_v), (q.dtype,))
    _need(S, "S", (n_seq, H, d_k, d_v), _F32)
    with _On(device):
        ws = _workspace(workspace, _workspace_bytes(rule, n_seq, H, HK, d_k, d_v, tokens, False),
                        device, stream)
        st = lib().seed_scan(RULES[rule], n_seq, H, HK, d_k, d_v, tokens, _ptr(cu_seqlens),
                             _ptr(q), _ptr(k), _ptr(v), 1 if q.dtype == torch.bfloat16 else 0,
                             _ptr(g), _ptr(beta), _ptr(S0), _ptr(o), _ptr(S), _ptr(ws),
                             ws.numel(), _stream(stream, device.index))
    _check("seed_scan", st)


def seed_scan_backward(rule: str, q, k, v, g, beta, do, dq, dk, dv, dg, dbeta, S0=None, dS=None,
                       dS0=None, cu_seqlens=None, workspace=None, stream=None) -> None:
    """Gradients of seed_scan's inputs from do (the gradient of o) and dS
    (that of S) into dq, dk, dv, dg, dbeta and, where given, dS0 (see
    include/seed_sequence.h).  Shapes and types are the inputs'."""
    device = _same_device(q=q, k=k, v=v, g=g, beta=beta, do=do, dq=dq, dk=dk, dv=dv, dg=dg,
                          dbeta=dbeta, S0=S0, dS=dS, dS0=dS0, cu_seqlens=cu_seqlens,
                          workspace=workspace)
    n_seq, tokens, lead, H, HK, d_k, d_v = _scan_inputs(rule, q, k, v, g, beta, S0, cu_seqlens)
    _need(do, "do", (*lead, H, d_v), (q.dtype,))
    _need(dq, "dq", (*lead, HK, d_k), (q.dtype,))
    _need(dk, "dk", (*lead, HK, d_k), (q.dtype,))
    _need(dv, "dv", (*lead, H, d_v), (q.dtype,))
    _need(dg, "dg", tuple(g.shape), _F32)
    if dbeta is not None:
        _need(dbeta, "dbeta", (*lead, H), _F32)
    for name, t in (("dS", dS), ("dS0", dS0)):
        if t is not None:
            _need(t, name, (n_seq, H, d_k, d_v), _F32)
    with _On(device):
        ws = _workspace(workspace, _workspace_bytes(rule, n_seq, H, HK, d_k, d_v, tokens, True),
                        device, stream)
        st = lib().seed_scan_backward(
            RULES[rule], n_seq, H, HK, d_k, d_v, tokens, _ptr(cu_seqlens), _ptr(q), _ptr(k),
            _ptr(v), 1 if q.dtype == torch.bfloat16 else 0, _ptr(g), _ptr(beta), _ptr(S0),
            _ptr(do), _ptr(dS), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta), _ptr(dS0),
            _ptr(ws), ws.numel(), _stream(stream, device.index))
    _check("seed_scan_backward", st)


def _norm_inputs(x, gate, io, weight, bias, activation):
    if x.dim() < 2:
        raise ValueError("x must be [..., groups, d]")
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    shape = tuple(x.shape)
    G, d = shape[-2:]
    rows = x.shape[:-2].numel()
    _need(x, "x", shape, _IN)
    if gate is not None:
        _need(gate, "gate", shape, (io,))
    wg = 1
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            if tuple(t.shape) not in ((d,), (G, d)):
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({d},) or ({G}, {d})")
            _need(t, name, tuple(t.shape), _F32)
            wg = t.shape[0] if t.dim() == 2 else 1
    if weight is not None and bias is not None and weight.shape != bias.shape:
        raise ValueError("weight and bias must have one shape")
    return shape, rows, G, d, wg


def _code(dtype) -> int:
    return 1 if dtype == torch.bfloat16 else 0


def seed_group_norm(x, y, weight=None, bias=None, gate=None, eps: float = 1e-5,
                    centered: bool = False, activation="silu", gate_first: bool = False,
                    stream=None) -> None:
    """Group norm of x [..., groups, d] with a gate and an activation into y
    (see include/seed_sequence.h): n = norm(x) weight + bias, y = n act(gate)
    (act(n) without a gate; gate_first normalises x act(gate)).  weight and
    bias are [d] or [groups, d] float32; gate and y share one type."""
    device = _same_device(x=x, y=y, weight=weight, bias=bias, gate=gate)
    shape, rows, G, d, wg = _norm_inputs(x, gate, y.dtype, weight, bias, activation)
    _need(y, "y", shape, _IN)
    with _On(device):
        st = lib().seed_group_norm(rows, G, d, _ptr(x), _code(x.dtype), _ptr(gate), _code(y.dtype),
                                   _ptr(weight), _ptr(bias), wg, eps, int(centered),
                                   ACTIVATIONS[activation], int(gate_first), _ptr(y),
                                   _stream(stream, device.index))
    _check("seed_group_norm", st)


def group_norm_workspace(x, weight=None) -> torch.Tensor:
    """A workspace for seed_group_norm_backward calls on x with weights of
    weight's shape (None: shared)."""
    G, d = x.shape[-2:]
    n = int(lib().seed_group_norm_workspace_bytes(x.shape[:-2].numel(), G, d,
                                                  weight.shape[0] if weight is not None
                                                  and weight.dim() == 2 else 1))
    if n == ctypes.c_size_t(-1).value:
        raise ValueError(binding.lib().seed_last_error().decode())
    return torch.empty(n, dtype=torch.uint8, device=x.device)


def seed_group_norm_backward(dy, x, dx, dgate=None, dweight=None, dbias=None, weight=None,
                             bias=None, gate=None, eps: float = 1e-5, centered: bool = False,
                             activation="silu", gate_first: bool = False, workspace=None,
                             stream=None) -> None:
    """Gradients of seed_group_norm from dy into dx, dgate (with a gate) and,
    where given, dweight and dbias (see include/seed_sequence.h)."""
    device = _same_device(dy=dy, x=x, dx=dx, dgate=dgate, dweight=dweight, dbias=dbias,
                          weight=weight, bias=bias, gate=gate, workspace=workspace)
    shape, rows, G, d, wg = _norm_inputs(x, gate, dy.dtype, weight, bias, activation)
    _need(dy, "dy", shape, _IN)
    _need(dx, "dx", shape, (x.dtype,))
    if dgate is not None:
        _need(dgate, "dgate", shape, (dy.dtype,))
    like = weight if weight is not None else bias
    for name, t in (("dweight", dweight), ("dbias", dbias)):
        if t is not None:
            if like is None:
                like = t
                if tuple(t.shape) not in ((d,), (G, d)):
                    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({d},) or "
                                     f"({G}, {d})")
                wg = t.shape[0] if t.dim() == 2 else 1
            _need(t, name, tuple(like.shape), _F32)
    with _On(device):
        ws = None
        if dweight is not None or dbias is not None:
            if workspace is None:
                with torch.cuda.stream(stream):
                    ws = group_norm_workspace(x, like)
            else:
                ws = _workspace(workspace, 0, device, stream)
        st = lib().seed_group_norm_backward(
            rows, G, d, _ptr(dy), _ptr(x), _code(x.dtype), _ptr(gate), _code(dy.dtype),
            _ptr(weight), _ptr(bias), wg, eps, int(centered), ACTIVATIONS[activation],
            int(gate_first), _ptr(dx), _ptr(dgate), _ptr(dweight), _ptr(dbias), _ptr(ws),
            0 if ws is None else ws.numel(), _stream(stream, device.index))
    _check("seed_group_norm_backward", st)
