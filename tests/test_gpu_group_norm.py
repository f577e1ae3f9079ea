"""The gated group norm and its backward pass against the float64 oracle.

Tolerances: n is a product of three fp32 factors (the statistic a sum of up
to 8192 squares in a tree of at most 32 serial additions) and the activation
has its argument and exponential rounded: 64 roundings of 2^-24 and an
exponential's argument of up to 8 give 4e-6 of a value's scale, taken
relative to the group's largest value, or, for a gradient that is a difference
of larger terms, to their size (a group of one channel without a mean has
dh = rstd dhat (1 - hat^2), hat^2 = 1 - eps rstd^2: the terms stay, the
difference all but vanishes; SiLU's slope is s + x s (1 - s), two terms of
opposite sign around x = -1.28).  dweight and dbias sum up to `rows`
values in runs of at most 64 in order: 1e-5 of the sum of magnitudes.  A
16-bit output adds half a step of its value, 2^-8."""
import numpy as np
import pytest
import torch

from gpu_util import f64, requires_gpu
from oracle import seed_sequence as oseq
from sink_rank_recurrent_amd import sequence

pytestmark = [pytest.mark.gpu, requires_gpu]

TOL = 4e-6


def make(rows, G, d, x_t, io_t, gate, shared, bias, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, device="cuda", generator=gen)

    w = (d,) if shared else (G, d)
    return {"x": (normal(rows, G, d) + 0.5).to(x_t), "gate": normal(rows, G, d).to(io_t) if gate else None,
            "weight": 1 + 0.2 * normal(*w), "bias": 0.2 * normal(*w) if bias else None}, \
        normal(rows, G, d).to(io_t)


def close(got, want, name, terms=None):
    half = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    scale = np.abs(want).max(-1, keepdims=True)
    if terms is not None:
        scale = np.maximum(scale, terms.max(-1, keepdims=True))
    # below the smallest normal fp32 number a value may be flushed to 0
    err = np.abs(f64(got) - want) - half * (1 + TOL) * np.abs(want) - TOL * scale - 2.0 ** -126
    assert err.max(initial=0.0) <= 0, (name, float(err.max()))


def both(case, dy, flags):
    a = {k: None if v is None else f64(v) for k, v in case.items()}
    y = torch.full_like(dy, 7.0)
    sequence.seed_group_norm(case["x"], y, weight=case["weight"], bias=case["bias"],
                             gate=case["gate"], **flags)
    close(y, oseq.group_norm(**a, **flags), "y")
    out = {k: torch.full_like(v, 7.0) for k, v in case.items() if v is not None}
    out.setdefault("bias", torch.full_like(case["weight"], 7.0))
    sequence.seed_group_norm_backward(dy, case["x"], out["x"], dgate=out.get("gate"),
                                      dweight=out["weight"], dbias=out["bias"], weight=case["weight"],
                                      bias=case["bias"], gate=case["gate"], **flags)
    want = oseq.group_norm(**a, **flags, dy=f64(dy))
    for name in ("x", "gate"):
        if name in out:
            close(out[name], want[name], name, want.get(name + "_scale"))
    m = np.abs(f64(dy)).sum(0)
    for name in ("weight", "bias"):
        size = (m.sum(0) if case["weight"].dim() == 1 else m).max()
        assert np.abs(f64(out[name]) - want[name]).max() <= 1e-5 * 8 * size, name
    return y, out


@pytest.mark.parametrize("gate", ["none", "after", "before"])
@pytest.mark.parametrize("activation", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("centered", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_forms(gate, activation, centered, shared):
    case, dy = make(37, 3, 128, torch.float32, torch.float32, gate != "none", shared, True, 1)
    both(case, dy, {"eps": 1e-5, "centered": centered, "activation": activation,
                    "gate_first": gate == "before"})


@pytest.mark.parametrize("d", [1, 7, 64, 65, 120, 256, 257, 512, 1000, 1023, 1024, 2040, 2047, 4096,
                               4099, 8192, 8191])
@pytest.mark.parametrize("types", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.bfloat16),
                                   (torch.bfloat16, torch.float32)], ids=str)
def test_widths_and_types(d, types):
    case, dy = make(5, 2, d, *types, True, False, False, 2)
    both(case, dy, {"eps": 1e-5, "centered": d > 1, "activation": "silu", "gate_first": False})


@pytest.mark.parametrize("rows", [0, 1, 2, 300, 9000])
@pytest.mark.parametrize("shared", [False, True])
def test_rows(rows, shared):
    case, dy = make(rows, 4, 64, torch.bfloat16, torch.bfloat16, True, shared, True, 3)
    _, out = both(case, dy, {"eps": 1e-6, "centered": False, "activation": "silu",
                             "gate_first": False}) if rows else _no_rows(case, dy)
    if not rows:
        assert not out["weight"].any() and not out["bias"].any()


def _no_rows(case, dy):
    out = {k: torch.full_like(v, 7.0) for k, v in case.items()}
    sequence.seed_group_norm(case["x"], torch.empty_like(dy), weight=case["weight"], bias=case["bias"],
                             gate=case["gate"])
    sequence.seed_group_norm_backward(dy, case["x"], out["x"], dgate=out["gate"], dweight=out["weight"],
                                      dbias=out["bias"], weight=case["weight"], bias=case["bias"],
                                      gate=case["gate"])
    return None, out


def test_no_weights_and_far_gates():
    """Without weight and bias; gates so far out that the activation is 0 or
    the gate itself, and a constant group (variance 0)."""
    case, dy = make(6, 2, 128, torch.float32, torch.float32, True, True, False, 4)
    case["gate"][0] = 200.0
    case["gate"][1] = -200.0
    case["x"][2] = 3.0
    flags = {"eps": 1e-5, "centered": True, "activation": "silu", "gate_first": False}
    case["weight"] = None
    a = {k: None if v is None else f64(v) for k, v in case.items()}
    y = torch.empty_like(dy)
    sequence.seed_group_norm(case["x"], y, gate=case["gate"], **flags)
    close(y, oseq.group_norm(**a, **flags), "y")
    dx, dz = torch.empty_like(dy), torch.empty_like(dy)
    sequence.seed_group_norm_backward(dy, case["x"], dx, dgate=dz, gate=case["gate"], **flags)
    want = oseq.group_norm(**a, **flags, dy=f64(dy))
    close(dz, want["gate"], "gate", want["gate_scale"])
    close(dx[[0, 1, 3, 4, 5]], want["x"][[0, 1, 3, 4, 5]], "x")


def test_in_place_and_graph():
    case, dy = make(200, 4, 128, torch.bfloat16, torch.bfloat16, True, True, True, 5)
    flags = {"eps": 1e-5, "centered": False, "activation": "silu", "gate_first": False}
    args = {"weight": case["weight"], "bias": case["bias"], **flags}
    y = torch.empty_like(dy)
    sequence.seed_group_norm(case["x"], y, gate=case["gate"], **args)
    x2 = case["x"].clone()
    sequence.seed_group_norm(x2, x2, gate=case["gate"], **args)
    assert torch.equal(y, x2)

    def back(out):
        sequence.seed_group_norm_backward(dy, case["x"], out[0], dgate=out[1], dweight=out[2],
                                          dbias=out[3], gate=case["gate"], **args)

    def buffers():
        return [torch.zeros_like(dy), torch.zeros_like(dy), torch.zeros(128, device="cuda"),
                torch.zeros(128, device="cuda")]

    ref, cap = buffers(), buffers()
    back(ref)
    torch.cuda.synchronize()
    dx, dz = case["x"].clone(), dy.clone()
    dw, db = torch.empty(128, device="cuda"), torch.empty(128, device="cuda")
    sequence.seed_group_norm_backward(dz, dx, dx, dgate=dz, dweight=dw, dbias=db, gate=case["gate"],
                                      **args)
    assert all(torch.equal(a, b) for a, b in zip(ref, (dx, dz, dw, db)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        back(cap)
    for _ in range(3):
        for t in cap:
            t.zero_()
        eager = buffers()
        back(eager)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, cap))
        assert all(torch.equal(a, b) for a, b in zip(ref, eager))
