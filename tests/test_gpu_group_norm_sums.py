"""The weights' gradients of the gated group norm, column by column: sums over
rows in registers, over a block's teams and over the blocks' parts.

Tolerance: each of a column's terms dn hat (dn for the bias) is within
TOL = 4e-6 of its scale (test_gpu_group_norm.py; the scale of hat is the
group's largest, of SiLU the sum of its terms), and the sums run over at most
64 terms in order and then in trees: with 2^-24 a rounding 4e-6 and 4e-6, under
1e-5 of the sum of the terms' sizes."""
import numpy as np
import pytest
import torch

from gpu_util import f64, requires_gpu
from oracle import seed_sequence as oseq
from sink_rank_recurrent_amd import sequence
from test_gpu_group_norm import close, make

pytestmark = [pytest.mark.gpu, requires_gpu]

FLAGS = {"eps": 1e-5, "centered": True, "activation": "silu", "gate_first": False}


def check_backward(case, dy):
    out = {k: torch.full_like(v, 7.0) for k, v in case.items() if v is not None}
    sequence.seed_group_norm_backward(dy, case["x"], out["x"], dgate=out["gate"], dweight=out["weight"],
                                      dbias=out["bias"], weight=case["weight"], bias=case["bias"],
                                      gate=case["gate"], **FLAGS)
    a = {k: f64(v) for k, v in case.items()}
    want = oseq.group_norm(**a, **FLAGS, dy=f64(dy))
    for name in ("x", "gate"):
        close(out[name], want[name], name, want[name + "_scale"])
    x = a["x"] - a["x"].mean(-1, keepdims=True)
    hat = np.abs(x) / np.sqrt((x * x).mean(-1, keepdims=True) + FLAGS["eps"])
    dn = np.abs(f64(dy) * a["gate"] / (1 + np.exp(-a["gate"])))
    over = (0, 1) if a["weight"].ndim == 1 else (0,)
    for name, size in (("weight", dn * hat.max(-1, keepdims=True)), ("bias", dn)):
        err = np.abs(f64(out[name]) - want[name])
        assert (err <= 1e-5 * size.sum(over)).all(), (name, float((err / size.sum(over)).max()))


def test_more_columns_than_one_grid():
    """40 groups of 4096 channels, weights of their own: 327680 columns, more
    than the 262144 that the blocks of one grid sum in one go."""
    check_backward(*make(3, 40, 4096, torch.bfloat16, torch.bfloat16, True, False, True, 6))


@pytest.mark.parametrize("d", [2047, 2048, 64, 128])
@pytest.mark.parametrize("shared", [False, True])
def test_every_item_counts_once(d, shared):
    """More items than blocks, so that a block takes several, also where a
    team is a whole block that sums through LDS (d > 1024): forwards and
    backwards."""
    rows = 2100 if d > 1024 else 9000
    groups = 2 if d > 1024 else 4
    types = (torch.float32, torch.float32) if d % 8 else (torch.bfloat16, torch.bfloat16)
    case, dy = make(rows, groups, d, *types, True, shared, True, 7)
    y = torch.full_like(dy, 7.0)
    sequence.seed_group_norm(case["x"], y, weight=case["weight"], bias=case["bias"], gate=case["gate"], **FLAGS)
    close(y, oseq.group_norm(**{k: f64(v) for k, v in case.items()}, **FLAGS), "y")
    check_backward(case, dy)


@pytest.mark.parametrize("d", [2047, 128])
@pytest.mark.parametrize("shared", [False, True])
def test_sums_of_ones(d, shared):
    """dy of 1, a gate whose sigmoid is 1 and groups of +-1: dbias is the
    number of rows (times groups) exactly, dweight the sum of signs: whole
    numbers of at most 9003, their terms within two roundings of 1 and the
    sums' own errors 9003 2^-22 together, far from half of one item."""
    rows, groups = 3001, 3
    gen = torch.Generator("cuda").manual_seed(8)
    x = torch.randint(0, 2, (rows, groups, d), device="cuda", generator=gen).float() * 2 - 1
    gate = torch.full_like(x, 100.0)
    w = torch.ones((d,) if shared else (groups, d), device="cuda")
    dx, dz, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    sequence.seed_group_norm_backward(torch.ones_like(x), x, dx, dgate=dz, dweight=dw, dbias=db, weight=w,
                                      gate=gate, eps=0.0, centered=False, activation="sigmoid",
                                      gate_first=False)
    over = (0, 1) if shared else (0,)
    assert torch.equal(db, torch.full_like(db, float(rows * (groups if shared else 1))))
    assert np.abs(f64(dw) - f64(x).sum(over)).max() < 0.5
