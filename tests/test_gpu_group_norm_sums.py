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
