"""What the recurrence's forward pass keeps of 32 bits, with bf16 inputs: the
last state against the norm it has, and the read-outs against the nearest bf16.

Inputs that show it: gates near 1 and of 1 (nothing is forgotten), and keys
with a common direction (each token corrects what the ones before wrote).

Tolerances.  512 tokens are 8 chunks.  In a chunk a value of the state and of
what is written to it goes through some 32 roundings (13 matrix instructions
and products on the state itself, the rest on the corrections): 256 in all, at
random sqrt(256) 2^-24 = 9.5e-7 of the norm, and 1e-6 is what the header says.
A read-out has 26 of its own, 2^-24 / sqrt(3) each on average, and the
state's share, sqrt(26 + 256) 2^-24 / sqrt(3) = 5.8e-7 of its unit's root mean
square.  It goes to another bf16 where it passes the middle between two: one
of 2 e rms / step, step at least 2^-8 |x|, and rms / |x| is 5 on average (0.8 ln
of the range, 2^-8 of the rms and up); so one in 650, 1.5e-3."""
import numpy as np
import pytest
import torch

from gpu_util import f64, requires_gpu
from oracle import seed_sequence as oseq
from sink_rank_recurrent_amd import sequence
from test_gpu_scan import RULES

pytestmark = [pytest.mark.gpu, requires_gpu]

T, H = 512, 4


def inputs(rule, kind, d_k, d_v):
    gen = torch.Generator("cuda").manual_seed(3)

    def normal(*s):
        return torch.randn(*s, device="cuda", generator=gen)

    def uniform(*s):
        return torch.rand(*s, device="cuda", generator=gen)

    unit = torch.nn.functional.normalize
    k = unit(normal(T, H, d_k), dim=-1)
    if kind == "common keys":
        k = unit(k + unit(normal(1, H, d_k), dim=-1), dim=-1)
    low, high = {"gates near 1": (0.99, 1.0), "gates of 1": (1.0, 1.0)}.get(kind, (0.9, 0.999))
    return {"q": unit(normal(T, H, d_k), dim=-1).bfloat16(), "k": k.bfloat16(),
            "v": (normal(1, H, d_v) + 0.3 * normal(T, H, d_v)).bfloat16(),
            "g": low + (high - low) * uniform(*((T, H, d_k) if rule == "kda" else (T, H))),
            "beta": None if rule == "mamba2" else uniform(T, H), "S0": None}


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("kind", ["far", "gates near 1", "gates of 1", "common keys"])
@pytest.mark.parametrize("batch", [1, 64])
def test_states_and_readouts_of_bf16_inputs(rule, kind, batch):
    """As one sequence (in segments) and as the first of 64 (whole, by eight
    waves where d_v is 128)."""
    d_k, d_v = 128, 64 if rule == "mamba2" else 128
    x = inputs(rule, kind, d_k, d_v)
    many = {k: None if v is None else v.repeat(batch, *[1] * (v.dim() - 1)) for k, v in x.items()}
    o = torch.empty_like(many["v"])
    S = torch.empty(batch, H, d_k, d_v, device="cuda")
    cu = torch.arange(0, batch * T + 1, T, dtype=torch.int32, device="cuda")
    sequence.seed_scan(rule, many["q"], many["k"], many["v"], many["g"], many["beta"], o, S,
                       cu_seqlens=cu)
    want_o, want_S = oseq.scan(rule, **{k: None if v is None else f64(v) for k, v in x.items()},
                               offsets=[0, T])
    err = np.linalg.norm(f64(S[:1]) - want_S, axis=(2, 3)) / np.linalg.norm(want_S, axis=(2, 3))
    assert err.max() <= 1e-6, err
    nearest = torch.tensor(want_o).to(torch.bfloat16)
    assert (nearest != o[:T].cpu()).double().mean() <= 1.5e-3
    assert torch.equal(o.view(batch, T, H, d_v)[1:], o[:T].expand(batch - 1, T, H, d_v))
    assert torch.equal(S[1:], S[:1].expand(batch - 1, H, d_k, d_v))
