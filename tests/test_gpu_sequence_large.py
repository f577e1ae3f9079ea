"""Arrays of more than 2^31 values: the last sequences and rows of a batch have
the bits that they have alone, so no offset is cut to 32 bits.  And the most
heads that a call takes."""
import pytest
import torch

from gpu_util import requires_gpu
from oracle import seed_sequence as oseq
from sink_rank_recurrent_amd import sequence
from test_gpu_scan import check, host, inputs

pytestmark = [pytest.mark.gpu, requires_gpu]


@pytest.fixture(autouse=True)
def memory():
    """Room before, and none kept after."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 200 << 30:
        pytest.skip("needs 200 GB of device memory")
    yield
    torch.cuda.empty_cache()


def outputs(x, n, H, d_k, d_v):
    out = {k: torch.full_like(v, 7.0) for k, v in x.items() if v is not None}
    return out, torch.full_like(x["v"], 7.0), torch.full((n, H, d_k, d_v), 7.0, device="cuda")


def run(rule, x, do, offsets, n, H, d):
    out, o, S = outputs(x, n, H, d, d)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    args = x["q"], x["k"], x["v"], x["g"], x["beta"]
    sequence.seed_scan(rule, *args, o, S, cu_seqlens=cu)
    dS0 = torch.empty_like(S)
    sequence.seed_scan_backward(rule, *args, do, out["q"], out["k"], out["v"], out["g"], out.get("beta"),
                                dS0=dS0, cu_seqlens=cu)
    torch.cuda.synchronize()
    return {**out, "o": o, "S": S, "dS0": dS0}


@pytest.mark.parametrize("rule,dtype", [("gdn", torch.bfloat16), ("mamba2", torch.float32),
                                        ("kda", torch.bfloat16)])
def test_last_sequences_of_a_large_batch(rule, dtype):
    H, d, n, L = 128, 128, 128, 1025
    T = n * L
    assert T * H * d > 1 << 31
    x = inputs(rule, T, H, H, d, d, n, dtype, 61, initial=False)
    do = torch.randn(x["v"].shape, device="cuda", dtype=dtype)
    offsets = [L * i for i in range(n + 1)]
    got = run(rule, x, do, offsets, n, H, d)
    tail = {k: None if v is None else v[-2 * L:].clone() for k, v in x.items()}
    want = run(rule, tail, do[-2 * L:].clone(), [0, L, 2 * L], 2, H, d)
    for name, w in want.items():
        assert torch.equal(got[name][-w.shape[0]:], w), name
        assert not (w == 7.0).all(), name


def test_last_rows_of_a_large_norm():
    rows, G, d = (1 << 17) + 77, 128, 128
    assert rows * G * d > 1 << 31
    x = torch.randn(rows, G, d, device="cuda", dtype=torch.bfloat16)
    gate, dy = torch.randn_like(x), torch.randn_like(x)
    w = 1 + 0.1 * torch.randn(G, d, device="cuda")

    def both(a, z, g):
        y, dx, dz = (torch.full_like(a, 7.0) for _ in range(3))
        dw = torch.empty_like(w)
        sequence.seed_group_norm(a, y, weight=w, gate=z)
        sequence.seed_group_norm_backward(g, a, dx, dgate=dz, dweight=dw, weight=w, gate=z)
        torch.cuda.synchronize()
        return (y, dx, dz), dw

    got, dw = both(x, gate, dy)
    want, _ = both(x[-100:].clone(), gate[-100:].clone(), dy[-100:].clone())
    for a, b in zip(got, want):
        assert torch.equal(a[-100:], b)
    half = sum(both(x[i::2].contiguous(), gate[i::2].contiguous(), dy[i::2].contiguous())[1] for i in (0, 1))
    # both sides within 1e-5 of a column's sum of magnitudes, at most 0.8 a row
    # (the mean of |dy|; |act(gate)| and |hat| are below 1 on average)
    assert (dw - half).abs().max() <= 2e-5 * 0.8 * rows


def test_most_heads():
    """65535 heads on five key heads: one token is the dense step."""
    H, HK, d = 65535, 5, 64
    x = inputs("gdn", 2, H, HK, d, d, 2, torch.bfloat16, 62)
    o, S = torch.empty_like(x["v"]), torch.empty_like(x["S0"])
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    sequence.seed_scan("gdn", x["q"], x["k"], x["v"], x["g"], x["beta"], o, S, S0=x["S0"], cu_seqlens=cu)
    for h in (0, 13106, 13107, 40000, 65534):
        one = {k: v[:, h:h + 1] if k not in ("q", "k") else v[:, h // 13107:h // 13107 + 1] for k, v in x.items()}
        want_o, want_S = oseq.scan("gdn", **host(one), offsets=[0, 1, 2])
        check(o[:, h:h + 1], want_o, [0, 1, 2], "o")
        check(S[:, h:h + 1], want_S, [0], "S")
