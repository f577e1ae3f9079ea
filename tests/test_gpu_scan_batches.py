"""The recurrence on batches that fill the chip (256 and more sequences x
heads: eight waves walk a head of 128 columns), on batches of many sequences
(the search for a chunk's sequence goes 64 at a time), with gates per key
channel on both sides of what is divided by, and with offsets that break
their order.  Tolerances: test_gpu_scan.py."""
import numpy as np
import pytest
import torch

from gpu_util import f64, requires_gpu
from oracle import seed_sequence as oseq
from sink_rank_recurrent_amd import sequence
from test_gpu_scan import RULES, check, host, inputs, run, run_back

pytestmark = [pytest.mark.gpu, requires_gpu]


def both_ways(rule, x, offsets, seed):
    n, H = len(offsets) - 1, x["v"].shape[1]
    d_k, d_v = x["q"].shape[2], x["v"].shape[2]
    o, S = run(rule, x, offsets)
    h = host(x)
    want_o, want_S = oseq.scan(rule, **h, offsets=offsets)
    check(o, want_o, offsets, "o")
    check(S, want_S, offsets, "S")
    gen = torch.Generator(device="cuda").manual_seed(seed)
    do = torch.randn(x["v"].shape, device="cuda", generator=gen).to(x["v"].dtype)
    dS = torch.randn(n, H, d_k, d_v, device="cuda", generator=gen)
    got = run_back(rule, x, offsets, do, dS)
    want = oseq.scan_backward(rule, **h, offsets=offsets, do=f64(do), dS=f64(dS))
    for name in got:
        check(got[name], want[name], offsets, name, terms=want.get(name + "_scale"))


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_short_sequences(rule, dtype):
    """70 sequences of 0 to 130 tokens, four heads on two key heads, rows
    before the first and behind the last."""
    lengths = np.random.default_rng(5).permutation(np.concatenate(
        [[0, 0, 0, 1, 1, 63, 64, 64, 65, 127, 128, 129, 130], np.arange(2, 116, 2)]))
    offsets = [3] + [int(e) for e in 3 + np.cumsum(lengths)]
    assert len(offsets) == 71
    x = inputs(rule, offsets[-1] + 5, 4, 2, 128, 128, 70, dtype, 41)
    both_ways(rule, x, offsets, 42)


@pytest.mark.parametrize("rule", RULES)
def test_thousands_of_sequences(rule):
    """4200 sequences of no, one or two tokens."""
    rng = np.random.default_rng(6)
    offsets = [0] + [int(e) for e in np.cumsum(rng.integers(0, 3, 4200))]
    x = inputs(rule, offsets[-1], 1, 1, 64, 64, 4200, torch.bfloat16, 43)
    o, S = run(rule, x, offsets)
    want_o, want_S = oseq.scan(rule, **host(x), offsets=offsets)
    check(o, want_o, offsets, "o")
    check(S, want_S, offsets, "S")


@pytest.mark.parametrize("dims", [(128, 128), (128, 64), (64, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gates", ["0.3 to 0.9", "0.5 to 0.6", "0.05 to 1", "one of 0.1", "one channel of 0.01"])
def test_gates_per_channel_between(dims, dtype, gates):
    """Chunks whose products stay above 2^-60 and those whose do not, and
    (backward) single gates below 1/4 in a chunk that is divided by."""
    offsets = [0, 130, 200]
    x = inputs("kda", 200, 2, 2, *dims, 2, dtype, 44)
    gen = torch.Generator(device="cuda").manual_seed(45)
    u = torch.rand(x["g"].shape, device="cuda", generator=gen)
    if " to " in gates:
        low, high = map(float, gates.split(" to "))
        x["g"] = low + (high - low) * u
    elif gates == "one of 0.1":
        x["g"][100, 1, 5] = 0.1
        x["g"][150, 0, 63] = 0.1
    else:
        x["g"][64:128, 0, 7] = 0.01
    both_ways("kda", x, offsets, 46)


class Fenced:
    """Arrays inside larger ones whose other values are watched."""

    def __init__(self):
        self.all = []

    def __call__(self, like=None, nbytes=None):
        n = nbytes if like is None else like.numel()
        dtype = torch.uint8 if like is None else like.dtype
        fence = 4096
        whole = torch.full((n + 2 * fence,), 7, dtype=dtype, device="cuda")
        self.all.append((whole, fence, n))
        part = whole[fence:fence + n]
        return part if like is None else part.view(like.shape)

    def whole(self):
        return all(bool((w[:f] == 7).all()) and bool((w[f + n:] == 7).all()) for w, f, n in self.all)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,offsets", [
    (200, [150, 20, 190, -7, 2 ** 31 - 1, 64]),
    (200, [-2 ** 31, -1, 300, 200, 0, 200]),
    (2600, [2500, 0, 2600, 70, 70, -1]),          # in segments
    (2600, [0, 2600, 0, 2600, 1300, 2 ** 31 - 1])])
def test_offsets_out_of_order_stay_inside(rule, dtype, tokens, offsets):
    """Wrong results, but every write inside its array, and the next call
    with good offsets and the same workspace is right."""
    n, H = len(offsets) - 1, 2
    x = inputs(rule, tokens, H, 1, 64, 64, n, dtype, 47)
    fenced = Fenced()
    o, S = fenced(x["v"]), fenced(x["S0"])
    out = {k: fenced(v) for k, v in x.items() if v is not None}
    ws = fenced(nbytes=sequence.scan_workspace(rule, x["q"], x["v"], n, backward=True).numel())
    do = torch.randn(x["v"].shape, device="cuda").to(dtype)
    dS = torch.randn(n, H, 64, 64, device="cuda")

    def call(cu):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        sequence.seed_scan(rule, x["q"], x["k"], x["v"], x["g"], x["beta"], o, S, S0=x["S0"], cu_seqlens=cu,
                           workspace=ws)
        sequence.seed_scan_backward(rule, x["q"], x["k"], x["v"], x["g"], x["beta"], do, out["q"], out["k"],
                                    out["v"], out["g"], out.get("beta"), S0=x["S0"], dS=dS, dS0=out["S0"],
                                    cu_seqlens=cu, workspace=ws)
        torch.cuda.synchronize()

    call(offsets)
    assert fenced.whole()
    good = [0, tokens // 3, tokens // 3, tokens - 70, tokens - 69, tokens]
    call(good)
    assert fenced.whole()
    h = host(x)
    want_o, want_S = oseq.scan(rule, **h, offsets=good)
    check(o, want_o, good, "o")
    check(S, want_S, good, "S")
    want = oseq.scan_backward(rule, **h, offsets=good, do=f64(do), dS=f64(dS))
    for name in out:
        check(out[name], want[name], good, name, terms=want.get(name + "_scale"))
