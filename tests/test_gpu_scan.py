"""The recurrence over sequences and its backward pass against the float64
oracle.

Tolerances, per (sequence, head) unit of an output, relative to the unit's
largest value.  Every fp32 result is a chain of at most four products, each a
sum of up to 192 terms in fp32, its operands kept to 2^-22: rounding errors
add up as their square root, 4 sqrt(192) 2^-22 = 1.3e-5 (F32).  A 16-bit
output adds half a step of its own value, 2^-8.  The gradients of gates and
write strengths are inner products of two such results, x + F32 |x| a / sqrt(n)
and y + F32 |y| b / sqrt(n) with a, b of n unrelated entries of size 1: the
sum's error is F32 |x| |y| / sqrt(n) even where the sum itself cancels, so that
is their scale where it is the larger."""
import numpy as np
import pytest
import torch

from gpu_util import f64, requires_gpu
from oracle import seed_sequence as oseq
from sink_rank_recurrent_amd import binding, sequence

pytestmark = [pytest.mark.gpu, requires_gpu]

F32 = 1.3e-5
RULES = ("gdn", "kda", "mamba2")
NAMES = ("q", "k", "v", "g", "beta", "S0")


def inputs(rule, T, H, HK, d_k, d_v, n, dtype, seed, initial=True, spread=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, device="cuda", generator=gen)

    x = {"q": torch.nn.functional.normalize(normal(T, HK, d_k), dim=-1).to(dtype),
         "k": torch.nn.functional.normalize(normal(T, HK, d_k), dim=-1).to(dtype),
         "v": (normal(1, H, d_v) + 0.3 * normal(T, H, d_v)).to(dtype),
         "g": 1 - spread * torch.rand(T, H, d_k, device="cuda", generator=gen) * 0.1
         if rule == "kda" else 1 - spread * torch.rand(T, H, device="cuda", generator=gen) * 0.1,
         "beta": None if rule == "mamba2" else torch.rand(T, H, device="cuda", generator=gen),
         "S0": 0.3 * normal(n, H, d_k, d_v) if initial else None}
    return x


def host(x):
    return {k: None if v is None else f64(v) for k, v in x.items()}


def run(rule, x, offsets, **kw):
    n = len(offsets) - 1
    H, d_k, d_v = x["v"].shape[1], x["q"].shape[2], x["v"].shape[2]
    o = torch.full_like(x["v"], 7.0)
    S = torch.full((n, H, d_k, d_v), 7.0, device="cuda")
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    sequence.seed_scan(rule, x["q"], x["k"], x["v"], x["g"], x["beta"], o, S, S0=x["S0"],
                       cu_seqlens=cu, **kw)
    return o, S


def run_back(rule, x, offsets, do, dS, **kw):
    n = len(offsets) - 1
    out = {k: torch.full_like(v, 7.0) for k, v in x.items() if v is not None}
    if "S0" not in out:
        out["S0"] = torch.full((n, x["v"].shape[1], x["q"].shape[2], x["v"].shape[2]), 7.0,
                               device="cuda")
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    sequence.seed_scan_backward(rule, x["q"], x["k"], x["v"], x["g"], x["beta"], do, out["q"],
                                out["k"], out["v"], out["g"], out.get("beta"), S0=x["S0"], dS=dS,
                                dS0=out["S0"], cu_seqlens=cu, **kw)
    return out


def check(got, want, offsets, name, f32=F32, terms=None):
    """Every value within f32 of its unit's largest (or of `terms`, the size
    of what it sums), plus half a step of a 16-bit type; nothing written
    outside the sequences."""
    half = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    g = f64(got)
    sizes = []
    if name in ("S", "S0"):
        units = [(g[s, h], want[s, h]) for s in range(g.shape[0]) for h in range(g.shape[1])]
    else:
        inside = np.zeros(g.shape[0], bool)
        units = []
        for s in range(len(offsets) - 1):
            a, b = offsets[s], offsets[s + 1]
            inside[a:b] = True
            if b > a:
                units += [(g[a:b, h], want[a:b, h]) for h in range(g.shape[1])]
                if terms is not None:
                    sizes += [terms[a:b, h].max() for h in range(g.shape[1])]
        assert (g[~inside] == 7.0).all(), f"{name}: rows outside the sequences were written"
    for i, (x, y) in enumerate(units):
        assert np.isfinite(x).all(), (name, i)
        scale = max(np.abs(y).max(), sizes[i] if sizes else 0.0)
        err = np.abs(x - y) - half * (1 + f32) * np.abs(y)
        assert err.max() <= f32 * scale, (name, i, float(err.max() / max(scale, 1e-300)))


DIMS = [(128, 128), (128, 64), (64, 64)]
LENGTHS = [[0, 1], [0, 63], [0, 64], [0, 65], [0, 130, 130, 131, 200]]


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offsets", LENGTHS, ids=str)
def test_forward(rule, dims, dtype, offsets):
    x = inputs(rule, offsets[-1], 2, 2, *dims, len(offsets) - 1, dtype, 1)
    o, S = run(rule, x, offsets)
    wo, wS = oseq.scan(rule, **host(x), offsets=offsets)
    check(o, wo, offsets, "o")
    check(S, wS, offsets, "S")


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offsets", LENGTHS, ids=str)
def test_backward(rule, dims, dtype, offsets):
    n = len(offsets) - 1
    x = inputs(rule, offsets[-1], 2, 2, *dims, n, dtype, 2)
    gen = torch.Generator(device="cuda").manual_seed(9)
    do = torch.randn(x["v"].shape, device="cuda", generator=gen).to(dtype)
    dS = torch.randn(n, 2, *dims, device="cuda", generator=gen)
    got = run_back(rule, x, offsets, do, dS)
    want = oseq.scan_backward(rule, **host(x), offsets=offsets, do=f64(do), dS=f64(dS))
    for name in got:
        check(got[name], want[name], offsets, name, terms=want.get(name + "_scale"))


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("initial", [False, True])
def test_segments(rule, dims, dtype, initial):
    """Few heads and long sequences go in segments side by side: sequences of
    27, 0, 1 and 7 chunks, the segments' ends inside and at a sequence's end,
    rows outside."""
    offsets = [70, 1770, 1770, 1830, 2240]
    T = 2250
    x = inputs(rule, T, 2, 1, *dims, 4, dtype, 12, initial=initial)
    o, S = run(rule, x, offsets)
    h = host(x)
    wo, wS = oseq.scan(rule, **h, offsets=offsets)
    check(o, wo, offsets, "o")
    check(S, wS, offsets, "S")
    gen = torch.Generator(device="cuda").manual_seed(13)
    do = torch.randn(x["v"].shape, device="cuda", generator=gen).to(dtype)
    dS = torch.randn(4, 2, *dims, device="cuda", generator=gen) if initial else None
    got = run_back(rule, x, offsets, do, dS)
    want = oseq.scan_backward(rule, **h, offsets=offsets, do=f64(do), dS=None if dS is None else f64(dS))
    for name in got:
        check(got[name], want[name], offsets, name, terms=want.get(name + "_scale"))


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_shared_keys_outside_rows_and_no_initial_state(rule, dtype):
    """Six heads on two key heads; tokens before the first sequence and
    behind the last hold NaN, which nothing may read."""
    offsets = [3, 80, 80, 150]
    T = 160
    x = inputs(rule, T, 6, 2, 128, 64, 3, dtype, 3, initial=False)
    do = torch.randn(x["v"].shape, device="cuda").to(dtype)
    for t in (x["q"], x["k"], x["v"], x["g"], x["beta"], do):
        if t is not None:
            t[:3] = float("nan")
            t[150:] = float("nan")
    o, S = run(rule, x, offsets)
    h = host(x)
    wo, wS = oseq.scan(rule, **h, offsets=offsets)
    check(o, wo, offsets, "o")
    check(S, wS, offsets, "S")
    got = run_back(rule, x, offsets, do, None)
    want = oseq.scan_backward(rule, **h, offsets=offsets, do=f64(do), dS=None)
    for name in got:
        check(got[name], want[name], offsets, name, terms=want.get(name + "_scale"))


@pytest.mark.parametrize("rule", RULES)
def test_gates_of_zero_and_one(rule):
    """Gates of exactly 0 (a state forgotten) and 1, tiny ones, write
    strengths of 0 and 1: values and gradients, no NaN."""
    offsets = [0, 100]
    x = inputs(rule, 100, 2, 2, 64, 64, 1, torch.float32, 4)
    x["g"][::5] = 1.0
    x["g"][7] = 0.0
    x["g"][40:42, 0] = 0.0
    x["g"][66] = 1e-30
    x["g"][70] = 2.0 ** -140
    x["g"][80:90] *= 0.01
    if rule == "kda":
        x["g"][20, :, ::3] = 0.0
    if x["beta"] is not None:
        x["beta"][::4] = 0.0
        x["beta"][1::4] = 1.0
    do = torch.randn(x["v"].shape, device="cuda")
    dS = torch.randn(1, 2, 64, 64, device="cuda")
    o, S = run(rule, x, offsets)
    wo, wS = oseq.scan(rule, **host(x), offsets=offsets)
    check(o, wo, offsets, "o")
    check(S, wS, offsets, "S")
    got = run_back(rule, x, offsets, do, dS)
    want = oseq.scan_backward(rule, **host(x), offsets=offsets, do=f64(do), dS=f64(dS))
    for name in got:
        check(got[name], want[name], offsets, name, terms=want.get(name + "_scale"))


@pytest.mark.parametrize("rule", RULES)
def test_one_token_is_the_dense_step(rule):
    B, H = 5, 4
    x = inputs(rule, B, H, H, 128, 128, B, torch.bfloat16, 5)
    o, S = run(rule, x, list(range(B + 1)))
    S1 = x["S0"].clone()
    o1 = torch.empty(B, H, 128, device="cuda")
    binding.dense_decode_step(rule, S1, x["q"], x["k"], x["v"], x["g"], x["beta"], o1)
    check(S, f64(S1), [0], "S")
    check(o, f64(o1), list(range(B + 1)), "o")


@pytest.mark.parametrize("rule", RULES)
def test_padded_layout_and_nan_stay_in_their_sequence(rule):
    """[n_seq, length, ...] arrays without offsets; a NaN token spoils its
    own sequence only."""
    n, L, H = 3, 70, 2
    x = inputs(rule, n * L, H, H, 64, 64, n, torch.float32, 6)
    x["v"][L + 5, 0, 0] = float("nan")
    y = {k: None if t is None else t if k == "S0" else t.view(n, L, *t.shape[1:]) for k, t in x.items()}
    o = torch.empty_like(y["v"])
    S = torch.empty(n, H, 64, 64, device="cuda")
    sequence.seed_scan(rule, y["q"], y["k"], y["v"], y["g"], y["beta"], o, S, S0=y["S0"])
    wo, wS = oseq.scan(rule, **host(x), offsets=[0, L, 2 * L, 3 * L])
    for s in (0, 2):
        check(o[s], wo[s * L:(s + 1) * L], [0, L], "o")
        check(S[s:s + 1], wS[s:s + 1], [0], "S")
    assert torch.isnan(S[1, 0]).any() and not torch.isnan(S[1, 1]).any()


@pytest.mark.parametrize("rule", RULES)
def test_same_bits_on_another_stream_and_in_a_graph(rule):
    """Repeated, on another stream, and captured: the same bits; the graph
    is replayed between eager calls of the same inputs."""
    offsets = [0, 90, 200]
    x = inputs(rule, 200, 4, 2, 128, 128, 2, torch.bfloat16, 7)
    do = torch.randn(x["v"].shape, device="cuda").to(torch.bfloat16)
    dS = torch.randn(2, 4, 128, 128, device="cuda")
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")

    def buffers():
        out = {k: torch.zeros_like(v) for k, v in x.items() if v is not None}
        return out, torch.zeros_like(x["v"]), torch.zeros(2, 4, 128, 128, device="cuda")

    def call(b, stream=None):
        out, o, S = b
        sequence.seed_scan(rule, x["q"], x["k"], x["v"], x["g"], x["beta"], o, S, S0=x["S0"],
                           cu_seqlens=cu, stream=stream)
        sequence.seed_scan_backward(rule, x["q"], x["k"], x["v"], x["g"], x["beta"], do, out["q"],
                                    out["k"], out["v"], out["g"], out.get("beta"), S0=x["S0"],
                                    dS=dS, dS0=out["S0"], cu_seqlens=cu, stream=stream)

    def flat(b):
        return list(b[0].values()) + [b[1], b[2]]

    ref = buffers()
    call(ref)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = buffers()
    side.wait_stream(torch.cuda.current_stream())
    call(other, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(flat(ref), flat(other)))
    graphed = buffers()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(graphed)
    for _ in range(3):
        for t in flat(graphed):
            t.zero_()
        eager = buffers()
        call(eager)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(flat(ref), flat(graphed)))
        assert all(torch.equal(a, b) for a, b in zip(flat(ref), flat(eager)))


def test_in_place_states_and_a_workspace_that_is_dirty():
    """S may be S0 and dS0 may be dS; what the workspace holds before a call
    does not matter."""
    offsets = [0, 100, 100, 170]
    x = inputs("gdn", 170, 2, 2, 64, 64, 3, torch.float32, 8)
    o, S = run("gdn", x, offsets)
    ws = sequence.scan_workspace("gdn", x["q"], x["v"], 3)
    ws.fill_(255)
    y = dict(x, S0=x["S0"].clone())
    o2 = torch.full_like(o, 7.0)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    sequence.seed_scan("gdn", y["q"], y["k"], y["v"], y["g"], y["beta"], o2, y["S0"], S0=y["S0"],
                       cu_seqlens=cu, workspace=ws)
    assert torch.equal(o, o2) and torch.equal(S, y["S0"])
    do, dS = torch.randn_like(x["v"]), torch.randn_like(S)
    a = run_back("gdn", x, offsets, do, dS)
    wsb = sequence.scan_workspace("gdn", x["q"], x["v"], 3, backward=True)
    wsb.fill_(255)
    d = dS.clone()
    out = {k: torch.full_like(v, 7.0) for k, v in x.items()}
    sequence.seed_scan_backward("gdn", x["q"], x["k"], x["v"], x["g"], x["beta"], do, out["q"],
                                out["k"], out["v"], out["g"], out["beta"], S0=x["S0"], dS=d, dS0=d,
                                cu_seqlens=cu, workspace=wsb)
    out["S0"] = d
    assert all(torch.equal(a[k], out[k]) for k in a)


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_in_place_states_in_segments(rule, dtype):
    """S is S0 and dS0 is dS where a sequence goes in segments, one of which
    writes them and another of which starts from them."""
    offsets = [0, 1700, 1800]
    x = inputs(rule, 1800, 2, 2, 128, 64, 2, dtype, 14)
    o, S = run(rule, x, offsets)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    o2, S2 = torch.full_like(o, 7.0), x["S0"].clone()
    sequence.seed_scan(rule, x["q"], x["k"], x["v"], x["g"], x["beta"], o2, S2, S0=S2, cu_seqlens=cu)
    assert torch.equal(o, o2) and torch.equal(S, S2)
    do, dS = torch.randn(x["v"].shape, device="cuda").to(dtype), torch.randn_like(S)
    want = run_back(rule, x, offsets, do, dS)
    out = {k: torch.full_like(v, 7.0) for k, v in x.items() if v is not None}
    out["S0"] = dS.clone()
    sequence.seed_scan_backward(rule, x["q"], x["k"], x["v"], x["g"], x["beta"], do, out["q"],
                                out["k"], out["v"], out["g"], out.get("beta"), S0=x["S0"],
                                dS=out["S0"], dS0=out["S0"], cu_seqlens=cu)
    assert all(torch.equal(want[k], out[k]) for k in want)


@pytest.mark.parametrize("rule", RULES)
def test_two_calls_at_once(rule):
    """Calls on two streams at the same time, each with a workspace of its
    own, given or made by the call: the bits of one call alone."""
    offsets = [0, 300, 1000]
    x = inputs(rule, 1000, 4, 2, 128, 128, 2, torch.bfloat16, 15)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    o, S = run(rule, x, offsets)
    do, dS = torch.randn(x["v"].shape, device="cuda").to(torch.bfloat16), torch.randn_like(S)
    want = run_back(rule, x, offsets, do, dS)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    sets = [({k: torch.full_like(v, 7.0) for k, v in x.items() if v is not None},
             torch.full_like(o, 7.0), torch.full_like(S, 7.0)) for _ in streams]
    given = sequence.scan_workspace(rule, x["q"], x["v"], 2, backward=True)
    torch.cuda.synchronize()
    for _ in range(3):
        for i, stream in enumerate(streams):
            ws = given if i else None
            out, oi, Si = sets[i]
            sequence.seed_scan(rule, x["q"], x["k"], x["v"], x["g"], x["beta"], oi, Si, S0=x["S0"],
                               cu_seqlens=cu, workspace=ws, stream=stream)
            sequence.seed_scan_backward(rule, x["q"], x["k"], x["v"], x["g"], x["beta"], do,
                                        out["q"], out["k"], out["v"], out["g"], out.get("beta"),
                                        S0=x["S0"], dS=dS, dS0=out["S0"], cu_seqlens=cu,
                                        workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for out, oi, Si in sets:
        assert torch.equal(o, oi) and torch.equal(S, Si)
        assert all(torch.equal(want[k], out[k]) for k in want)


@pytest.mark.parametrize("backward", [False, True])
def test_no_tokens(backward):
    x = inputs("gdn", 0, 2, 2, 64, 64, 2, torch.float32, 9)
    if not backward:
        o, S = run("gdn", x, [0, 0, 0])
        assert torch.equal(S, x["S0"])
        return
    dS = torch.randn(2, 2, 64, 64, device="cuda")
    got = run_back("gdn", x, [0, 0, 0], x["v"].clone(), dS)
    assert torch.equal(got["S0"], dS)


@pytest.mark.parametrize("rule", RULES)
def test_long_sequence_against_steps(rule):
    """3000 tokens against the single-token kernel, which keeps the state in
    fp32: the errors of a step do not pile up."""
    T, H = 3000, 2
    x = inputs(rule, T, H, H, 128, 128, 1, torch.bfloat16, 10)
    o, S = run(rule, x, [0, T])
    S1 = x["S0"].clone()
    o1 = torch.empty(T, H, 128, device="cuda")
    for t in range(T):
        binding.dense_decode_step(rule, S1, x["q"][t:t + 1], x["k"][t:t + 1], x["v"][t:t + 1],
                                  x["g"][t:t + 1].clone(),
                                  None if x["beta"] is None else x["beta"][t:t + 1].clone(),
                                  o1[t:t + 1])
    check(S, f64(S1), [0], "S", 4 * F32)
    check(o, f64(o1), [0, T], "o", 4 * F32)
