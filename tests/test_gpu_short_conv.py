"""The short convolution, its backward pass and its step against the float64
oracle, value by value within the oracle's bounds: every rounding followed
through the formulas (oracle/seed_channels.py), a 16-bit result half a step
more.  Below the smallest normal fp32 number a value may be flushed to 0."""
import numpy as np
import pytest
import torch

from gpu_util import f64, requires_gpu
from oracle import seed_channels as och
from sink_rank_recurrent_amd import channels

pytestmark = [pytest.mark.gpu, requires_gpu]

TINY = 2.0 ** -126
MARK = 77.0        # what rows outside the sequences hold


def half(dtype):
    return torch.finfo(dtype).eps / 2


def make(T, C, K, n, dtype, seed, row=None, initial=True, at=0):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, device="cuda", generator=gen)

    x = normal(T, row or C).to(dtype)[:, at:at + C]
    return {"x": x, "w": normal(C, K) / K ** 0.5, "b": 0.3 * normal(C),
            "S0": normal(n, K - 1, C).to(dtype) if initial else None,
            "dy": normal(T, C).to(dtype), "dS": normal(n, K - 1, C).to(dtype)}


def check(got, want, off, name):
    """NaN in `want`: rows outside the sequences, left as they were."""
    got = f64(got)
    out = np.isnan(want)
    assert (got[out] == MARK).all(), name
    err = np.abs(got - want) - off - TINY
    assert not (err > 0).any() and not np.isnan(got[~out]).any(), (name, np.nanmax(err), off.max())


def depth(offsets, T):
    """Additions in a row of the weights' sums: runs of at most 32 tokens,
    every 128th at most, then a block's runs (256 at most), a quarter of the
    128 blocks and the four waves."""
    runs = T // 8 + len(offsets) - 1
    return 32 * -(-runs // 128) + min(runs, 256) + -(-min(runs, 128) // 4) + 4


def run_all(p, offsets, silu, bias, T, C, K, dtype, cu=None, lead=None):
    """Forward and backward through the kernels and against the oracle; both
    results."""
    act, n = "silu" if silu else None, len(offsets) - 1
    b = p["b"] if bias else None
    S0 = p["S0"]

    def shaped(t):
        return t if lead is None else t.reshape(*lead, C)

    y = torch.full((T, C), MARK, device="cuda", dtype=dtype)
    S = torch.full((n, K - 1, C), MARK, device="cuda", dtype=dtype)
    channels.seed_short_conv(shaped(p["x"]), p["w"], shaped(y), bias=b, activation=act, S0=S0, S=S, cu_seqlens=cu)
    dx = torch.full((T, C), MARK, device="cuda", dtype=dtype)
    dw, db = torch.full((C, K), MARK, device="cuda"), torch.full((C,), MARK, device="cuda")
    dS0 = torch.full((n, K - 1, C), MARK, device="cuda", dtype=dtype) if S0 is not None else None
    channels.seed_short_conv_backward(shaped(p["dy"]), shaped(p["x"]), p["w"], shaped(dx), dweight=dw, dbias=db,
                                      bias=b, activation=act, S0=S0, dS=p["dS"], dS0=dS0, cu_seqlens=cu)
    h = {k: None if v is None else f64(v) for k, v in p.items()}
    hb = h["b"] if bias else None
    io = 0.0 if dtype == torch.float32 else half(dtype)
    wy, y_off, wS = och.conv(h["x"], h["w"], hb, h["S0"], silu, offsets, io)
    check(y, wy, y_off, "y")
    assert np.array_equal(f64(S), wS)          # the inputs themselves
    want = och.conv_backward(h["x"], h["w"], hb, h["S0"], silu, offsets, h["dy"], h["dS"], depth(offsets, T), io)
    for name, got in (("x", dx), ("weight", dw), ("bias", db), ("S0", dS0)):
        if got is not None:
            check(got, *want[name], name)
    return y, S, dx, dw, db, dS0


CASES = [
    # offsets, channels, taps: lengths of 0 and 1, shorter than the taps, at and around a run of 32
    ([0, 1], 1, 4), ([0, 0], 8, 3), ([0, 0, 1, 3, 3], 64, 4), ([0, 2, 5, 5, 37], 72, 2),
    ([0, 31, 63, 96, 129], 40, 3), ([0, 32, 64], 256, 4), ([0, 33], 2048, 4), ([0, 100, 101, 300], 101, 4),
    ([0, 5, 64, 64, 200], 520, 3), ([0, 7], 4104, 2),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offsets,C,K", CASES)
def test_packed(offsets, C, K, dtype):
    T = offsets[-1]
    if T == 0:
        T = 3                                  # rows that belong to no sequence
    p = make(T, C, K, len(offsets) - 1, dtype, 1 + C)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    run_all(p, offsets, C % 3 != 0, C % 2 == 0, T, C, K, dtype, cu)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_equal_lengths(K, bias, silu):
    n, length, C = 3, 50, 136
    p = make(n * length, C, K, n, torch.bfloat16, 2, initial=False)
    run_all(p, [0, 50, 100, 150], silu, bias, n * length, C, K, torch.bfloat16, lead=(n, length))


@pytest.mark.parametrize("row,at", [(264, 0), (264, 8), (264, 64), (263, 5), (301, 100)])
def test_slices_of_wider_rows(row, at):
    """Rows of a projection: aligned ones take the wide loads, others do not;
    the same bits."""
    C, K, offsets = 200, 4, [0, 20, 45]
    T = 50                                     # five rows behind the last sequence
    p = make(T, C, K, 2, torch.bfloat16, 3, row=row, at=at)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    got = run_all(p, offsets, True, True, T, C, K, torch.bfloat16, cu)
    dense = run_all({**p, "x": p["x"].contiguous()}, offsets, True, True, T, C, K, torch.bfloat16, cu)
    assert all(torch.equal(a, b) for a, b in zip(got, dense))
    # outputs into slices of one buffer, beside what must stay
    wide = torch.full((T, 2 * C + 9), MARK, device="cuda", dtype=torch.bfloat16)
    channels.seed_short_conv(p["x"], p["w"], wide[:, 4:4 + C], bias=p["b"], S0=p["S0"], cu_seqlens=cu)
    assert torch.equal(wide[:, 4:4 + C], got[0])
    assert (wide[:, :4] == MARK).all() and (wide[:, 4 + C:] == MARK).all()


@pytest.mark.parametrize("n_seq", [65, 1000, 5000])
def test_many_sequences(n_seq):
    """More sequences than a wave looks at in one step, empty ones among them."""
    gen = np.random.default_rng(n_seq)
    lens = gen.integers(0, 4, n_seq)
    lens[gen.integers(0, n_seq, 3)] = 70
    offsets = [0, *np.cumsum(lens).tolist()]
    T, C, K = offsets[-1], 16, 4
    p = make(T, C, K, n_seq, torch.float32, 4)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    run_all(p, offsets, True, True, T, C, K, torch.float32, cu)


def test_state_in_place_and_parts():
    """A prompt in two parts, the state in place, is the prompt at once."""
    offsets, cut = [0, 40, 41, 90], [0, 17, 17, 30]
    C, K, n = 64, 4, 3
    p = make(90, C, K, n, torch.bfloat16, 5)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    y = torch.empty(90, C, device="cuda", dtype=torch.bfloat16)
    S = torch.empty_like(p["S0"])
    channels.seed_short_conv(p["x"], p["w"], y, S0=p["S0"], S=S, cu_seqlens=cu)
    held = p["S0"].clone()
    lens = [b - a for a, b in zip(offsets, offsets[1:])]
    first = [b - a for a, b in zip(cut, cut[1:])]
    parts = [(offsets[i], offsets[i] + first[i]) for i in range(n)], [(offsets[i] + first[i], offsets[i + 1]) for i in range(n)]
    for part in parts:
        rows = torch.cat([torch.arange(a, b) for a, b in part]).cuda()
        off = torch.tensor([0, *np.cumsum([b - a for a, b in part])], dtype=torch.int32, device="cuda")
        out = torch.empty(len(rows), C, device="cuda", dtype=torch.bfloat16)
        channels.seed_short_conv(p["x"][rows].contiguous(), p["w"], out, S0=held, S=held, cu_seqlens=off)
        assert torch.equal(out, y[rows])
    assert torch.equal(held, S) and sum(lens) == 90


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,C,K,row", [(1, 1, 2, 1), (3, 7, 4, 9), (64, 2048, 4, 6144), (5, 72, 3, 72), (1000, 8, 4, 24)])
def test_step_is_a_sequence_of_one(batch, C, K, row, dtype):
    p = make(batch, C, K, batch, dtype, 6, row=row, at=row - C if row % 8 else 0)
    cu = torch.arange(batch + 1, dtype=torch.int32, device="cuda")
    y, S = torch.empty(batch, C, device="cuda", dtype=dtype), torch.empty_like(p["S0"])
    channels.seed_short_conv(p["x"], p["w"], y, bias=p["b"], S0=p["S0"], S=S, cu_seqlens=cu)
    y1, S1 = torch.empty_like(y), torch.empty_like(S)
    channels.seed_short_conv_step(p["x"], p["w"], y1, S1, bias=p["b"], S0=p["S0"])
    assert torch.equal(y, y1) and torch.equal(S, S1)
    held, out = p["S0"].clone(), p["x"].clone()
    channels.seed_short_conv_step(out, p["w"], out, held, bias=p["b"])     # both in place
    assert torch.equal(y, out) and torch.equal(S, held)
    h = {k: f64(v) for k, v in p.items()}
    want, off, _ = och.conv(h["x"], h["w"], h["b"], h["S0"], True, list(range(batch + 1)),
                            0.0 if dtype == torch.float32 else half(dtype))
    check(y, want, off, "y")


def test_nan_and_infinity_reach_their_taps_only():
    C, K, T = 8, 4, 40
    p = make(T, C, K, 2, torch.float32, 7)
    cu = torch.tensor([0, 20, 40], dtype=torch.int32, device="cuda")
    clean = torch.empty(T, C, device="cuda")
    channels.seed_short_conv(p["x"], p["w"], clean, cu_seqlens=cu)
    p["x"][5, 2], p["x"][18, 3] = float("nan"), float("inf")
    y = torch.empty(T, C, device="cuda")
    channels.seed_short_conv(p["x"], p["w"], y, cu_seqlens=cu)
    touched = torch.zeros(T, C, dtype=torch.bool, device="cuda")
    touched[5:9, 2] = True
    touched[18:20, 3] = True                    # the next sequence starts at 20
    assert torch.isnan(y[5:9, 2]).all() and not torch.isfinite(y[18:20, 3]).any()
    assert torch.equal(y[~touched], clean[~touched])


def test_gradients_are_differences():
    """Along a random direction, the float32 gradients against central
    differences of the oracle: h^2 of the third derivative and the gradients'
    own bounds."""
    offsets, C, K, T = [0, 3, 40, 75], 24, 4, 75
    p = make(T, C, K, 3, torch.float32, 8)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    got = dict(zip(("y", "S", "x", "w", "b", "S0"), run_all(p, offsets, True, True, T, C, K, torch.float32, cu)))
    h = {k: f64(v) for k, v in p.items()}
    rng = np.random.default_rng(9)
    names = ("x", "w", "b", "S0")
    along = {k: rng.standard_normal(h[k].shape) for k in names}
    along = {k: v / np.linalg.norm(v) for k, v in along.items()}

    def loss(e):
        q = {k: h[k] + e * along[k] for k in names}
        y, _, S = och.conv(q["x"], q["w"], q["b"], q["S0"], True, offsets)
        return (y * h["dy"]).sum() + (S * h["dS"]).sum()

    want = (loss(1e-4) - loss(-1e-4)) / 2e-4
    value = sum((f64(got[k]) * along[k]).sum() for k in names)
    bounds = och.conv_backward(h["x"], h["w"], h["b"], h["S0"], True, offsets, h["dy"], h["dS"], depth(offsets, T))
    off = sum((np.abs(along[k]) * bounds[n][1]).sum() for k, n in zip(names, ("x", "weight", "bias", "S0")))
    assert abs(value - want) <= off + 1e-7 * sum(np.linalg.norm(f64(got[k])) for k in names), (value, want, off)


def test_graph_stream_and_workspace():
    """On another stream with a shared workspace, and captured and replayed
    with eager calls between: the same bits."""
    offsets, C, K, T = [0, 100, 164, 164, 400], 264, 4, 400
    p = make(T, C, K, 4, torch.bfloat16, 10)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ws = channels.short_conv_workspace(p["x"], p["w"], 4)

    def both(out, stream=None):
        y, S, dx, dw, db, dS0 = out
        channels.seed_short_conv(p["x"], p["w"], y, bias=p["b"], S0=p["S0"], S=S, cu_seqlens=cu, stream=stream)
        channels.seed_short_conv_backward(p["dy"], p["x"], p["w"], dx, dweight=dw, dbias=db, bias=p["b"], S0=p["S0"],
                                          dS=p["dS"], dS0=dS0, cu_seqlens=cu, workspace=ws, stream=stream)
        channels.seed_short_conv_step(p["x"][:4], p["w"], y[:4], S, bias=p["b"], S0=p["S0"], stream=stream)

    def buffers():
        e = {"device": "cuda", "dtype": torch.bfloat16}
        return [torch.zeros(T, C, **e), torch.zeros(4, K - 1, C, **e), torch.zeros(T, C, **e),
                torch.zeros(C, K, device="cuda"), torch.zeros(C, device="cuda"), torch.zeros(4, K - 1, C, **e)]

    ref = buffers()
    both(ref)
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), buffers()
    side.wait_stream(torch.cuda.current_stream())
    both(other, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, other))
    cap = buffers()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both(cap)
    for _ in range(3):
        for t in cap:
            t.zero_()
        eager = buffers()
        both(eager)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, cap))
        assert all(torch.equal(a, b) for a, b in zip(ref, eager))


def test_refusals_on_device():
    p = make(10, 16, 4, 2, torch.bfloat16, 11)
    y = torch.full((10, 16), MARK, device="cuda", dtype=torch.bfloat16)
    cu = torch.tensor([0, 4, 10], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="y has dtype"):
        channels.seed_short_conv(p["x"], p["w"], y.float(), cu_seqlens=cu)
    with pytest.raises(ValueError, match="S0 has shape"):
        channels.seed_short_conv(p["x"], p["w"], y, S0=p["S0"][:1], cu_seqlens=cu)
    with pytest.raises(ValueError, match="activation"):
        channels.seed_short_conv(p["x"], p["w"], y, activation="sigmoid", cu_seqlens=cu)
    with pytest.raises(ValueError, match="dimensions"):
        channels.seed_short_conv(p["x"], p["w"], y)
    with pytest.raises(ValueError, match="cu_seqlens has dtype"):
        channels.seed_short_conv(p["x"], p["w"], y, cu_seqlens=cu.long())
    assert (y == MARK).all()
