"""The selective scan, its backward pass and its step against the float64
oracle, value by value within the oracle's bounds: every rounding followed
through the formulas and the recurrence (oracle/seed_channels.py), a 16-bit
result half a step more.  Below the smallest normal fp32 number a value may be
flushed to 0."""
import numpy as np
import pytest
import torch

from gpu_util import f64, requires_gpu
from oracle import seed_channels as och
from sink_rank_recurrent_amd import channels
from test_gpu_short_conv import MARK, TINY, check, half

pytestmark = [pytest.mark.gpu, requires_gpu]

NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")
FULL = {"D", "z", "dt_bias", "S0", "softplus"}


def make(T, W, G, N, n, dtype, seed, have=FULL, row=None):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, device="cuda", generator=gen)

    xz = normal(T, row or 2 * W).to(dtype)
    bc = normal(T, 2, G, N).to(dtype)
    dt = normal(T, W) - 1
    p = {"x": xz[:, :W], "z": xz[:, W:2 * W] if row is None or row >= 2 * W else normal(T, W).to(dtype),
         "dt": (dt if "softplus" in have else 0.3 * torch.exp(dt)).to(dtype),
         "A": -torch.exp(0.7 * normal(W, N)), "B": bc[:, 0], "C": bc[:, 1], "D": normal(W),
         "dt_bias": 0.5 * normal(W) if "softplus" in have else 0.1 * torch.rand(W, device="cuda", generator=gen),
         "S0": normal(n, W, N), "dy": normal(T, W).to(dtype), "dS": normal(n, W, N)}
    for k in ("D", "z", "dt_bias", "S0"):
        if k not in have:
            p[k] = None
    return p


def outputs(p, n, back=True):
    """Marked buffers for every output of a call."""
    out = {"y": torch.full_like(p["x"], MARK, memory_format=torch.contiguous_format),
           "S": torch.full((n, *p["A"].shape), MARK, device="cuda")}
    if back:
        for k in (*NAMES, "S0"):
            if p[k] is not None:
                out["d" + k] = torch.full_like(p[k], MARK, memory_format=torch.contiguous_format)
    return out


def forward(p, out, softplus, cu=None, **more):
    channels.seed_selective_scan(*(p[k] for k in NAMES[:5]), out["y"], out["S"], D=p["D"], z=p["z"],
                                 dt_bias=p["dt_bias"], softplus=softplus, S0=p["S0"], cu_seqlens=cu, **more)


def backward(p, out, softplus, cu=None, **more):
    channels.seed_selective_scan_backward(p["dy"], *(p[k] for k in NAMES[:5]), *(out["d" + k] for k in NAMES[:5]),
                                          D=p["D"], z=p["z"], dt_bias=p["dt_bias"], dD=out.get("dD"),
                                          dz=out.get("dz"), ddt_bias=out.get("ddt_bias"), softplus=softplus,
                                          S0=p["S0"], dS=p["dS"], dS0=out.get("dS0"), cu_seqlens=cu, **more)


def depth(offsets, W, G, T):
    """Additions in a row of the sums over tokens (a segment of at most 128
    after the other, then the parts) and over channels (six folds of a wave's
    lanes, the blocks)."""
    segments = T // 128 + len(offsets) - 1
    return 128 * segments + 8, 6 + W // G // 64 + 8


def run_all(p, offsets, softplus, cu=None, lead=None):
    """Forward and backward through the kernels and against the oracle."""
    n, T, W = len(offsets) - 1, *p["x"].shape
    G, dtype = p["B"].shape[1], p["x"].dtype
    out = outputs(p, n)
    rows = ("x", "dt", "B", "C", "z", "dy")
    q, o = p, out
    if lead is not None:
        q = {k: v.reshape(*lead, *v.shape[1:]) if k in rows and v is not None else v for k, v in p.items()}
        o = {k: v.view(*lead, *v.shape[1:]) if k == "y" or k[1:] in rows else v for k, v in out.items()}
    forward(q, o, softplus, cu)
    backward(q, o, softplus, cu)
    h = {k: None if v is None else f64(v) for k, v in p.items()}
    io = 0.0 if dtype == torch.float32 else half(dtype)
    y, S = och.select(*(h[k] for k in NAMES), softplus, h["S0"], offsets, io)
    check(out["y"], *y, "y")
    check(out["S"], *S, "S")
    want = och.select_backward(*(h[k] for k in NAMES), softplus, h["S0"], offsets, h["dy"], h["dS"],
                               max(depth(offsets, W, G, T)), io)
    for k in (*NAMES, "S0"):
        if p[k] is not None:
            check(out["d" + k], *want[k], "d" + k)
    return out


CASES = [
    # offsets, channels, groups, d_state: lengths of 0 and 1, around the tiles of 8 and the segments of 64
    # (forward, from 129 tokens a sequence on) and 128 (backward)
    ([0, 1], 1, 1, 1), ([0, 0, 2], 3, 3, 16), ([0, 7, 8, 17], 64, 1, 16), ([0, 63, 127, 192], 70, 2, 5),
    ([0, 64, 129], 130, 1, 16), ([0, 300], 24, 4, 16),
    ([0, 192], 40, 1, 8), ([0, 1, 257, 400], 70, 1, 16), ([0, 385], 3, 1, 40), ([0, 512, 513], 33, 3, 4), ([0, 128, 128, 257], 260, 1, 8), ([0, 65, 70], 66, 1, 32),
    ([0, 40], 40, 2, 64), ([0, 3, 90], 129, 1, 33), ([0, 9], 513, 1, 16), ([0, 130], 10, 2, 17),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offsets,W,G,N", CASES)
def test_packed(offsets, W, G, N, dtype):
    p = make(offsets[-1] + W % 3, W, G, N, len(offsets) - 1, dtype, W + N)
    run_all(p, offsets, True, torch.tensor(offsets, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("have", [set(), {"D"}, {"z"}, {"dt_bias"}, {"S0"}, {"softplus"}, {"D", "z", "softplus"}])
def test_parts_of_the_formula(have):
    p = make(3 * 70, 72, 1, 16, 3, torch.bfloat16, 3, have)
    run_all(p, [0, 70, 140, 210], "softplus" in have, lead=(3, 70))


def test_enough_sequences_to_run_whole():
    """50 sequences of eleven blocks of channels go from end to end, the
    longest first."""
    n, W = 50, 700
    lens = [(70 * i) % 130 for i in range(n)]
    offsets = [0, *np.cumsum(lens).tolist()]
    p = make(offsets[-1], W, 1, 16, n, torch.float32, 4)
    run_all(p, offsets, True, torch.tensor(offsets, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("n_seq", [65, 4200])
def test_many_sequences(n_seq):
    rng = np.random.default_rng(n_seq)
    lens = rng.integers(0, 3, n_seq)
    lens[rng.integers(0, n_seq, 2)] = 140      # (whole: 129 tokens a sequence would go in segments)
    offsets = [0, *np.cumsum(lens).tolist()]
    p = make(offsets[-1], 5, 1, 3, n_seq, torch.bfloat16, 5)
    run_all(p, offsets, True, torch.tensor(offsets, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("n_seq,W,G,N", [(2100, 330, 1, 6), (4200, 150, 1, 16), (2100, 300, 2, 20), (4200, 130, 1, 50)])
def test_blocks_of_channels_one_after_the_other(n_seq, W, G, N):
    """Segments enough for a workgroup to take several blocks of 64 channels in
    turn, the last one fewer, and to go on to further segments (backward)."""
    rng = np.random.default_rng(N)
    lens = rng.integers(0, 2, n_seq)
    lens[:2], lens[rng.integers(2, n_seq, 3)] = (9, 140), 17
    offsets = [0, *np.cumsum(lens).tolist()]
    dtype = torch.float32 if N == 20 else torch.bfloat16
    p = make(offsets[-1], W, G, N, n_seq, dtype, N, {"D", "z", "dt_bias", "softplus"} if N != 16 else {"softplus"})
    run_all(p, offsets, True, torch.tensor(offsets, dtype=torch.int32, device="cuda"))


def test_extreme_steps_and_rates():
    """Steps and rates whose decays vanish or stay at one, softplus far out on
    both sides, and rows of zeros."""
    p = make(150, 64, 1, 16, 1, torch.float32, 6)
    p["dt"][:, :8], p["dt"][:, 8:16] = 30.0, -60.0
    p["A"][:, 0], p["A"][:, 1], p["A"][:, 2] = 0.0, -1e4, -1e-6
    p["x"][:, 16:24], p["z"][:, 24:32] = 0.0, 0.0
    p["z"][:, 32:40], p["z"][:, 40:48] = 60.0, -60.0
    run_all(p, [0, 150], True, torch.tensor([0, 150], dtype=torch.int32, device="cuda"))


def test_nan_and_infinity_stay_in_their_channel():
    W, T = 70, 400
    offsets = [0, 90, 400]
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    p = make(T, W, 1, 5, 2, torch.float32, 7)
    clean = outputs(p, 2, back=False)
    forward(p, clean, True, cu)
    p["x"][40, 3], p["dt"][100, 64], p["z"][10, 8] = float("nan"), float("inf"), float("nan")
    out = outputs(p, 2, back=False)
    forward(p, out, True, cu)
    touched = torch.zeros(T, W, dtype=torch.bool, device="cuda")
    touched[40:90, 3], touched[100:400, 64], touched[10, 8] = True, True, True
    assert not torch.isfinite(out["y"][touched]).any()
    assert torch.equal(out["y"][~touched], clean["y"][~touched])
    ok = torch.ones(2, W, dtype=torch.bool, device="cuda")
    ok[0, 3] = ok[1, 64] = False
    assert torch.equal(out["S"][ok], clean["S"][ok]) and not torch.isfinite(out["S"][~ok]).any()


def test_prompt_in_parts_and_in_place():
    """A prompt in two parts, its state in place, within the sum of the bounds
    of the whole."""
    p = make(300, 33, 1, 16, 1, torch.float32, 8)   # in segments; its parts, 140 and 160 tokens, too
    whole = outputs(p, 1, back=False)
    cu = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    forward(p, whole, True, cu)
    held = p["S0"].clone()
    for a, b in ((0, 140), (140, 300)):
        q = {k: v[a:b] if k in ("x", "dt", "B", "C", "z") else v for k, v in p.items()}
        q["S0"] = held
        forward(q, {"y": whole["y"][a:b], "S": held}, True, torch.tensor([0, b - a], dtype=torch.int32, device="cuda"))
    h = {k: f64(v) for k, v in p.items()}
    y, S = och.select(*(h[k] for k in NAMES), True, h["S0"], [0, 300])
    check(whole["y"], *y, "y")
    check(held, *S, "S")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch,W,G,N", [(1, 1, 1, 1), (3, 7, 7, 4), (5, 66, 2, 16), (17, 130, 1, 7), (64, 512, 1, 16),
                                         (9, 100, 4, 32), (4, 30, 1, 64)])
def test_step(batch, W, G, N, dtype):
    """Against the oracle; in place the same bits."""
    have = FULL if N % 2 == 0 else {"softplus"}
    p = make(batch, W, G, N, batch, dtype, 9 + N, have | {"S0"})
    out = outputs(p, batch, back=False)
    args = dict(D=p["D"], z=p["z"], dt_bias=p["dt_bias"], softplus=True)
    channels.seed_selective_step(*(p[k] for k in NAMES[:5]), out["y"], out["S"], S0=p["S0"], **args)
    h = {k: None if v is None else f64(v) for k, v in p.items()}
    y, S = och.select(*(h[k] for k in NAMES), True, h["S0"], list(range(batch + 1)),
                      0.0 if dtype == torch.float32 else half(dtype))
    check(out["y"], *y, "y")
    check(out["S"], *S, "S")
    held, x = p["S0"].clone(), p["x"].clone()
    channels.seed_selective_step(x, *(p[k] for k in NAMES[1:5]), x, held, **args)
    assert torch.equal(x, out["y"]) and torch.equal(held, out["S"])


def test_gradients_are_differences():
    """Along a random direction, the float32 gradients against central
    differences of the oracle: h^2 of the third derivative and the gradients'
    own bounds."""
    offsets = [0, 3, 80, 80, 150]
    p = make(150, 20, 2, 6, 4, torch.float32, 10)
    got = run_all(p, offsets, True, torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    h = {k: f64(v) for k, v in p.items()}
    rng = np.random.default_rng(11)
    names = (*NAMES, "S0")
    along = {k: rng.standard_normal(h[k].shape) for k in names}
    along = {k: v / np.linalg.norm(v) for k, v in along.items()}

    def loss(e):
        q = {k: h[k] + e * along[k] for k in names}
        (y, _), (S, _) = och.select(*(q[k] for k in NAMES), True, q["S0"], offsets)
        return (y * h["dy"]).sum() + (S * h["dS"]).sum()

    want = (loss(1e-4) - loss(-1e-4)) / 2e-4
    value = sum((f64(got["d" + k]) * along[k]).sum() for k in names)
    bounds = och.select_backward(*(h[k] for k in NAMES), True, h["S0"], offsets, h["dy"], h["dS"], 400)
    off = sum((np.abs(along[k]) * bounds[k][1]).sum() for k in names)
    assert abs(value - want) <= off + 1e-7 * sum(np.linalg.norm(f64(got["d" + k])) for k in names), (value, want, off)


def test_gradients_that_are_not_asked_for():
    """dD and ddt_bias where D and dt_bias are NULL, and none of them; no
    gradient of the last states."""
    p = make(100, 64, 1, 16, 1, torch.bfloat16, 12, {"softplus"})
    p["dS"] = None
    cu = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    a, b = outputs(p, 1), outputs(p, 1)
    b.update(dD=torch.empty(64, device="cuda"), ddt_bias=torch.empty(64, device="cuda"))
    backward(p, a, True, cu)
    backward(p, b, True, cu)
    assert all(torch.equal(a[k], b[k]) for k in a)
    h = {k: None if v is None else f64(v) for k, v in p.items()}
    want = och.select_backward(*(h[k] for k in NAMES), True, None, [0, 100], h["dy"], None, 400)
    check(b["dD"], *want["D"], "dD")
    check(b["ddt_bias"], *want["dt_bias"], "ddt_bias")


def test_no_tokens():
    """Empty sequences pass states and gradients on; the weights' are zero."""
    p = make(0, 10, 1, 3, 2, torch.float32, 13)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = outputs(p, 2)
    forward(p, out, True, cu)
    backward(p, out, True, cu)
    assert torch.equal(out["S"], p["S0"]) and torch.equal(out["dS0"], p["dS"])
    assert all((out[k] == 0).all() for k in ("dA", "dD", "ddt_bias"))


@pytest.mark.parametrize("W,N", [(72, 16), (600, 40)])
def test_graph_stream_and_workspace(W, N):
    """On another stream with shared workspaces, and captured and replayed
    with eager calls between: the same bits."""
    offsets = [0, 100, 164, 164, 1200]
    p = make(1200, W, 1, N, 4, torch.bfloat16, 14)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    ws = [channels.selective_scan_workspace(p["x"], p["B"], 4, backward=b) for b in (False, True)]

    def both(out, stream=None):
        forward(p, out, True, cu, workspace=ws[0], stream=stream)
        backward(p, out, True, cu, workspace=ws[1], stream=stream)

    ref = outputs(p, 4)
    both(ref)
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), outputs(p, 4)
    side.wait_stream(torch.cuda.current_stream())
    both(other, side)
    torch.cuda.synchronize()
    assert all(torch.equal(ref[k], other[k]) for k in ref)
    alloc = outputs(p, 4)                       # workspaces made by the calls, on the side stream
    side.wait_stream(torch.cuda.current_stream())
    forward(p, alloc, True, cu, stream=side)
    backward(p, alloc, True, cu, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(ref[k], alloc[k]) for k in ref)
    cap = outputs(p, 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both(cap)
    for _ in range(3):
        for t in cap.values():
            t.fill_(MARK)
        eager = outputs(p, 4)
        both(eager)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(ref[k], cap[k]) for k in ref)
        assert all(torch.equal(ref[k], eager[k]) for k in ref)


def test_gradients_into_slices_of_one_buffer():
    """dx and dz, dB and dC side by side in the rows of a projection's
    gradient, dS0 in dS's place: the bits of dense outputs."""
    offsets = [0, 90, 200]
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    p = make(200, 96, 2, 16, 2, torch.bfloat16, 15)
    ref = outputs(p, 2)
    backward(p, ref, True, cu)
    fused = torch.full((200, 96 * 2 + 64 + 8), MARK, device="cuda", dtype=torch.bfloat16)
    out = outputs(p, 2)
    out["dx"], out["dz"] = fused[:, :96], fused[:, 96:192]
    out["dB"], out["dC"] = fused[:, 192:224].view(200, 2, 16), fused[:, 224:256].view(200, 2, 16)
    q = {**p, "dS": p["dS"].clone()}
    out["dS0"] = q["dS"]
    backward(q, out, True, cu)
    assert all(torch.equal(ref[k], out[k]) for k in ref if k not in ("y", "S"))
    assert (fused[:, 256:] == MARK).all()


def test_refusals_on_device():
    p = make(10, 16, 2, 4, 2, torch.bfloat16, 16)
    cu = torch.tensor([0, 4, 10], dtype=torch.int32, device="cuda")
    out = outputs(p, 2)
    with pytest.raises(ValueError, match="C has shape"):
        forward({**p, "C": p["C"][:, :1]}, out, True, cu)
    with pytest.raises(ValueError, match="dt has dtype"):
        forward({**p, "dt": p["dt"].float()}, out, True, cu)
    with pytest.raises(ValueError, match="S0 has shape"):
        forward({**p, "S0": p["S0"][:1]}, out, True, cu)
    with pytest.raises(ValueError, match="workspace"):
        forward(p, out, True, cu, workspace=torch.empty(4, device="cuda"))
    with pytest.raises(RuntimeError, match="needed"):
        forward(p, out, True, cu, workspace=torch.empty(4, device="cuda", dtype=torch.uint8))
    with pytest.raises(RuntimeError, match="exactly if"):
        backward({**p, "z": None}, out, True, cu)
    assert all((t == MARK).all() for t in out.values())
