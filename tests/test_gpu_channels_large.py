"""Operators on channels where offsets pass 32 bits: rows that lie far apart,
states and workspaces of more than 2^31 values."""
import pytest
import torch

from gpu_util import requires_gpu
from sink_rank_recurrent_amd import channels
from test_gpu_selective_scan import FULL, NAMES, backward, forward, make, outputs

pytestmark = [pytest.mark.gpu, requires_gpu]


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def test_rows_far_apart():
    """Every array over tokens a slice of one buffer whose rows lie 2^22 values
    apart, the last ones behind 2^32: the bits of dense arrays."""
    T, W = 1040, 72
    offsets = torch.tensor([0, 500, T], dtype=torch.int32, device="cuda")
    p = make(T, W, 1, 16, 2, torch.bfloat16, 1)
    p = {k: v.contiguous() for k, v in p.items()}
    wide = torch.empty(T, 1 << 22, device="cuda", dtype=torch.bfloat16)
    at = 0

    def far(t):
        nonlocal at
        cols = t[0].numel()
        view = wide[:, at:at + cols].view(t.shape) if t.dim() == 2 else wide[:, at:at + cols].unflatten(1, t.shape[1:])
        at += (cols + 7) // 8 * 8
        view.copy_(t)
        return view

    rows = ("x", "dt", "B", "C", "z", "dy")
    q = {k: far(v) if k in rows else v for k, v in p.items()}
    ref, out = outputs(p, 2), outputs(p, 2)
    out = {k: far(v) if k == "y" or k[1:] in rows else v for k, v in out.items()}
    for a, o in ((p, ref), (q, out)):
        forward(a, o, True, offsets)
        backward(a, o, True, offsets)
    assert all(torch.equal(ref[k], out[k]) for k in ref)
    w = torch.randn(W, 4, device="cuda")
    e = [torch.empty_like(p["x"]) for _ in range(2)] + [torch.empty_like(w)]
    f = [far(e[0]), far(e[1]), torch.empty_like(w)]
    for a, (y, dx, dw) in ((p, e), (q, f)):
        channels.seed_short_conv(a["x"], w, y, cu_seqlens=offsets)
        channels.seed_short_conv_backward(a["dy"], a["x"], w, dx, dweight=dw, cu_seqlens=offsets)
    assert all(torch.equal(a, b) for a, b in zip(e, f))


def test_workspace_beyond_32_bits():
    """136 equal sequences of 1024 tokens: the backward pass keeps 2.3e9
    values.  Every sequence has the first one's bits."""
    n, L, W = 136, 1024, 8192
    p = make(L, W, 1, 16, 1, torch.bfloat16, 2, FULL - {"S0"})
    p = {k: v if v is None or k in ("A", "D", "dt_bias", "dS") else v.repeat(n, *[1] * (v.dim() - 1)) for k, v in p.items()}
    p["dS"] = None
    cu = torch.arange(0, n * L + 1, L, dtype=torch.int32, device="cuda")
    assert channels.selective_scan_workspace(p["x"], p["B"], n, backward=True).numel() > 4 * 2 ** 31
    out = outputs(p, n)
    forward(p, out, True, cu)
    backward(p, out, True, cu)
    for k in ("y", "dx", "ddt", "dB", "dC", "dz"):
        t = out[k].view(n, L, -1)
        assert not torch.isnan(t[0]).any() and t[0].any()
        assert all(torch.equal(t[0], t[i]) for i in (1, n // 2, n - 1)), k
    assert all(torch.equal(out["S"][0], out["S"][i]) for i in (1, n - 1))


def test_states_beyond_32_bits():
    """A step of 1100 requests of 2^17 channels: 2.3e9 states, in place; every
    request has the first one's bits."""
    B, W, N = 1100, 1 << 17, 16
    p = make(1, W, 1, N, 1, torch.bfloat16, 3)
    rows = {k: p[k].expand(B, *p[k].shape[1:]).contiguous() for k in ("x", "dt", "B", "C", "z")}
    S = p["S0"].expand(B, W, N).contiguous()
    y = torch.empty_like(rows["x"])
    channels.seed_selective_step(rows["x"], rows["dt"], p["A"], rows["B"], rows["C"], y, S, D=p["D"], z=rows["z"],
                                 dt_bias=p["dt_bias"])
    one = torch.empty_like(p["S0"])
    out = torch.empty(1, W, device="cuda", dtype=torch.bfloat16)
    channels.seed_selective_step(*(p[k] for k in NAMES[:5]), out, one, D=p["D"], z=p["z"], dt_bias=p["dt_bias"],
                                 S0=p["S0"])
    for b in (0, 1, B // 2, B - 1):
        assert torch.equal(S[b], one[0]) and torch.equal(y[b], out[0])
    held = torch.randn(1, 3, W, device="cuda").bfloat16()
    many, w = held.repeat(8000, 1, 1), torch.randn(W, 4, device="cuda")     # 3.1e9 values
    x = p["x"].expand(8000, W).contiguous()
    y = torch.empty_like(x)
    channels.seed_short_conv_step(x, w, y, many)
    channels.seed_short_conv_step(p["x"].contiguous(), w, out, held)
    for b in (0, 7999):
        assert torch.equal(many[b], held[0]) and torch.equal(y[b], out[0])


@pytest.mark.parametrize("in_place", [True, False])
def test_step_of_many_requests(in_place):
    """States of 32 MB and more are stored past the caches: the same values as
    from calls of a few requests each, two steps running."""
    batch, channels_, d_state = 131, 4096, 16     # 34 MB, an odd batch
    gen = torch.Generator("cuda").manual_seed(7)

    def normal(*s):
        return torch.randn(*s, device="cuda", generator=gen)

    A = -torch.exp(normal(channels_, d_state))
    S = normal(batch, channels_, d_state)
    want = S.clone()
    for _ in range(2):
        x, dt, z = (normal(batch, channels_).bfloat16() for _ in range(3))
        B, C = (normal(batch, 1, d_state).bfloat16() for _ in range(2))
        y, y_want = torch.empty_like(x), torch.empty_like(x)
        S0, S = S, S if in_place else torch.empty_like(S)
        channels.seed_selective_step(x, dt, A, B, C, y, S, z=z, S0=S0)
        for lo in range(0, batch, 50):
            p = slice(lo, min(lo + 50, batch))
            channels.seed_selective_step(x[p], dt[p], A, B[p], C[p], y_want[p], want[p], z=z[p])
        assert torch.equal(y, y_want) and torch.equal(S, want)
